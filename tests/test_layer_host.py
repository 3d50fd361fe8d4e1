"""The decoder-layer entry points without a GPU: they reject bad arguments on the host before touching
a device, and qg_rope_turns computes its table there."""
import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def qg():
    from gguf_block_quantized_quant_gb300 import build
    build.build()
    import gguf_block_quantized_quant_gb300 as m
    m.lib()
    return m


A = 0x10000  # fake, never dereferenced


class Paged(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("type", "kv_heads", "dim", "page", "n_pages", "batch", "table_width", "pad")] +
                [(n, ctypes.c_int64) for n in ("page_stride", "head_stride", "slot_stride", "step_stride", "table_stride")] +
                [(n, ctypes.c_void_p) for n in ("k", "v", "kd", "vd", "q_start", "kv_len", "pages")])


def cache(**kw):
    f = dict(type=1, kv_heads=2, dim=128, page=16, n_pages=4, batch=1, table_width=2, pad=0, page_stride=4096, head_stride=2048,
             slot_stride=128, step_stride=128, table_stride=2, k=A, v=A, kd=None, vd=None, q_start=A, kv_len=A, pages=A)
    f.update(kw)
    return Paged(**f)


def test_struct_matches_the_header():
    assert ctypes.sizeof(Paged) == 8 * 4 + 5 * 8 + 7 * 8


BAD_CACHES = [(dict(type=0), -1), (dict(type=2), -1), (dict(kv_heads=0), -1), (dict(dim=96), -1), (dict(page=8), -1), (dict(page=24), -1),
              (dict(n_pages=0), -1), (dict(batch=0), -1), (dict(table_width=0), -1), (dict(table_stride=1), -1), (dict(k=None), -1),
              (dict(kv_len=None), -1), (dict(pages=None), -1), (dict(type=8), -1), (dict(type=8, kd=A, vd=A, step_stride=64), -1),
              (dict(slot_stride=64), -1), (dict(k=A + 8), -3), (dict(head_stride=2052), -3), (dict(pages=A + 2), -3),
              (dict(type=8, kd=A + 4, vd=A), -3)]


def attn(L, c=None, **kw):
    a = dict(q=A, ldq=512, hdq=128, q_type=1, tokens=1, heads=4, max_new=1, scale=1.0, window=0, out=A, out_type=1, lse=None, ws=A, n=1 << 40)
    a.update(kw)
    c = cache() if c is None else c
    p = lambda v: ctypes.c_void_p(v)  # noqa: E731
    return L.qg_attn_paged(p(a["q"]), a["ldq"], a["hdq"], a["q_type"], a["tokens"], a["heads"], a["max_new"], a["scale"], a["window"],
                           p(a["out"]), a["out_type"], p(a["lse"]), bytes(c), p(a["ws"]), a["n"], None)


def rope(L, c=None, **kw):
    a = dict(q=A, ldq=1024, hdq=128, k=A, v=A, in_type=0, tokens=1, heads=4, turns=A, rot=128, pairs=0, amp=1.0, wq=None, wk=None,
             eps=1e-6, out=A)
    a.update(kw)
    c = cache() if c is None else c
    p = lambda v: ctypes.c_void_p(v)  # noqa: E731
    return L.qg_rope_append(p(a["q"]), a["ldq"], a["hdq"], p(a["k"]), 1024, 128, p(a["v"]), 1024, 128, a["in_type"], a["tokens"], a["heads"],
                            p(a["turns"]), a["rot"], a["pairs"], a["amp"], p(a["wq"]), p(a["wk"]), a["eps"], p(a["out"]), bytes(c), None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(qg, kw, status):
    assert attn(qg.lib(), cache(**kw)) == status
    assert rope(qg.lib(), cache(**kw)) == status


def test_attention_arguments(qg):
    L = qg.lib()
    for kw in (dict(q=None), dict(out=None), dict(tokens=0), dict(heads=0), dict(heads=3), dict(q_type=0), dict(q_type=30), dict(out_type=30),
               dict(window=-1), dict(max_new=-1), dict(scale=math.nan), dict(ldq=64), dict(hdq=64)):
        assert attn(L, **kw) == -1, kw
    assert attn(L, cache(type=30), q_type=1) == -1  # fp16 queries beside a bf16 cache
    for kw in (dict(q=A + 8), dict(ldq=516), dict(out=A + 4), dict(lse=A + 2), dict(ws=A + 8)):
        assert attn(L, **kw) == -3, kw
    assert attn(L, ws=None) == -2
    need = qg.qg_attn_workspace_size(128, 4, 2, 1, 1)
    assert attn(L, n=need - 1) == -2


def test_rope_arguments(qg):
    L = qg.lib()
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(in_type=8), dict(tokens=0), dict(heads=0), dict(heads=3),
               dict(rot=3), dict(rot=130), dict(rot=-2), dict(turns=None), dict(eps=-1.0), dict(hdq=64)):
        assert rope(L, **kw) == -1, kw
    for kw in (dict(q=A + 4), dict(ldq=1026), dict(out=A + 8), dict(turns=A + 4), dict(wq=A + 2)):
        assert rope(L, **kw) == -3, kw


def test_row_counts_beyond_32_bits(qg):
    L = qg.lib()
    assert attn(L, tokens=1 << 29, heads=4, n=1 << 60) == -1
    assert rope(L, tokens=(1 << 31) - 1, heads=64) == -1


def norm(L, **kw):
    a = dict(y=A, yt=0, ldy=64, res=A, rt=0, ldr=64, wpost=None, gate=None, ldg=0, wpre=A, eps=1e-6, ro=A, xo=A, xt=0, M=2, H=64)
    a.update(kw)
    p = lambda v: ctypes.c_void_p(v)  # noqa: E731
    return L.qg_norm_residual(p(a["y"]), a["yt"], a["ldy"], p(a["res"]), a["rt"], a["ldr"], p(a["wpost"]), p(a["gate"]), a["ldg"], p(a["wpre"]),
                              0.0, 1.0, a["eps"], p(a["ro"]), p(a["xo"]), a["xt"], a["M"], a["H"], None)


def test_norm_arguments(qg):
    L = qg.lib()
    for kw in (dict(y=None), dict(ro=None, xo=None), dict(M=0), dict(H=0), dict(H=16385, ldy=20000, ldr=20000), dict(yt=8), dict(xt=8),
               dict(rt=1), dict(ldy=32), dict(ldr=32), dict(gate=A, ldg=32), dict(wpre=None), dict(eps=-1.0), dict(ldr=128)):
        # rows of res apart from those of res_out, in place
        assert norm(L, **kw) == -1, kw
    for kw in (dict(y=A + 2), dict(res=A + 1, ro=A + 64), dict(xo=A + 2), dict(wpre=A + 1)):
        assert norm(L, **kw) == -3, kw


def test_workspace_sizes(qg):
    ok = qg.qg_attn_workspace_size(128, 32, 8, 100, 4)
    assert 0 < ok < qg.qg_attn_workspace_size(128, 32, 8, 1 << 20, 4)
    for bad in ((96, 8, 8, 1, 1), (128, 7, 2, 1, 1), (128, 0, 1, 1, 1), (128, 8, 0, 1, 1), (128, 8, 8, 0, 1), (128, 8, 8, 1, 0)):
        assert qg.qg_attn_workspace_size(*bad) == qg.WS_INVALID


def test_rope_turns_table(qg):
    turns, amp = qg.qg_rope_turns(128, 10000.0)
    f = turns.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    assert amp == 1.0 and np.allclose(f, 10000.0 ** (-np.arange(64) / 64), rtol=1e-13, atol=0)
    with pytest.raises(qg.QGError):
        qg.qg_rope_turns(128, 10000.0, qg.ROPE_YARN, 0.5)
