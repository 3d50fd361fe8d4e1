"""The entry points of shaped and tree attention, trees, kept drafts and logits without a GPU: they reject bad arguments on the host
before touching a device."""
import ctypes
import math

import pytest

from test_layer_host import A, BAD_CACHES, cache, qg  # noqa: F401  (qg: the module's fixture)

P = ctypes.c_void_p
EINVAL, EWORKSPACE, EALIGN = -1, -2, -3


def attn(L, name, c=None, **kw):
    a = dict(q=A, ldq=512, hdq=128, q_type=1, tokens=1, heads=4, max_new=1, scale=1.0, window=0, cap=0.0, slopes=None, prefix=None, first=None,
             tree=A, words=1, positions=None, out=A, out_type=1, lse=None, ws=A, n=1 << 40)
    a.update(kw)
    c = cache() if c is None else c
    own = [P(a["prefix"]), P(a["first"])] if name == "shaped" else [P(a["tree"]), a["words"], P(a["positions"])]
    return getattr(L, f"qg_attn_{name}")(P(a["q"]), a["ldq"], a["hdq"], a["q_type"], a["tokens"], a["heads"], a["max_new"], a["scale"], a["window"],
                                         a["cap"], P(a["slopes"]), *own, P(a["out"]), a["out_type"], P(a["lse"]), bytes(c), P(a["ws"]), a["n"], None)


@pytest.mark.parametrize("name", ["shaped", "tree"])
def test_attention(qg, name):  # noqa: F811
    L = qg.lib()
    for kw, status in BAD_CACHES:
        assert attn(L, name, cache(**kw)) == status
    for kw in (dict(q=None), dict(out=None), dict(tokens=0), dict(heads=0), dict(heads=3), dict(q_type=0), dict(out_type=30), dict(window=-1),
               dict(max_new=-1), dict(scale=math.nan), dict(ldq=64), dict(cap=-1.0), dict(cap=math.nan), dict(cap=math.inf), dict(cap=1e-39),
               dict(cap=3e38), dict(cap=1.0, scale=math.inf), dict(cap=1e-30, scale=1e30)):
        assert attn(L, name, **kw) == EINVAL, kw
    for kw in (dict(q=A + 8), dict(ldq=516), dict(out=A + 4), dict(lse=A + 2), dict(ws=A + 8), dict(slopes=A + 2)):
        assert attn(L, name, **kw) == EALIGN, kw
    for kw in ((dict(prefix=A + 1), dict(first=A + 2)) if name == "shaped" else (dict(tree=A + 1), dict(positions=A + 2))):
        assert attn(L, name, **kw) == EALIGN, kw
    if name == "tree":
        assert attn(L, name, tree=None) == EINVAL and attn(L, name, words=0) == EINVAL
    assert attn(L, name, ws=None) == EWORKSPACE
    assert attn(L, name, n=qg.qg_attn_workspace_size(128, 4, 2, 1, 1) - 1) == EWORKSPACE
    assert attn(L, name, tokens=1 << 29, heads=4, n=1 << 60) == EINVAL


def test_tree_masks(qg):  # noqa: F811
    ok = dict(parents=A, q_start=A, kv_len=A, tokens=3, batch=1, tree=A, words=1, positions=A)

    def call(**kw):
        a = dict(ok, **kw)
        return qg.lib().qg_tree_masks(P(a["parents"]), P(a["q_start"]), P(a["kv_len"]), a["tokens"], a["batch"], P(a["tree"]), a["words"],
                                      P(a["positions"]), None)
    for kw in (dict(parents=None), dict(q_start=None), dict(kv_len=None), dict(tree=None), dict(positions=None), dict(tokens=0), dict(batch=0),
               dict(words=0), dict(words=33), dict(batch=(1 << 31) - 1)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(parents=A + 2), dict(tree=A + 1), dict(positions=A + 3)):
        assert call(**kw) == EALIGN, kw


def test_cache_keep(qg):  # noqa: F811
    ok = dict(keep=A, stride=4, keep_len=A, width=4, layers=1, apart=0, steps=0, kv_out=A)

    def call(c=None, **kw):
        a = dict(ok, **kw)
        return qg.lib().qg_cache_keep(P(a["keep"]), a["stride"], P(a["keep_len"]), a["width"], a["layers"], a["apart"], a["steps"], P(a["kv_out"]),
                                      bytes(cache() if c is None else c), None)
    for kw, status in BAD_CACHES:
        assert call(cache(**kw)) == status
    for kw in (dict(keep=None), dict(keep_len=None), dict(kv_out=None), dict(width=0), dict(width=1025, stride=2000), dict(stride=3), dict(layers=0),
               dict(layers=65536), dict(layers=2, apart=0)):
        assert call(**kw) == EINVAL, kw
    assert call(cache(type=8, kd=A, vd=A), layers=2, apart=4096, steps=0) == EINVAL
    assert call(cache(batch=65536)) == EINVAL
    for kw in (dict(keep=A + 2), dict(keep_len=A + 1), dict(kv_out=A + 3), dict(layers=2, apart=4100)):
        assert call(**kw) == EALIGN, kw
    assert call(cache(type=8, kd=A, vd=A), layers=2, apart=4096, steps=260) == EALIGN


class Logits(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("batch", "words", "history_width", "bias_entries")] +
                [(n, P) for n in ("seq", "history", "history_len", "prompt_len")] + [("history_stride", ctypes.c_int64)] +
                [(n, P) for n in ("repetition", "frequency", "presence", "bias_start", "bias_ids", "bias", "allow")] + [("allow_stride", ctypes.c_int64)] +
                [(n, P) for n in ("drafts", "tree", "q_start")])


def test_logits(qg):  # noqa: F811
    how = dict(batch=1, words=1, history_width=8, bias_entries=1, history=A, history_len=A, history_stride=8, repetition=A, frequency=A, presence=A,
               bias_start=A, bias_ids=A, bias=A, allow=A, allow_stride=4, drafts=A, tree=A, q_start=A)
    ok = dict(x=A, type=0, ld=128, out=A + 4096, out_type=0, ldo=128, rows=1, V=128)

    def call(h=None, **kw):
        a, s = dict(ok, **kw), Logits(**dict(how, **(h or {})))
        return qg.lib().qg_logits_adjust(P(a["x"]), a["type"], a["ld"], P(a["out"]), a["out_type"], a["ldo"], a["rows"], a["V"], bytes(s), None)
    for kw in (dict(x=None), dict(out=None), dict(type=8), dict(out_type=2), dict(rows=0), dict(V=0), dict(V=(1 << 31) - 1, ld=1 << 31, ldo=1 << 31),
               dict(ld=127), dict(ldo=127), dict(out=A, ldo=256), dict(out=A, out_type=1), dict(rows=(1 << 31) - 1, V=9000, ld=9000, ldo=9000)):
        assert call(**kw) == EINVAL, kw
    for h in (dict(batch=0), dict(batch=-1), dict(history_len=None), dict(history_stride=-1), dict(history_width=-1), dict(drafts=None), dict(tree=None),
              dict(q_start=None), dict(words=0), dict(bias_ids=None), dict(bias=None), dict(bias_entries=-1), dict(allow_stride=3)):
        assert call(h) == EINVAL, h
    assert qg.lib().qg_logits_adjust(P(A), 0, 128, P(A + 4096), 0, 128, 1, 128, None, None) == EINVAL
    for kw in (dict(x=A + 2), dict(out=A + 4098), dict(type=1, x=A + 1)):
        assert call(**kw) == EALIGN, kw
    for name in ("seq", "history", "history_len", "prompt_len", "repetition", "bias_start", "bias_ids", "bias", "allow", "drafts", "tree", "q_start"):
        assert call({name: A + 2}) == EALIGN, name


def test_rotary_positions(qg):  # noqa: F811
    def call(positions):
        return qg.lib().qg_rope_append_at(P(A), 1024, 128, P(A), 1024, 128, P(A), 1024, 128, 0, 1, 4, P(A), 128, 0, 1.0, None, None, 1e-6,
                                          P(positions), P(A), bytes(cache()), None)
    assert call(A + 2) == EALIGN
