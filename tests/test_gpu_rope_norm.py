"""qg_rope_append, qg_rope_turns and qg_norm_residual against their formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

from layer_testlib import BF16, F16, F32, UNIT, gen, make_cache, tables, values, within
from qg_testlib import qg_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    return qg_module()


def rotate(x, pos, turns, amp, pairs):
    """x (tokens, heads, dim) in 64 bits, rotated; the phase by integers, exact at any position."""
    half = len(turns)
    ph = np.array([[(int(p) * int(t)) % (1 << 64) for t in turns] for p in pos], dtype=object)
    ang = torch.tensor((ph / float(1 << 64)).astype(np.float64), device=x.device) * (2 * math.pi)
    c, s = amp * torch.cos(ang)[:, None], amp * torch.sin(ang)[:, None]
    i, j = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    y = x.clone()
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    return y


def rope_check(qg, kind, src, D, H, Hk, rot, pairs, page, new, kv_len, norm=False, amp=1.0, seed=1, nhd=False, base=10000.0, fused=True):
    g = gen(seed)
    q_start, lens, pages, n_pages = tables(new, kv_len, page, 2, g)
    k, v, kd, vd = make_cache(kind, n_pages, Hk, page, D, g, nhd)
    dt = BF16 if kind == BF16 else F16
    T = sum(new)
    qkv = torch.randn((T, H + 2 * Hk, D), generator=g, device="cuda").to(src)
    q, nk, nv = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    if not fused:
        q, nk, nv = q.contiguous(), nk.contiguous(), nv.contiguous()
    turns = None
    if rot:
        turns, _ = qg.qg_rope_turns(rot, base)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")) for _ in range(2)) if norm else (None, None)
    before = [None if t is None else t.clone() for t in (k, v, kd, vd)]
    got = qg.qg_rope_append(q, nk, nv, None if turns is None else turns.cuda(), k, v, q_start, lens, pages, kd=kd, vd=vd,
                            pairs=pairs, amp=amp, wq=wq, wk=wk)
    torch.cuda.synchronize()

    x = {}
    for name, t, w in (("q", q, wq), ("k", nk, wk)):
        t = t.double()
        if w is not None:
            t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w.double()
        x[name] = t
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(new, kv_len)] + [np.zeros(0)]).astype(np.int64)
    table = [] if turns is None else turns.numpy().view(np.uint64).tolist()
    rq, rk = (rotate(x[n], pos, table, amp, pairs) if rot else x[n] for n in ("q", "k"))
    # fp32: the norm, sine and products, a few roundings of a pair's largest terms; then one rounding
    reach = max(1.0, amp)
    mag = lambda t: reach * t.abs().amax(-1, keepdim=True)  # noqa: E731
    ok = torch.from_numpy(pos >= 0).cuda()
    want = torch.where(ok[:, None, None], rq, 0.0)
    within(got, want, UNIT[dt] * want.abs() + 2.0 ** -20 * mag(x["q"]) + 2.0 ** -24, "q")
    # every slot that was not written keeps its bits
    seq = np.repeat(np.arange(len(new)), new)
    live = pos >= 0
    pg = pages.cpu().numpy()[seq[live], pos[live] // page]
    where = (torch.from_numpy(pg).long().cuda(), torch.from_numpy(pos[live] % page).cuda())
    for pool, steps, old, old_steps, t, m in ((k, kd, before[0], before[2], rk, mag(x["k"])), (v, vd, before[1], before[3], nv.double(), 0)):
        written = torch.zeros((n_pages, page), dtype=torch.bool, device="cuda")
        written[where] = True
        keep = ~written[:, None].expand(-1, Hk, -1)
        same = lambda a, b: torch.equal(a[keep].view(torch.int8), b[keep].view(torch.int8))  # noqa: E731
        assert same(pool, old)
        if steps is not None:
            assert same(steps, old_steps)
        have = values(pool, steps)[where[0], :, where[1]]
        t = t[ok]
        slack = 2.0 ** -20 * (m[ok] if torch.is_tensor(m) else t.abs())
        if kind == "q8":
            d = (t.reshape(t.shape[0], Hk, -1, 32).abs().amax(-1) / 127).repeat_interleave(32, -1)
            # half a step, the fp16 rounding of the step under a code of up to 127, the fp32 work
            bound = (0.5 + 127 * 2.0 ** -11 + 2.0 ** -10) * d + slack + 127 * 2.0 ** -25
            assert int(pool.view(torch.int8).min()) >= -127
        else:
            bound = UNIT[kind] * t.abs() + slack + 2.0 ** -24
        within(have, t, bound, "cache")


KINDS = [F16, BF16, "q8"]
IDS = ["f16", "bf16", "q8"]


@pytest.mark.parametrize("pairs", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_rope_types_and_dims(qg, kind, D, pairs):
    for src in (F32, BF16 if kind == BF16 else F16):
        rope_check(qg, kind, src, D, 4, 2, D, pairs, 16, [1, 5, 1], [1, 9, 40])
        rope_check(qg, kind, src, D, 4, 2, D // 4, pairs, 32, [1, 5, 1], [1, 9, 40], norm=True)


@pytest.mark.parametrize("rot", [0, 2, 6, 10, 30, 62, 64, 100, 126, 128])
@pytest.mark.parametrize("pairs", [False, True], ids=["half", "pairs"])
def test_rope_part_of_the_head(qg, rot, pairs):
    rope_check(qg, F16, F32, 128, 3, 1, rot, pairs, 16, [3, 2], [20, 2], norm=True, seed=rot)
    rope_check(qg, "q8", F32, 128, 6, 2, rot, pairs, 16, [3, 2], [20, 2], amp=1.2, seed=rot)


def test_rope_far_positions(qg):
    """Phases stay exact where a 32-bit angle would have lost its fraction of a turn."""
    for D in (64, 128):
        g = gen(3)
        page, n = 64, 1 << 14
        width = (1 << 20) // page
        k, v, _, _ = make_cache(F16, 4, 1, page, D, g)
        pages = torch.zeros((1, width), dtype=torch.int32, device="cuda")
        turns, _ = qg.qg_rope_turns(D, 10000.0)
        x = torch.randn((2, 1, D), generator=g, device="cuda")
        L = (1 << 20) - 3
        q = qg.qg_rope_append(x, x, x, turns.cuda(), k, v, torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
                              torch.tensor([L], dtype=torch.int32, device="cuda"), pages)
        want = rotate(x.double(), np.array([L - 2, L - 1]), turns.numpy().view(np.uint64).tolist(), 1.0, False)
        within(q, want, UNIT[F16] * want.abs() + 2.0 ** -20 * x.double().abs().amax(-1, keepdim=True), "far")


def test_rope_ragged_batches(qg):
    rope_check(qg, F16, F32, 128, 8, 2, 128, False, 16, [0, 1, 0, 0, 7, 3, 0], [0, 1, 5, 0, 4, 3, 9])     # padding rows
    rope_check(qg, BF16, F32, 64, 2, 2, 64, True, 48, [1] * 1500, [1 + (i * 7) % 60 for i in range(1500)])
    rope_check(qg, "q8", F32, 128, 32, 8, 128, False, 64, [300, 700], [300, 1100], norm=True)
    rope_check(qg, F16, F32, 256, 16, 2, 64, False, 32, [33], [64], fused=False)
    for kind in KINDS:
        rope_check(qg, kind, F32, 128, 4, 4, 128, False, 16, [9, 1], [50, 17], nhd=True)


def test_rope_gated_query_layout(qg):
    """Queries beside gates: heads 2 * dim apart."""
    g = gen(6)
    q_start, lens, pages, n = tables([4], [20], 16, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 16, 128, g)
    wide = torch.randn((4, 8, 256), generator=g, device="cuda")
    kv = torch.randn((4, 2, 2, 128), generator=g, device="cuda")
    turns = qg.qg_rope_turns(128)[0].cuda()
    a = qg.qg_rope_append(wide[..., :128], kv[:, 0], kv[:, 1], turns, k, v, q_start, lens, pages)
    b = qg.qg_rope_append(wide[..., :128].contiguous(), kv[:, 0].contiguous(), kv[:, 1].contiguous(), turns, k, v, q_start, lens, pages)
    assert torch.equal(a, b)


@pytest.mark.parametrize("src", [F32, F16], ids=["f32", "f16"])
@pytest.mark.parametrize("off", [(2, 0, 0), (0, 2, 0), (0, 0, 2)])
@pytest.mark.parametrize("D,pairs", [(64, False), (64, True), (128, False), (256, True)])
def test_rope_heads_off_a_vector_boundary(qg, src, off, D, pairs):
    """Heads that start, or lie, dim / 32 elements off a boundary of four: a view's base, token stride or head stride."""
    g = gen(8)
    q_start, lens, pages, n = tables([5, 1], [20, 1], 16, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 16, D, g)
    base, row, head = (o * D // 64 for o in off)
    hd = D + head
    ld = 8 * hd + row
    buf = torch.randn(base + 6 * ld, generator=g, device="cuda").to(src)
    x = torch.as_strided(buf, (6, 8, D), (ld, hd, 1), base)
    turns = qg.qg_rope_turns(D)[0]
    got = qg.qg_rope_append(x[:, :4], x[:, 4:6], x[:, 6:], turns.cuda(), k, v, q_start, lens, pages, pairs=pairs)
    pos = np.concatenate([np.arange(15, 20), np.zeros(1)]).astype(np.int64)
    want = rotate(x.double(), pos, turns.numpy().view(np.uint64).tolist(), 1.0, pairs)
    slack = 2.0 ** -20 * x.double().abs().amax(-1, keepdim=True) + 2.0 ** -24
    bound = UNIT[F16] * want.abs() + slack
    within(got, want[:, :4], bound[:, :4], "q")
    pg = pages.cpu().numpy()[[0] * 5 + [1], pos // 16]
    where = (torch.from_numpy(pg).long().cuda(), torch.from_numpy(pos % 16).cuda())
    within(values(k, None)[where[0], :, where[1]], want[:, 4:6], bound[:, 4:6], "k")
    want = x[:, 6:].double()
    within(values(v, None)[where[0], :, where[1]], want, UNIT[F16] * want.abs() + 2.0 ** -24, "v")


def test_rope_zero_and_extreme_blocks_of_q8(qg):
    g = gen(7)
    q_start, lens, pages, n = tables([2], [2], 16, 0, g)
    k, v, kd, vd = make_cache("q8", n, 1, 16, 64, g)
    x = torch.zeros((2, 1, 64), device="cuda")
    x[1, 0, 3], x[1, 0, 40] = 6e4, -1e-3
    qg.qg_rope_append(x, x, x, None, k, v, q_start, lens, pages, kd=kd, vd=vd)
    got = values(v, vd)[pages[0, 0].long(), 0, :2]
    assert (got[0] == 0).all()
    assert abs(got[1, 3].item() - 6e4) <= 6e4 * 2.0 ** -11 and abs(got[1, 40].item() + 1e-3) <= 1e-3 * 2.0 ** -6
    assert (got[1, 4:40] == 0).all()


@pytest.mark.parametrize("scaling", ["plain", "linear", "ntk", "yarn"])
def test_rope_turns(qg, scaling):
    rot, base, factor, original = 64, 500000.0, 4.0, 8192.0
    kind = {"plain": qg.ROPE_PLAIN, "linear": qg.ROPE_LINEAR, "ntk": qg.ROPE_NTK, "yarn": qg.ROPE_YARN}[scaling]
    turns, amp = qg.qg_rope_turns(rot, base, kind, factor, original)
    j = np.arange(rot // 2)
    b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" else base
    f = b ** (-2.0 * j / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        edge = lambda turn: rot * math.log(original / (turn * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(edge(32)), 0), min(math.ceil(edge(1)), rot // 2 - 1)
        ramp = np.clip((j - lo) / (hi - lo), 0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        assert abs(amp - (0.1 * math.log(4.0) + 1)) < 1e-6
    else:
        assert amp == 1.0
    got = turns.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    assert np.allclose(got, f, rtol=1e-13, atol=0)


def test_rope_refusals(qg):
    g = gen(8)
    q_start, lens, pages, n = tables([1], [4], 16, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 16, 128, g)
    q, kv = torch.randn((1, 4, 128), device="cuda"), torch.randn((1, 2, 128), device="cuda")
    turns = qg.qg_rope_turns(128)[0].cuda()
    ok = (q, kv, kv, turns, k, v, q_start, lens, pages)
    qg.qg_rope_append(*ok)
    for i, bad in ((0, q.half()), (1, kv[..., :64]), (0, q.cpu()), (3, turns.int()), (3, torch.zeros(65, dtype=torch.int64, device="cuda")),
                   (4, k.float()), (6, q_start.long()), (0, q[:, :3])):
        args = list(ok)
        args[i] = bad
        with pytest.raises((ValueError, qg.QGError)):
            qg.qg_rope_append(*args)
    with pytest.raises(ValueError):
        qg.qg_rope_append(*ok, q_dtype=BF16)
    for kw in (dict(rot=3), dict(rot=0), dict(rot=64, base=0.5), dict(rot=64, scaling=qg.ROPE_LINEAR, factor=0.5), dict(rot=64, scaling=9)):
        with pytest.raises(qg.QGError):
            qg.qg_rope_turns(**kw)


# ------------------------------------------------------------------------------------- norms
def norm_check(qg, M, H, ydt, rdt, xdt, post=False, gate=None, alpha=1.0, w_offset=0.0, res=True, seed=1, pad=0, scale=1.0):
    g = gen(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    y = (scale * rand(M, H + pad)).to(ydt)[:, :H]
    r0 = (2 * rand(M, H + pad)).to(rdt)[:, :H] if res else None
    w_pre, w_post = 1 + 0.2 * rand(H) - w_offset, 1 + 0.2 * rand(H) - w_offset
    gt = None if gate is None else rand(M, H).to(ydt) if gate == "rows" else rand(H).to(ydt)
    r, x = qg.qg_norm_residual(y, r0, w_pre, w_post=w_post if post else None, gate=gt, alpha=alpha, eps=1e-6, w_offset=w_offset, x_dtype=xdt)
    torch.cuda.synchronize()
    t = y.double()
    rms = lambda a, w: a / torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-6) * (w_offset + w.double())  # noqa: E731
    if post:
        t = rms(t, w_post)
    if gt is not None:
        t = t * gt.double()
    want = alpha * t + (r0.double() if res else 0)
    # about ten fp32 roundings of the terms of the sum, then the output's own
    terms = abs(alpha) * t.abs() + (r0.double().abs() if res else 0)
    within(r, want, UNIT[r.dtype] * want.abs() + 10 * 2.0 ** -24 * terms + 2.0 ** -24, "r")
    xw = rms(want, w_pre)
    k = (xw / torch.where(want == 0, 1.0, want)).abs()
    within(x, xw, UNIT[x.dtype] * xw.abs() + 20 * 2.0 ** -24 * (xw.abs() + k * terms) + 2.0 ** -24, "x")
    assert r.dtype == (rdt if res else ydt) and x.dtype == xdt


@pytest.mark.parametrize("xdt", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("ydt,rdt", [(F32, F32), (F16, F32), (F16, F16), (BF16, F32), (BF16, BF16)])
def test_norm_types(qg, ydt, rdt, xdt):
    for M, H in ((1, 5120), (7, 2048), (3, 333)):
        norm_check(qg, M, H, ydt, rdt, xdt)
        norm_check(qg, M, H, ydt, rdt, xdt, post=True, gate="rows", alpha=0.5)


@pytest.mark.parametrize("H", [1, 2, 3, 4, 31, 32, 100, 127, 128, 129, 512, 516, 1000, 1023, 4096, 4097, 5121, 8192, 16380, 16383, 16384])
def test_norm_widths(qg, H):
    for M in (1, 2, 9, 130):
        norm_check(qg, M, H, F32, F32, F32, post=True, gate="row", alpha=0.7, w_offset=1.0, seed=H)


def test_norm_options(qg):
    norm_check(qg, 5, 2048, F32, F32, F32, res=False)
    norm_check(qg, 5, 2048, F16, F16, F32, res=False, post=True)
    norm_check(qg, 65, 640, BF16, F32, BF16, pad=8, post=True)       # rows apart
    norm_check(qg, 65, 640, F32, F32, F16, pad=3)                    # and off the vector boundary
    norm_check(qg, 3000, 96, F32, F32, F32, alpha=-2.0)
    norm_check(qg, 2, 5120, F32, F32, F32, scale=1e-6)               # eps counts
    norm_check(qg, 2, 5120, F32, F32, F32, scale=1e15)


def test_norm_in_place_zero_rows_and_streams(qg):
    g = gen(4)
    y, res = torch.randn((33, 2048), generator=g, device="cuda"), torch.randn((33, 2048), generator=g, device="cuda")
    y[3], res[3] = 0, 0
    w = torch.ones(2048, device="cuda")
    want_r, want_x = qg.qg_norm_residual(y, res, w, w_post=w)
    assert (want_x[3] == 0).all() and (want_r[3] == 0).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mine = res.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r, x = qg.qg_norm_residual(y, mine, w, w_post=w, res_out=mine)
    side.synchronize()
    assert r is mine and torch.equal(r, want_r) and torch.equal(x, want_x)
    r, x = qg.qg_norm_residual(y, res, None)  # the sum alone
    assert x is None and torch.equal(r, res + y)


def test_norm_refusals(qg):
    y, w = torch.randn((2, 64), device="cuda"), torch.ones(64, device="cuda")
    for a, kw in (((y, y.half(), w), {}), ((y, y[:1], w), {}), ((y, y, w.half()), {}), ((y, y, w[:32]), {}), ((y.t(), None, w), {}),
                  ((y, y, w), dict(gate=y.half())), ((y, y, w), dict(eps=-1.0)), ((y.cpu(), None, w), {}),
                  ((torch.randn((1, 16385), device="cuda"), None, torch.ones(16385, device="cuda")), {})):
        with pytest.raises((ValueError, qg.QGError)):
            qg.qg_norm_residual(*a, **kw)
