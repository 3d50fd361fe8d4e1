"""qg_logits_adjust, qg_cache_keep and rotary positions beside the slots, against plain forms."""
import math
import random

import numpy as np
import pytest
import torch

from draft_testlib import ancestors, words_of
from layer_testlib import BF16, F16, F32, UNIT, gen, make_cache, tables
from qg_testlib import qg_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    return qg_module()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------- logits
def plain(x, case):
    """The logits in 64 bits, and the sum of magnitudes that their rounding errors are relative to."""
    y = x.double().cpu()
    mag = y.abs().nan_to_num(0.0, 0.0, 0.0)
    rows, V = y.shape
    for r in range(rows):
        s = case["seq"][r] if case.get("seq") else r
        if 0 <= s < case["batch"]:
            if case.get("bias"):
                for i, v in dict(case["bias"][s]).items():  # the last entry of an id counts
                    if 0 <= i < V:
                        y[r, i] += v
                        mag[r, i] += abs(v)
            said, count = set(), {}
            if case.get("history"):
                h, p = case["history"][s], case["prompt"][s] if case.get("prompt") else 0
                said |= set(h)
                for i in h[max(p, 0):]:
                    count[i] = count.get(i, 0) + 1
            if case.get("tree"):
                lo, hi = case["q_start"][s], case["q_start"][s + 1]
                for j in range(min(hi - lo, 32 * case["words"])):
                    if case["tree"][r] >> j & 1:
                        i = case["drafts"][lo + j]
                        said.add(i)
                        count[i] = count.get(i, 0) + 1
            rep, freq, pres = (case[w][s] if case.get(w) else d for w, d in (("repetition", 1.0), ("frequency", 0.0), ("presence", 0.0)))
            for i in said:
                if 0 <= i < V:
                    f = 1 / rep if y[r, i] > 0 else rep
                    y[r, i] *= f
                    mag[r, i] *= f
            for i, n in count.items():
                if 0 <= i < V:
                    y[r, i] -= freq * n + pres
                    mag[r, i] += abs(freq) * n + abs(pres)
        if case.get("allow"):
            bits = np.frombuffer(case["allow"][r].to_bytes(-(-V // 8), "little"), dtype=np.uint8)
            y[r, torch.from_numpy(np.unpackbits(bits, bitorder="little")[:V] == 0)] = -math.inf
    return y.cuda(), mag.cuda()


def f32(values):
    return torch.tensor(values, dtype=torch.float32).tolist()


def make(seed, rows, V, batch=None, drafts=False, bias=True, allow=True, longest=300, wild=True, words=1):
    r = random.Random(seed)
    batch = rows if batch is None else batch
    ids = lambda n: [r.randrange(-2 if wild else 0, V + 3 if wild else V) if r.random() < 0.2 else r.randrange(min(V, 40)) for _ in range(n)]  # noqa: E731
    c = {"batch": batch, "history": [ids(r.randrange(longest)) for _ in range(batch)],
         "repetition": f32([r.uniform(0.6, 2) for _ in range(batch)]), "frequency": f32([r.uniform(-0.2, 0.5) for _ in range(batch)]),
         "presence": f32([r.uniform(-0.2, 0.5) for _ in range(batch)])}
    c["prompt"] = [r.randrange(-1, len(h) + 3) for h in c["history"]]
    if batch != rows or drafts:
        cut = sorted(r.randrange(rows + 1) for _ in range(batch - 1))
        c["q_start"] = [0] + cut + [rows]
        c["seq"] = [max(s for s in range(batch) if c["q_start"][s] <= i) for i in range(rows)]
        if wild and rows > 3:
            c["seq"][1], c["seq"][2] = -1, batch
    if drafts:
        c["drafts"], c["tree"], c["words"] = ids(rows), [], words
        for s in range(batch):
            n = c["q_start"][s + 1] - c["q_start"][s]
            c["tree"] += ancestors([r.randrange(-1, i) if i else -1 for i in range(n)])[0]
        c["tree"] = [t & (1 << 32 * words) - 1 for t in c["tree"]]
    if bias:
        c["bias"] = [list(zip(ids(n), f32([r.uniform(-5, 5) for _ in range(n)]))) for n in (r.choice([0, 1, 7, 60]) for _ in range(batch))]
    if allow:
        c["allow"] = [r.choice([r.getrandbits(V), 0, (1 << V) - 1, 1 << V - 1]) for _ in range(rows)]
    return c


def call(qg, x, c, **kw):
    rows, V = x.shape
    a = {}
    if c.get("seq"):
        a["seq"] = ints(c["seq"])
    if c.get("history"):
        width = max(1, max(map(len, c["history"])))
        a["history"] = ints([h + [5] * (width - len(h)) for h in c["history"]])  # past the length: not read
        a["history_len"] = ints([len(h) for h in c["history"]])
        if c.get("prompt"):
            a["prompt_len"] = ints(c["prompt"])
    for w in ("repetition", "frequency", "presence"):
        if c.get(w):
            a[w] = torch.tensor(c[w], device="cuda")
    if c.get("bias"):
        start = [0]
        for b in c["bias"]:
            start.append(start[-1] + len(b))
        a["bias_start"] = ints(start)
        a["bias_ids"] = ints([i for b in c["bias"] for i, _ in b])
        a["bias"] = torch.tensor([v for b in c["bias"] for _, v in b], device="cuda", dtype=torch.float32)
    if c.get("allow"):
        a["allow"] = words_of(c["allow"], -(-V // 32))
    if c.get("tree"):
        a.update(drafts=ints(c["drafts"]), tree=words_of(c["tree"], c["words"]), q_start=ints(c["q_start"]))
    return qg.qg_logits_adjust(x, **a, **kw)


def check(qg, x, c, **kw):
    want, mag = plain(x, c)
    got = call(qg, x, c, **kw)
    # up to five roundings of fp32 (bias, quotient, product, difference, difference), then the output type's; halves below
    # their smallest normal number are off by up to 2^-25
    inside = want.to(torch.float32).to(got.dtype)  # values beyond the type's range are infinite there
    fine = torch.isfinite(inside)
    bound = 5 * 2.0 ** -24 * mag + UNIT[got.dtype] * want.abs() + (2.0 ** -24 if got.dtype == F16 else 0.0) + 1e-37
    assert torch.equal(torch.isfinite(got), fine)
    assert torch.equal(got[~fine].double().nan_to_num(7.0, 8.0, 9.0), inside[~fine].double().nan_to_num(7.0, 8.0, 9.0))
    assert ((got.double() - want).abs()[fine] <= bound[fine]).all()
    return got


@pytest.mark.parametrize("out", [F32, F16, BF16])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_types(qg, dtype, out):
    for V in (1, 3, 33, 1000, 1027):
        x = (3 * torch.randn((5, V), generator=gen(V), device="cuda")).to(dtype)
        check(qg, x, make(V, 5, V), out_dtype=out)


@pytest.mark.parametrize("V", [8191, 8192, 8193, 20001, 65536])
@pytest.mark.parametrize("rows", [1, 7])
def test_segments(qg, V, rows):
    """Rows of several segments, whose starts fall off the vectors' boundaries where ids are odd in number."""
    x = 3 * torch.randn((rows, V), generator=gen(V), device="cuda")
    check(qg, x, make(V, rows, V, longest=5000))


@pytest.mark.parametrize("what", ["history", "bias", "allow", "nothing", "no prompt"])
def test_parts(qg, what):
    c = make(3, 6, 777, bias=what == "bias", allow=what == "allow")
    if what not in ("history", "no prompt"):
        for w in ("history", "prompt", "repetition", "frequency", "presence"):
            c.pop(w)
    if what == "no prompt":
        c.pop("prompt")
    x = torch.randn((6, 777), generator=gen(1), device="cuda")
    got = check(qg, x, c)
    if what == "nothing":
        assert torch.equal(got, x)


@pytest.mark.parametrize("words,rows,batch", [(1, 20, 3), (2, 100, 2), (1, 50, 1), (1, 1, 1)])
def test_drafts(qg, words, rows, batch):
    x = torch.randn((rows, 500), generator=gen(rows), device="cuda")
    check(qg, x, make(rows, rows, 500, batch=batch, drafts=True, words=words))


@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, F32), (F16, F32), (F32, BF16), (BF16, F16)])
def test_large_calls_in_two_kernels(qg, dtype, out):
    """Enough rows and ids that the stream has a kernel of its own; rows of a sequence together, apart and of none; in place."""
    V, rows, batch = 20001, 170, 11
    x = (3 * torch.randn((rows, V), generator=gen(7), device="cuda")).to(dtype)
    c = make(70, rows, V, batch=batch, drafts=True, words=1, longest=3000)
    got = check(qg, x, c, out_dtype=out)
    r = random.Random(5)
    for s in range(len(c["seq"])):
        if r.random() < 0.3:
            c["seq"][s] = r.randrange(batch)
    c.pop("tree"), c.pop("drafts")
    check(qg, x, c, out_dtype=out)
    for part in ("bias", "history", "allow"):
        less = {k: v for k, v in c.items() if k != part and not (part == "history" and k == "prompt")}
        check(qg, x, less, out_dtype=out)
    if dtype == out:
        y = x.clone()
        call(qg, y, c, out=y)
        assert torch.equal(y.nan_to_num(7.0), call(qg, x, c, out_dtype=out).nan_to_num(7.0))
        c.pop("allow")
        y = x.clone()
        call(qg, y, c, out=y)
        assert torch.equal(y, call(qg, x, c, out_dtype=out))
    assert got.shape == x.shape


@pytest.mark.parametrize("V", [200, 9000])
def test_many_drafts_of_one_segment(qg, V):
    """A chain of 200 drafts, most of them a few ids: more than a row's list of a segment holds."""
    n = 200
    c = make(3, n, V, batch=1, drafts=True, words=7)
    r = random.Random(1)
    c["drafts"] = [r.choice([5, 6, 7, r.randrange(V)]) for _ in range(n)]
    c["tree"] = [(1 << i + 1) - 1 for i in range(n)]
    c["seq"] = [0] * n
    x = torch.randn((n, V), generator=gen(2), device="cuda")
    check(qg, x, c)
    c.pop("history"), c.pop("prompt"), c.pop("bias")
    check(qg, x, c)


def test_special_values(qg):
    """Infinities, NaN and the least values of the types go through; masked ones become -inf whatever they are."""
    for dtype in (F32, F16, BF16):
        x = torch.randn((4, 640), generator=gen(2), device="cuda").to(dtype)
        x[:, ::7], x[:, 1::7], x[:, 2::7], x[:, 3::7] = math.inf, -math.inf, math.nan, torch.finfo(dtype).min
        check(qg, x, make(9, 4, 640), out_dtype=F32)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_in_place_is_the_same(qg, dtype):
    for V in (64, 1001, 20000):
        for seed in range(3):
            x = (3 * torch.randn((6, V), generator=gen(V), device="cuda")).to(dtype)
            c = make(seed, 6, V, longest=30)
            want = call(qg, x, c, out_dtype=dtype)
            y = x.clone()
            assert call(qg, y, c, out=y) is y
            assert torch.equal(y.nan_to_num(7.0), want.nan_to_num(7.0))


def test_strides_and_starts(qg):
    """Rows apart from each other, off every boundary, and in and out off it differently; nothing beside them is written."""
    c = make(4, 3, 501)
    for shift in range(4):
        for ld in (501, 512, 519):
            for oshift in (0, 3):
                wide = torch.randn((3, ld + 8), generator=gen(shift), device="cuda")
                x = wide.view(-1)[shift:shift + 3 * ld].as_strided((3, 501), (ld, 1), shift)
                big = torch.full((3 * 530,), 77.0, device="cuda")
                out = big.as_strided((3, 501), (520, 1), oshift)
                want = call(qg, x.contiguous(), c)
                call(qg, x, c, out=out)
                assert torch.equal(out, want)
                left = torch.ones_like(big, dtype=torch.bool)
                left.as_strided((3, 501), (520, 1), oshift).fill_(False)
                assert (big[left] == 77).all()


def test_more_rows_than_a_grid_axis(qg):
    x = torch.randn((70000, 8), generator=gen(1), device="cuda")
    allow = torch.full((70000, 1), 0x55, dtype=torch.int32, device="cuda")
    got = qg.qg_logits_adjust(x, allow=allow)
    want = x.clone()
    want[:, 1::2] = -math.inf
    assert torch.equal(got, want)


def test_counts_are_exact_and_the_order_changes_nothing(qg):
    """One id said 100001 times, by all threads of a block at once."""
    h = torch.full((1, 200003), 7, dtype=torch.int32, device="cuda")
    h[0, ::2] = torch.arange(100002, device="cuda").int() % 4096 + 8
    x = torch.zeros((1, 5000), device="cuda")
    got = qg.qg_logits_adjust(x, history=h, history_len=ints([200003]), frequency=torch.full((1,), 0.5, device="cuda"))
    assert got[0, 7].item() == -0.5 * 100001
    for _ in range(3):
        assert torch.equal(got, qg.qg_logits_adjust(x, history=h, history_len=ints([200003]), frequency=torch.full((1,), 0.5, device="cuda")))


def test_logits_replay(qg):
    x = torch.randn((3, 3000), generator=gen(3), device="cuda")
    h, n = torch.randint(0, 3000, (3, 50), device="cuda", dtype=torch.int32), ints([50, 3, 20])
    rep = torch.full((3,), 1.5, device="cuda")
    run = lambda: qg.qg_logits_adjust(x, history=h, history_len=n, repetition=rep)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    n.copy_(ints([1, 40, 0]))
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, run())


# ----------------------------------------------------------------------------- accepted drafts
def moved(k, steps, pages, page, new, kv_len, keep, keep_len, n_pages):
    """The pool after the moves, one slot after another."""
    k = k.clone()
    steps = None if steps is None else steps.clone()
    for b, (n, L) in enumerate(zip(new, kv_len)):
        base = L - n
        for i in range(min(max(keep_len[b], 0), len(keep[b]), n)):
            src, dst = base + keep[b][i], base + i
            if not i < keep[b][i] < n or dst < 0:
                continue
            p, q = int(pages[b, src // page]), int(pages[b, dst // page])
            if not 0 <= q < n_pages:
                continue
            for x in (k, steps):
                if x is not None:
                    x[..., q, :, dst % page, :] = x[..., p, :, src % page, :] if 0 <= p < n_pages else 0
    return k, steps


@pytest.mark.parametrize("layers", [None, 1, 3])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", [F16, BF16, "q8"], ids=["f16", "bf16", "q8"])
def test_keep(qg, kind, D, layers):
    g, r = gen(D), random.Random(D)
    page, new, kv = 16, [16, 40, 1, 0, 300, 5], [100, 40, 77, 9, 1000, 3]
    keep = [sorted(r.sample(range(max(n, 1)), min(n, 20))) + [0] * (20 - min(n, 20)) for n in new]
    keep[4][5:] = range(250, 265)
    keep_len = [5, 20, 1, 4, 20, 2]
    q_start, lens, pages, n_pages = tables(new, kv, page, 2, g)
    pages[1, 1], pages[4, 58] = -3, n_pages + 9
    L = layers or 1
    pools = [make_cache(kind, n_pages, 3, page, D, g) for _ in range(L)]
    k, v, kd, vd = (None if pools[0][i] is None else torch.stack([p[i] for p in pools]) for i in range(4))
    if layers is None:
        k, v, kd, vd = (None if x is None else x[0] for x in (k, v, kd, vd))
    want_k, want_v = (moved(x, d, pages, page, new, kv, keep, keep_len, n_pages) for x, d in ((k, kd), (v, vd)))
    out = qg.qg_cache_keep(k, v, q_start, lens, pages, ints(keep), ints(keep_len), kd=kd, vd=vd)
    assert torch.equal(k, want_k[0]) and torch.equal(v, want_v[0])
    if kd is not None:
        assert torch.equal(kd, want_k[1]) and torch.equal(vd, want_v[1])
    assert out.tolist() == [max(0, L_ - n + min(m, n, 20)) for n, L_, m in zip(new, kv, keep_len)]
    # over the lengths themselves; nothing is left to move then but what a second pass of the same indices would
    want = [qg.qg_cache_keep(k.clone(), v.clone(), q_start, lens, pages, ints(keep), ints(keep_len),
                             kd=None if kd is None else kd.clone(), vd=None if vd is None else vd.clone())][0]
    same = qg.qg_cache_keep(k, v, q_start, lens, pages, ints(keep), ints(keep_len), kd=kd, vd=vd, kv_out=lens)
    assert same is lens and torch.equal(lens, want)


def test_keep_odd_indices(qg):
    """Lengths below zero and beyond the drafts or the width; indices that fall, repeat, or name no draft."""
    g = gen(1)
    new, kv = [10, 10, 10, 10], [50, 50, 10, 60]
    keep = [[9, 8, 7, 3, 2], [0, 5, 5, 5, 1], [-4, 3, 99, 1 << 30, 9], [1, 2, 3, 4, 5]]
    q_start, lens, pages, n = tables(new, kv, 16, 1, g)
    for lengths in ([5, 5, 5, 5], [-1, 99, 3, 0]):
        k, v, _, _ = make_cache(F16, n, 2, 16, 64, g)
        want = [moved(x, None, pages, 16, new, kv, keep, lengths, n)[0] for x in (k, v)]
        out = qg.qg_cache_keep(k, v, q_start, lens, pages, ints(keep), ints(lengths))
        assert torch.equal(k, want[0]) and torch.equal(v, want[1])
        assert out.tolist() == [L - m + min(max(x, 0), 5) for L, m, x in zip(kv, new, lengths)]


def test_keep_in_strided_pools(qg):
    """Slots before heads, keys and values of one allocation; layers apart by more than a pool."""
    g = gen(2)
    new, kv, keep = [20, 7], [90, 33], [[0, 3, 9, 19], [1, 2, 6, 6]]
    q_start, lens, pages, n = tables(new, kv, 16, 1, g)
    both = torch.randn((2, 3, n, 16, 2, 128), generator=g, device="cuda").half()
    layers = both.transpose(3, 4)[:, ::2]  # (2, layers, pages, heads, page, dim)
    k, v = layers[0], layers[1]
    want = [moved(x, None, pages, 16, new, kv, keep, [4, 3], n)[0] for x in (k, v)]
    between = both[:, 1].clone()
    qg.qg_cache_keep(k, v, q_start, lens, pages, ints(keep), ints([4, 3]))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and torch.equal(both[:, 1], between)


# ----------------------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("kind", [F16, BF16, "q8"], ids=["f16", "bf16", "q8"])
@pytest.mark.parametrize("rot,pairs", [(128, False), (128, True), (100, False), (36, True)])
def test_rotary_positions_beside_the_slots(qg, kind, rot, pairs):
    """Tokens turned by given positions are, bit for bit, those whose slots are at these positions."""
    g = gen(rot)
    D, H, Hk, page = 128, 4, 2, 16
    new, kv = [6, 3], [40, 25]
    q_start, lens, pages, n = tables(new, kv, page, 1, g)
    q, k1, v1 = (torch.randn((9, h, D), generator=g, device="cuda") for h in (H, Hk, Hk))
    turns = qg.qg_rope_turns(rot)[0].cuda()
    pos = [34, 35, 35, 36, 36, 36, 22, 1000000, 0]
    k, v, kd, vd = make_cache(kind, n, Hk, page, D, g)
    got = qg.qg_rope_append(q, k1, v1, turns, k, v, q_start, lens, pages, kd=kd, vd=vd, pairs=pairs, positions=ints(pos))
    same = qg.qg_rope_append(q, k1, v1, turns, k.clone(), v.clone(), q_start, lens, pages, kd=None if kd is None else kd.clone(),
                             vd=None if vd is None else vd.clone(), pairs=pairs, positions=ints([34 + i for i in range(6)] + [22, 23, 24]))
    assert torch.equal(same, qg.qg_rope_append(q, k1, v1, turns, k.clone(), v.clone(), q_start, lens, pages, kd=None if kd is None else kd.clone(),
                                               vd=None if vd is None else vd.clone(), pairs=pairs))
    for t, p in enumerate(pos):  # a sequence of its own for each token, whose only page holds slot p
        k2, v2, kd2, vd2 = make_cache(kind, 1, Hk, page, D, g)
        one = torch.zeros((1, p // page + 1), dtype=torch.int32, device="cuda")
        want = qg.qg_rope_append(q[t:t + 1], k1[t:t + 1], v1[t:t + 1], turns, k2, v2, ints([0, 1]), ints([p + 1]), one, kd=kd2, vd=vd2, pairs=pairs)
        assert torch.equal(got[t:t + 1], want)
        b = int(t >= 6)
        slot = kv[b] - new[b] + t - 6 * b
        at = int(pages[b, slot // page])
        for mine, other in ((k, k2), (v, v2), (kd, kd2), (vd, vd2)):
            if mine is not None:
                assert torch.equal(mine[at, :, slot % page], other[0, :, p % page])


# ----------------------------------------------------------------------------- streams and devices
def test_other_streams(qg):
    from test_gpu_streams import crossed
    g = gen(3)
    q_start, lens, pages, n = tables([40, 1], [300, 90], 16, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 16, 128, g)
    q = torch.randn((41, 8, 128), generator=g, device="cuda").half()
    tree = words_of([(1 << i + 1) - 1 for m in (40, 1) for i in range(m)], 2)
    ws = qg.qg_attn_workspace_size(128, 8, 2, 41, 2)
    crossed(qg, lambda s: [qg.qg_attn_shaped(q, k, v, q_start, lens, pages, cap=9.0, max_new=40, stream=s)], [ws, q.nbytes])
    crossed(qg, lambda s: [qg.qg_attn_tree(q, k, v, q_start, lens, pages, tree, max_new=1, stream=s)], [ws, q.nbytes])
    parents = ints([-1] + list(range(39)) + [-1])
    crossed(qg, lambda s: list(qg.qg_tree_masks(parents, q_start, lens, 2, stream=s)), [41 * 4, 41 * 8])
    keep, one = ints([[0, 5, 9], [0, 0, 0]]), ints([1, 1])
    crossed(qg, lambda s: [qg.qg_cache_keep(k, v, q_start, lens, pages, keep, one, stream=s)], [8])
    x = torch.randn((300, 20000), generator=g, device="cuda")
    h, m = torch.randint(0, 20000, (300, 50), generator=g, device="cuda", dtype=torch.int32), ints([50] * 300)
    rep = torch.full((300,), 1.5, device="cuda")
    crossed(qg, lambda s: [qg.qg_logits_adjust(x, history=h, history_len=m, repetition=rep, stream=s)], [x.nbytes])


def test_inputs_written_just_before(qg):
    """What the calls read is the last thing that the stream wrote, by a kernel that has just ended."""
    x = torch.randn((300, 20000), generator=gen(4), device="cuda")
    h, m = torch.zeros((300, 60), dtype=torch.int32, device="cuda"), ints([60] * 300)
    rep = torch.full((300,), 1.5, device="cuda")
    wanted = [torch.randint(0, 20000, (300, 60), generator=gen(i), device="cuda", dtype=torch.int32) for i in range(6)]
    want = [qg.qg_logits_adjust(x, history=w, history_len=m, repetition=rep).clone() for w in wanted]
    got = []
    for w in wanted:
        h.copy_(w)
        got.append(qg.qg_logits_adjust(x, history=h, history_len=m, repetition=rep))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_bad_tensors_are_refused(qg):
    g = gen(5)
    q_start, lens, pages, n = tables([3], [30], 16, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 16, 64, g)
    q = torch.randn((3, 4, 64), generator=g, device="cuda").half()
    where = (q, k, v, q_start, lens, pages)
    tree = ints([[1], [3], [7]])
    for kw in (dict(slopes=torch.ones(3, device="cuda")), dict(slopes=torch.ones(4, device="cuda").half()), dict(slopes=torch.ones(4)),
               dict(prefix=ints([1, 2])), dict(first=ints([0, 0])), dict(first=ints([0, 0, 0]).long())):
        with pytest.raises(ValueError):
            qg.qg_attn_shaped(*where, **kw)
    for bad in (tree[:2], tree.long(), tree.view(-1), torch.zeros((3, 0), dtype=torch.int32, device="cuda"), ints([[1, 0], [3, 0], [7, 0]]).t()):
        with pytest.raises(ValueError):
            qg.qg_attn_tree(*where, bad)
    with pytest.raises(ValueError):
        qg.qg_attn_tree(*where, tree, positions=ints([1, 2]))
    for cap in (-1.0, math.nan, math.inf):
        with pytest.raises(qg.QGError):
            qg.qg_attn_shaped(*where, cap=cap)
    for args in ((ints([-1, 0, 1]), q_start, lens, 0), (ints([-1, 0, 1]).long(), q_start, lens, 1), (ints([-1, 0, 1]), q_start, ints([30, 1]), 1)):
        with pytest.raises(ValueError):
            qg.qg_tree_masks(*args)
    with pytest.raises(qg.QGError):
        qg.qg_tree_masks(ints([-1, 0, 1]), q_start, lens, 33)
    keep, one = ints([[0, 2]]), ints([2])
    for args in ((k, v[:, :1], q_start, lens, pages, keep, one), (k, v, q_start, lens, pages, keep.view(-1), one), (k, v, q_start, lens, pages, keep, ints([1, 1])),
                 (k, v, q_start, lens, pages, keep.long(), one), (k[None], v, q_start, lens, pages, keep, one)):
        with pytest.raises(ValueError):
            qg.qg_cache_keep(*args)
    x = torch.randn((2, 100), generator=g, device="cuda")
    h = ints([[1, 2], [3, 4]])
    for kw in (dict(history=h), dict(history=h, history_len=ints([1])), dict(repetition=torch.ones(2)), dict(bias_start=ints([0, 1, 2])),
               dict(allow=ints([[1, 2, 3], [1, 2, 3]])), dict(drafts=ints([1, 2])), dict(seq=ints([0])), dict(out=torch.empty((2, 99), device="cuda")),
               dict(out=torch.empty((2, 100), dtype=torch.int32, device="cuda")), dict(out_dtype=torch.int8)):
        with pytest.raises(ValueError):
            qg.qg_logits_adjust(x, **kw)
