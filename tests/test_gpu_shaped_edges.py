"""qg_attn_shaped and qg_attn_tree where fp32 is short: distances between positions that fp32 does not hold, scores near 0 under large caps."""
import pytest
import torch

from draft_testlib import attention, bounds, intervals, trees, words_of
from layer_testlib import BF16, F16, F32, gen, make_cache, tables, within
from qg_testlib import qg_module
from test_gpu_shaped import alibi, check, ints, random_trees

pytestmark = pytest.mark.gpu
KINDS, IDS = [F16, BF16, "q8"], ["f16", "bf16", "q8"]


@pytest.fixture(scope="module")
def qg():
    return qg_module()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_distances_between_slots_past_2_to_24(qg, kind, D):
    """A sequence of more than 2^24 slots, whose table names three pages over and over: distances of 1 in a window, where the
    slots themselves are even numbers in fp32.  Behind whole pages that nobody sees the sequence is a short one."""
    g, page, window, Hk, H = gen(D), 1024, 300, 2, 4
    k, v, kd, vd = make_cache(kind, 3, Hk, page, D, g)
    for L in ((1 << 24) + 37, (1 << 25) + 1027):
        pages = (torch.arange(L // page + 1, device="cuda") % 3).int()[None].contiguous()
        for n in (1, 3, 100):  # the row kernel twice, the chunk kernel
            lo = (L - n - window) // page * page
            q = (2 * torch.randn((n, H, D), generator=g, device="cuda")).to(F16 if kind == "q8" else kind)
            for slopes, cap in ((alibi(H), 0.0), (torch.full((H,), 0.5, device="cuda"), 20.0)):
                lse = torch.empty((n, H), device="cuda")
                out = qg.qg_attn_shaped(q, k, v, ints([0, n]), ints([L]), pages, kd=kd, vd=vd, slopes=slopes, cap=cap, window=window, lse=lse, max_new=n,
                                        out_dtype=F32)
                ref = attention(q, k, v, kd, vd, [n], [L - lo], pages[:, lo // page:], D ** -0.5, intervals([n], [L - lo], window), cap, slopes, kind == "q8")
                bound, lse_bound = bounds(*ref, q.dtype, F32, kind == "q8")
                within(out, ref[0], bound, "out")
                assert ((lse.double() - ref[1]).abs() <= lse_bound).all()
    assert qg.qg_device_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("start", [1 << 24, (1 << 25) + 1, (1 << 31) - 300, -(1 << 31)])
def test_distances_between_positions_past_2_to_24(qg, kind, D, start):
    """Drafts at positions that fp32 does not tell apart, in the row kernel and the chunk kernel, behind slots and at a sequence's start."""
    new, kv = [40, 7, 130], [40, 300, 150]
    _, depth = random_trees(new, new, seed=3)  # lengths as many as drafts: positions from 0 on
    bits, _ = random_trees(new, kv, seed=3)
    for hint in (1, 130):
        check(qg, kind, 4, 2, D, 16, new, kv, tree=bits, words=5, positions=[start + x for x in depth], slopes=alibi(4), max_new=hint, seed=D)
        check(qg, kind, 2, 1, D, 32, new, kv, tree=bits, words=5, positions=[start + x for x in depth], slopes=alibi(2), cap=15.0, window=50, max_new=hint)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_caps_where_only_unlikely_scores_reach_them(qg, kind, D, biased):
    """Scores near 0 lead and others lie at the lower end of a large cap, so that the fit of tanh near 0 counts and not that of its ends.

    With entries of 1 and -1 in u, keys are u / 32 or -112 u and queries 33 to 128 times u / 64: products and their sums are whole
    multiples of 2^-11 below 2^5, or of 2^-2 below 2^17, and exact in fp32, as are 8-bit keys in fp16 (codes 1 and -112, steps 2^-5 and 1)
    and scale / cap.  What is left for the scores near 0, z = 1 to 4, is the fit and the products around it, 2^-19 z, and the rounding of exponents and
    of the logarithm, 2^-22 of each; exponentials and their sum in fp32 are 2^-18 on the logarithm.  Scores near the lower end,
    below -0.69 caps, have a probability of 0.  (2^-22 of the cap would be 1e-3.)"""
    g, page, Hk, H, n, cap = gen(D), 32, 2, 4, 300, 4096.0
    q_start, lens, pages, n_pages = tables([n, 1], [n, n], page, 1, g)
    u = torch.randint(0, 2, (Hk, D), generator=g, device="cuda") * 2 - 1
    k, v, kd, vd = make_cache(kind, n_pages, Hk, page, D, g)
    far = torch.arange(n_pages * page, device="cuda").view(n_pages, 1, page, 1) % 16 == 5
    keys = u.view(1, Hk, 1, D) * torch.where(far, -112.0, 2.0 ** -5)
    if kind == "q8":
        step = torch.where(far, 1.0, 2.0 ** -5)
        k.copy_((keys / step).to(torch.int8))
        kd.copy_(step.expand(n_pages, Hk, page, D // 32))
    else:
        k.copy_(keys)
    c = torch.randint(33, 129, (n + 1, H, 1), generator=g, device="cuda").double() / 64
    q = (c * u.repeat_interleave(H // Hk, 0)).to(F16 if kind == "q8" else kind)
    scale = 64.0 / D
    slopes = torch.zeros((H,), device="cuda") if biased else None
    for hint in (1, n):
        lse = torch.empty((n + 1, H), device="cuda")
        qg.qg_attn_shaped(q, k, v, q_start, lens, pages, kd=kd, vd=vd, cap=cap, slopes=slopes, scale=scale, max_new=hint, lse=lse)
        want = attention(q, k, v, kd, vd, [n, 1], [n, n], pages, scale, intervals([n, 1], [n, n]), cap, slopes)[1]
        bound = 2.0 ** -18 + 2.0 ** -19 * 4 + 2.0 ** -22 * (4 + want.abs())
        worst = ((lse.double() - want).abs() / bound).max().item()
        assert worst <= 1, (hint, worst)
    assert qg.qg_device_error() == 0


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_scores_in_the_row_kernel(qg, kind):
    """Caps and biases to the last bits that fp32 leaves them.  The row kernel multiplies 8-bit codes as they are and probabilities as two
    addends, so that scores are off as on 16-bit caches and, but for 8-bit values, the result as by its rounding alone (bounds' term of the
    probabilities' type is fp32's; the 2^-16 beside it holds two addends of 8 bits)."""
    for D in (64, 128, 256):
        for new, kv, tree in (([1, 1, 1], [3, 333, 2500], False), ([2, 1, 3], [40, 900, 3], False), ([5, 8], [700, 8], True)):
            g = gen(D)
            q_start, lens, pages, n_pages = tables(new, kv, 32, 1, g)
            k, v, kd, vd = make_cache(kind, n_pages, 2, 32, D, g)
            q = (2 * torch.randn((sum(new), 4, D), generator=g, device="cuda")).to(F16 if kind == "q8" else kind)
            bits, pos = random_trees(new, kv, seed=D)
            views = trees(new, kv, bits, pos) if tree else intervals(new, kv)
            for cap, slopes in ((3.0, None), (30.0, None), (0.0, alibi(4)), (20.0, alibi(4) / 8)):
                lse = torch.empty((sum(new), 4), device="cuda")
                kw = dict(kd=kd, vd=vd, cap=cap, slopes=slopes, max_new=1, lse=lse, out_dtype=F32)
                if tree:
                    out = qg.qg_attn_tree(q, k, v, q_start, lens, pages, words_of(bits, 1), positions=ints(pos), **kw)
                else:
                    out = qg.qg_attn_shaped(q, k, v, q_start, lens, pages, **kw)
                ref = attention(q, k, v, kd, vd, new, kv, pages, D ** -0.5, views, cap, slopes)
                bound, lse_bound = bounds(*ref, F32, F32, kind == "q8")
                within(out, ref[0], bound, "out")
                assert ((lse.double() - ref[1]).abs() <= lse_bound).all()
    assert qg.qg_device_error() == 0


# ----------------------------------------------------------------------------- plans of many tiles
def documents(new, kv_len, every):
    """The first slot of each token's document: one begins at every `every`-th new token; those before the first go on with the past."""
    return [max(0, L - n + i // every * every if i >= every else 0) for n, L in zip(new, kv_len) for i in range(n)]


@pytest.mark.parametrize("sequences,tokens", [(9, 490), (3, 1300), (20, 460)])
def test_plans_of_hundreds_and_thousands_of_row_tiles(qg, sequences, tokens):
    """Eight tokens to a row tile (16 heads to a cache head of 256): 561, 490 and 1172 tiles, past what the plan puts in order and past a
    round of its threads, where it looks every token's range up."""
    new = [tokens + 3 * (b % 5) for b in range(sequences)]
    kv = [n + (0, 5, 70)[b % 3] for b, n in enumerate(new)]
    check(qg, F16, 16, 1, 256, 64, new, kv, first=documents(new, kv, 37), cap=20.0, window=90, seed=sequences)


def test_plans_of_more_sequences_than_a_round(qg):
    """2100 sequences, most of a token or none: the plan's lists of sequences are made anew twice."""
    new = [(1, 0, 3, 9, 1, 2)[b % 6] for b in range(2100)]
    kv = [n + (0, 3, 17, 40)[b % 4] for b, n in enumerate(new)]
    check(qg, F16, 16, 1, 64, 16, new, kv, first=documents(new, kv, 4), max_new=30, seed=1)
    check(qg, "q8", 16, 1, 256, 16, new, kv, slopes=alibi(16), max_new=30, seed=2)
    bits, pos = random_trees(new, kv, seed=4)
    check(qg, BF16, 16, 1, 128, 16, new, kv, tree=bits, positions=pos, window=20, cap=9.0, max_new=30, seed=3)


@pytest.mark.parametrize("cap", [1e-3, 1.0, 4.0, 20.0, 1e4, 1e8, 1e30])
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.25, None])
def test_caps_and_biases_against_the_scores_size(qg, cap, scale):
    """Scores far beyond the cap, around it and far below, beside biases that count, and that are nothing; in prefixes ahead of their rows too."""
    for slopes in (alibi(4), torch.zeros((4,), device="cuda")):
        for kind, D in ((F16, 128), (BF16, 256), ("q8", 64), ("q8", 256)):
            check(qg, kind, 4, 2, D, 16, [1, 90], [300, 400], cap=cap, scale=scale, slopes=slopes, prefix=[0, 380])
