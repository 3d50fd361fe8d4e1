"""qg_attn_shaped and qg_attn_tree against attention in 64 bits: caps, distances, documents, prefixes and trees, over both kernels,
all caches and head sizes, lengths from none on, rows that see nothing, and unseen slots that hold NaN."""
import math
import random

import pytest
import torch

from draft_testlib import ancestors, attention, bounds, intervals, trees, words_of
from layer_testlib import BF16, F16, F32, gen, make_cache, tables, within
from qg_testlib import qg_module

pytestmark = pytest.mark.gpu
KINDS, IDS = [F16, BF16, "q8"], ["f16", "bf16", "q8"]


@pytest.fixture(scope="module")
def qg():
    return qg_module()


def poison(k, v, kd, vd, pages, kv_len, views):
    """NaN (wild codes and NaN steps) in every slot from kv_len on and before the first that a row of the sequence sees."""
    page = k.shape[2]
    used = torch.zeros((k.shape[0], page), dtype=torch.bool, device=k.device)
    for b, n in enumerate(kv_len):
        seen = views[b][0].any(0).nonzero() if n and views[b][0].numel() else torch.zeros((0, 1))
        lo = int(seen[0]) if len(seen) else n
        for j in range(lo, n):
            used[int(pages[b, j // page]), j % page] = True
    off = ~used[:, None].expand(-1, k.shape[1], -1)
    for x, d in ((k, kd), (v, vd)):
        x[off] = -128 if d is not None else math.nan
        if d is not None:
            d[off] = math.nan


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(qg, kind, H, Hk, D, page, new, kv_len, cap=0.0, slopes=None, prefix=None, first=None, window=0, tree=None, words=1, positions=None,
          scale=None, out_dtype=None, seed=1, max_new=None, spread=2.0):
    """tree: bits of each token's row."""
    g = gen(seed)
    dtype = F16 if kind == "q8" else kind
    q_start, lens, pages, n_pages = tables(new, kv_len, page, 3, g)
    k, v, kd, vd = make_cache(kind, n_pages, Hk, page, D, g)
    T = sum(new)
    views = (intervals(new, kv_len, window, prefix, first) if tree is None else trees(new, kv_len, tree, positions, window, words))
    poison(k, v, kd, vd, pages, kv_len, views)
    q = (spread * torch.randn((T, H, D), generator=g, device="cuda")).to(dtype)
    lse = torch.empty((T, H), device="cuda")
    kw = dict(kd=kd, vd=vd, cap=cap, slopes=slopes, window=window, scale=scale, lse=lse, out_dtype=out_dtype,
              max_new=max(new) if max_new is None else max_new)
    if tree is None:
        out = qg.qg_attn_shaped(q, k, v, q_start, lens, pages, prefix=None if prefix is None else ints(prefix),
                                first=None if first is None else ints(first), **kw)
    else:
        out = qg.qg_attn_tree(q, k, v, q_start, lens, pages, words_of(tree, words), positions=None if positions is None else ints(positions), **kw)
    torch.cuda.synchronize()
    assert qg.qg_device_error() == 0
    ref = attention(q, k, v, kd, vd, new, kv_len, pages, D ** -0.5 if scale is None else scale, views, cap, slopes, kind == "q8")
    bound, lse_bound = bounds(*ref, dtype, out.dtype, kind == "q8")
    within(out, ref[0], bound, "out")
    empty = ref[1] == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert (((lse.double() - ref[1]).abs() <= lse_bound) | empty).all()
    assert (out[empty] == 0).all()
    return out


def alibi(H):
    return torch.tensor([2.0 ** (-8 * (i + 1) / H) for i in range(H)], device="cuda")


LENGTHS = [([1] * 6, [1, 15, 33, 100, 777, 2111]), ([1, 130, 5, 64], [900, 131, 5, 320]), ([3, 2, 1], [40, 2, 300])]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("new,kv", LENGTHS)
def test_caps(qg, kind, D, new, kv):
    check(qg, kind, 8, 2, D, 32, new, kv, cap=50.0, seed=D)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("new,kv", LENGTHS)
def test_distances(qg, kind, D, new, kv):
    check(qg, kind, 8, 2, D, 32, new, kv, slopes=alibi(8), seed=D + 1)
    check(qg, kind, 8, 2, D, 16, new, kv, slopes=alibi(8), cap=30.0, prefix=[7, 0, 300, 64, 5, 2000][:len(new)], seed=D + 2)


@pytest.mark.parametrize("cap", [1e-3, 1.0, 4.0, 20.0, 1e4, 1e30])
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.25, None])
def test_caps_against_the_scores_size(qg, cap, scale):
    """Scores far beyond the cap, around it and far below; zero and negative scales."""
    check(qg, F16, 4, 2, 128, 16, [1, 90], [300, 400], cap=cap, scale=scale)
    check(qg, "q8", 2, 2, 256, 16, [1, 90], [300, 400], cap=cap, scale=scale)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefixes(qg, kind, D):
    """Prefixes of nothing, inside the new tokens, ending before them, of all, beyond the length, negative; with windows."""
    new, kv = [1, 1, 40, 200, 200, 300, 3], [50, 9, 40, 200, 333, 300, 3]
    for window in (0, 50):
        check(qg, kind, 4, 2, D, 16, new, kv, prefix=[0, 100, 20, 150, 100, (1 << 31) - 1, -(1 << 31)], window=window, seed=window)
    check(qg, kind, 4, 4, D, 48, [2, 4], [80, 4], prefix=[79, 4])


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_documents(qg, kind, D):
    """Documents that end inside tiles, tokens behind them that see all, and rows that see nothing."""
    def starts(n, base, cuts, tail):
        out = []
        for i in range(n):
            out.append(0 if i >= n - tail else base + max(c for c in [0] + cuts if c <= i))
        return out
    for G, window in ((2, 0), (3, 33), (1, 0)):
        first = starts(300, 10, [1, 5, 130, 131, 255], 20) + starts(200, 0, [64], 0) + starts(1, 500, [], 0) + starts(7, 90, [3], 1)
        first[50:60] = [1 << 30] * 10  # nothing
        first[310] = -7
        check(qg, kind, 2 * G, 2, D, 32, [300, 200, 1, 7], [310, 200, 501, 97], first=first, window=window, seed=G)
    check(qg, kind, 4, 2, D, 16, [1, 1, 2, 1], [700, 700, 300, 40], first=[699, 350, 299, 0, 40])  # the last sees nothing
    check(qg, kind, 4, 2, D, 16, [1, 40], [700, 100], first=[701] + [200] * 40)  # nobody sees anything


def test_all_at_once(qg):
    for kind, D in ((F16, 128), (BF16, 64), ("q8", 256), (F16, 256)):
        first = [0] * 50 + [100] * 150 + [3] * 20 + [0]
        check(qg, kind, 12, 4, D, 48, [220, 1], [300, 900], cap=20.0, slopes=alibi(12), prefix=[130, 40], first=first, window=150, seed=D)


@pytest.mark.parametrize("group", [1, 2, 3, 6, 8, 16, 20])
def test_head_groups(qg, group):
    H = 2 * group
    check(qg, F16, H, 2, 128, 16, [1, 1, 2], [77, 300, 129], cap=10.0, slopes=alibi(H), seed=group)
    check(qg, BF16, H, 2, 64, 16, [30, 90], [77, 300], cap=10.0, slopes=-alibi(H) / 16, prefix=[50, 299], seed=group)


def test_long_context_is_split(qg):
    for kind in KINDS:
        check(qg, kind, 8, 1, 128, 64, [1], [20001], cap=50.0, slopes=alibi(8) / 64)
        check(qg, kind, 4, 2, 256, 64, [40], [9000], cap=30.0)
        check(qg, kind, 4, 2, 64, 64, [70], [9000], slopes=alibi(4) / 256)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_sequences_without_tokens_or_slots(qg, kind):
    for D in (64, 128, 256):
        check(qg, kind, 4, 2, D, 16, [0, 1, 0, 5, 3], [0, 0, 40, 2, 3], cap=5.0, prefix=[3, 3, 3, 2, 9])
        check(qg, kind, 4, 2, D, 16, [0, 100, 300, 40], [10, 30, 0, 40], cap=5.0, first=[0] * 440)


def test_hint_only_chooses_the_kernel(qg):
    for hint in (0, 1, 4, 1000):
        first = [0] + [5] * 50 + [0] * 100 + [600] * 100
        check(qg, F16, 8, 2, 128, 32, [1, 50, 200], [70, 60, 700], max_new=hint, first=first, cap=9.0)
        bits, pos = random_trees([1, 50, 40], [70, 60, 700], seed=hint)
        check(qg, "q8", 8, 2, 64, 32, [1, 50, 40], [70, 60, 700], max_new=hint, tree=bits, positions=pos, words=2, window=40)


def test_nothing_given_is_plain_attention(qg):
    g = gen(3)
    q_start, lens, pages, n = tables([1, 40], [300, 90], 16, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 16, 128, g)
    q = torch.randn((41, 8, 128), generator=g, device="cuda").half()
    for hint in (1, 40):
        assert torch.equal(qg.qg_attn_shaped(q, k, v, q_start, lens, pages, max_new=hint, window=50),
                           qg.qg_attn_paged(q, k, v, q_start, lens, pages, max_new=hint, window=50))


# ----------------------------------------------------------------------------- trees
def random_trees(new, kv_len, seed=0, wide=2):
    r = random.Random(seed)
    bits, pos = [], []
    for n, L in zip(new, kv_len):
        parents = [-1 if i == 0 or r.random() < 0.1 else r.randrange(max(0, i - wide - i // 2), i) for i in range(n)]
        b, d = ancestors(parents)
        bits += b
        pos += [L - n + x for x in d]
    return bits, pos


TREES = [([16], [716]), ([1, 7, 31, 32, 33], [40, 7, 100, 1000, 33]), ([64, 2, 100], [2000, 300, 611]), ([4, 2, 3], [5, 444, 90])]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("new,kv", TREES)
def test_trees(qg, kind, D, new, kv):
    bits, pos = random_trees(new, kv, seed=D)
    words = -(-max(new) // 32)
    check(qg, kind, 8, 2, D, 32, new, kv, tree=bits, words=words, seed=D)
    check(qg, kind, 4, 2, D, 16, new, kv, tree=bits, words=words + 1, positions=pos, cap=20.0, slopes=alibi(4), window=77, seed=D)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_masks_of_any_bits(qg, kind):
    """Rows of arbitrary bits, some beyond the drafts, some empty; drafts beyond the words; windows shorter than the tree."""
    r = random.Random(7)
    for new, kv, words in (([130, 5], [200, 5], 5), ([300], [1000], 3), ([9, 1], [9, 333], 1), ([2, 2], [2, 130], 2)):
        T = sum(new)
        bits = [r.getrandbits(32 * words) & r.getrandbits(32 * words) for _ in range(T)]
        for i in range(0, T, 5):
            bits[i] |= 1 << i % new[0] if i < new[0] else 1
        # every draft is seen by somebody, so that its values are finite ones
        bits[T - 1] |= (1 << 32 * words) - 1
        bits[0] |= (1 << 32 * words) - 1
        for G in (1, 3):
            check(qg, kind, 2 * G, 2, 128, 16, new, kv, tree=bits, words=words, seed=T)
            check(qg, kind, G, 1, 64, 16, new, kv, tree=bits, words=words, window=3, seed=T, slopes=alibi(G), positions=[kv[0] - 2] * T)
            # drafts that see later ones, whose distance counts as any
            check(qg, kind, 2 * G, 2, 128, 16, new, kv, tree=bits, words=words, seed=T, slopes=alibi(2 * G), cap=(0.0, 25.0)[G // 3])


def test_rows_of_a_tree_that_see_nothing(qg):
    """No slots before the drafts and no bits: zeros.  Drafts that have no slot (longer than their sequence) too."""
    for kind in KINDS:
        bits = [0b1, 0, 0b101, 0, 0b11111]
        check(qg, kind, 4, 2, 128, 16, [5], [5], tree=bits)
        check(qg, kind, 4, 2, 64, 16, [5], [3], tree=[0b11111] * 5)
        check(qg, kind, 4, 2, 256, 16, [40], [20], tree=[(1 << 40) - 1] * 40, words=2)


def test_a_chain_is_causal_attention(qg):
    g = gen(5)
    new, kv = [40, 3], [333, 90]
    q_start, lens, pages, n = tables(new, kv, 32, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 32, 128, g)
    q = torch.randn((43, 4, 128), generator=g, device="cuda").half()
    tree = words_of([(1 << i + 1) - 1 for m in new for i in range(m)], 2)
    for hint in (1, 40):
        got = qg.qg_attn_tree(q, k, v, q_start, lens, pages, tree, max_new=hint, out_dtype=F32)
        want = qg.qg_attn_paged(q, k, v, q_start, lens, pages, max_new=hint, out_dtype=F32)
        # the same products and sums but for where slot tiles begin and are joined
        assert (got - want).abs().max() <= 2 ** -9


def test_masks_from_parents(qg):
    r = random.Random(1)
    new, kv = [1, 40, 0, 64, 33, 5], [9, 100, 3, 64, 1000, 3]
    parents = [[-1] + [r.randrange(-1, i) for i in range(1, n)] if n else [] for n in new]
    parents[1][7], parents[1][9], parents[3][2] = 9, 9, -77  # not before their draft: roots
    flat = ints(sum(parents, []) + [0, 0])
    q_start = ints([0] + [sum(new[:i + 1]) for i in range(len(new))])
    tree, pos = qg.qg_tree_masks(flat, q_start, ints(kv), 3)
    want, depth = [], []
    for p, n, L in zip(parents, new, kv):
        b, d = ancestors(p)
        want += b
        depth += [L - n + x for x in d]
    assert torch.equal(tree[:-2], words_of(want, 3)) and torch.equal(pos[:-2], ints(depth))
    assert (tree[-2:] == 0).all() and (pos[-2:] == 0).all()
    # more drafts than bits
    tree, pos = qg.qg_tree_masks(flat, q_start, ints(kv), 1)
    cut, at = [], 0
    for n in new:
        cut += [w if i < 32 else 0 for i, w in enumerate(want[at:at + n])]
        at += n
    assert torch.equal(tree[:-2], words_of(cut, 1))


def test_results_do_not_depend_on_timing_and_replay(qg):
    """Two runs are equal, and so is a captured call replayed on other contents."""
    g = gen(8)
    new, kv = [20, 40, 1], [5000, 333, 900]
    q_start, lens, pages, n = tables(new, kv, 32, 1, g)
    k, v, kd, vd = make_cache("q8", n, 2, 32, 128, g)
    q = torch.randn((61, 8, 128), generator=g, device="cuda").half()
    bits, pos = random_trees(new, kv)
    tree, pos, slopes = words_of(bits, 2), ints(pos), alibi(8)
    first = ints([0] * 61)
    for hint in (1, 40):
        calls = [lambda: qg.qg_attn_tree(q, k, v, q_start, lens, pages, tree, kd=kd, vd=vd, positions=pos, cap=30.0, slopes=slopes, max_new=hint),
                 lambda: qg.qg_attn_shaped(q, k, v, q_start, lens, pages, kd=kd, vd=vd, cap=30.0, first=first, max_new=hint)]
        for call in calls:
            want = call()
            assert torch.equal(want, call())
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = call()
            kept = q.clone()
            q.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert not torch.equal(out, want)
            q.copy_(kept)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_rows_and_tokens_of_no_sequence(qg):
    """Tokens before the first sequence's and behind the last one's give zeros; what the masks hold for them is not looked at."""
    g = gen(6)
    new, kv = [30, 2], [90, 40]
    q_start, lens, pages, n = tables(new, kv, 16, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 16, 64, g)
    q = torch.randn((40, 4, 64), generator=g, device="cuda").half()
    bits, pos = random_trees(new, kv, seed=2)
    pad = lambda x, fill: [fill] * 3 + list(x) + [fill] * 5  # noqa: E731
    for hint in (1, 30):
        out = qg.qg_attn_tree(q, k, v, q_start + 3, lens, pages, words_of(pad(bits, 0xffffffff), 1), positions=ints(pad(pos, -9)), max_new=hint)
        want = qg.qg_attn_tree(q[3:35].contiguous(), k, v, q_start, lens, pages, words_of(bits, 1), positions=ints(pos), max_new=hint)
        assert torch.equal(out[3:35], want) and (out[:3] == 0).all() and (out[35:] == 0).all()
        first = [0] * 10 + [70] * 20 + [0, 39]
        out = qg.qg_attn_shaped(q, k, v, q_start + 3, lens, pages, first=ints(pad(first, 1 << 30)), cap=9.0, max_new=hint)
        want = qg.qg_attn_shaped(q[3:35].contiguous(), k, v, q_start, lens, pages, first=ints(first), cap=9.0, max_new=hint)
        assert torch.equal(out[3:35], want) and (out[:3] == 0).all() and (out[35:] == 0).all()


def test_bad_lengths_and_pages_stay_inside(qg):
    """Lengths, starts and page ids beyond the arrays are held to them, whatever the masks."""
    g = gen(7)
    k, v, _, _ = make_cache(F16, 6, 2, 16, 64, g)
    q = torch.randn((20, 4, 64), generator=g, device="cuda").half()
    pages = ints([[0, 1, 99], [-4, 2, 1 << 30]])
    tree, positions, first = words_of([(1 << 32) - 1] * 20, 1), ints([1 << 30, -5] * 10), ints([-3, 1 << 30] * 10)
    for starts in ([0, 10, 20], [-7, 15, 900], [5, 2, 20], [0, 0, 0]):
        for lens in ([48, 48], [1 << 30, -5], [0, 3]):
            for hint in (1, 20):
                a = qg.qg_attn_tree(q, k, v, ints(starts), ints(lens), pages, tree, positions=positions, window=7, slopes=alibi(4), cap=5.0, max_new=hint)
                b = qg.qg_attn_shaped(q, k, v, ints(starts), ints(lens), pages, prefix=ints([1 << 30, -1]), first=first, cap=5.0, max_new=hint)
                torch.cuda.synchronize()
                assert a.shape == b.shape == q.shape and qg.qg_device_error() == 0
        qg.qg_tree_masks(ints([7, -9] * 10), ints(starts), ints([48, -2]), 1)
        for keep_len in ([5, 5], [99, -1]):
            qg.qg_cache_keep(k, v, ints(starts), ints([48, 40]), pages, ints([[0, 3, 5, 1 << 30, -8], [9, 9, 9, 9, 9]]), ints(keep_len))
        torch.cuda.synchronize()
