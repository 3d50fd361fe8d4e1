"""qg_attn_paged against softmax attention in 64 bits: types, head layouts, chunk and context
lengths from none to long, pages that end inside a tile, windows, rows that see nothing, and
unused slots and pages that hold NaN."""
import math

import pytest
import torch

from layer_testlib import (BF16, F16, F32, attention, attention_bound, gen, make_cache, tables, within)
from qg_testlib import qg_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    return qg_module()


def poison(k, v, kd, vd, pages, kv_len):
    """NaN (or wild codes and NaN steps) in every slot that no sequence uses."""
    used = torch.zeros((k.shape[0], k.shape[2]), dtype=torch.bool, device=k.device)
    for b, n in enumerate(kv_len):
        for i in range(-(-n // k.shape[2])):
            used[int(pages[b, i]), :min(k.shape[2], n - i * k.shape[2])] = True
    off = ~used[:, None].expand(-1, k.shape[1], -1)
    for x, d in ((k, kd), (v, vd)):
        x[off] = -128 if d is not None else math.nan
        if d is not None:
            d[off] = math.nan


def check(qg, kind, H, Hk, D, page, new, kv_len, window=0, scale=None, out_dtype=None, seed=1, nhd=False, max_new=None, spread=2.0):
    g = gen(seed)
    dtype = F16 if kind == "q8" else kind
    q_start, lens, pages, n_pages = tables(new, kv_len, page, 3, g)
    k, v, kd, vd = make_cache(kind, n_pages, Hk, page, D, g, nhd)
    poison(k, v, kd, vd, pages, kv_len)
    T = sum(new)
    q = (spread * torch.randn((T, H, D), generator=g, device="cuda")).to(dtype)
    lse = torch.empty((T, H), device="cuda")
    out = qg.qg_attn_paged(q, k, v, q_start, lens, pages, kd=kd, vd=vd, window=window, scale=scale, lse=lse,
                           out_dtype=out_dtype, max_new=max(new) if max_new is None else max_new)
    torch.cuda.synchronize()
    assert qg.qg_device_error() == 0
    sc = D ** -0.5 if scale is None else scale
    o, want_lse, A, B = attention(q, k, v, kd, vd, new, kv_len, pages, sc, window)
    r = within(out, o, attention_bound(o, A, B, dtype, out.dtype, kind == "q8"), "out")
    empty = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    # natural logs: scores off by dS as in the bound above, the fp32 log of the sum and its rounding
    tol = (2.0 ** -18 + (2.0 ** -11 if kind == "q8" else 0)) * B + 2.0 ** -18 + 2.0 ** -22 * want_lse.masked_fill(empty, 0).abs()
    assert (((lse.double() - want_lse).abs() <= tol) | empty).all()
    assert (out[empty] == 0).all()
    return r


KINDS = [F16, BF16, "q8"]
IDS = ["f16", "bf16", "q8"]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_single_tokens_ragged(qg, kind, D):
    check(qg, kind, 8, 2, D, 32, [1] * 9, [1, 2, 15, 16, 17, 33, 100, 1000, 2111])


@pytest.mark.parametrize("group", [1, 2, 3, 6, 8, 12, 16, 20, 40])
def test_head_groups(qg, group):
    check(qg, F16, 2 * group, 2, 128, 16, [1, 1, 2], [77, 300, 129], seed=group)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_page_sizes(qg, kind, page):
    check(qg, kind, 4, 2, 128, page, [1, 3, 40], [page - 1, page + 1, 3 * page + 7], seed=page)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("new,kv", [([7], [7]), ([64], [64]), ([129], [129]), ([200], [555]), ([1, 130, 5, 64], [900, 131, 5, 320]),
                                    ([257, 1], [1300, 1])])
def test_chunks(qg, kind, D, new, kv):
    check(qg, kind, 8, 2, D, 32, new, kv, seed=sum(new))


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (6, 1), (24, 4), (5, 1)])
def test_chunk_head_layouts(qg, H, Hk):
    check(qg, F16, H, Hk, 128, 64, [100, 30], [180, 64], seed=H)
    check(qg, BF16, H, Hk, 64, 16, [100, 30], [180, 64], seed=H + 1)


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 5000])
@pytest.mark.parametrize("new,kv", [([1, 1, 1], [1, 40, 700]), ([150, 20], [400, 20])])
def test_window(qg, window, new, kv):
    check(qg, F16, 4, 2, 128, 16, new, kv, window=window, seed=window)
    check(qg, "q8", 4, 2, 128, 48, new, kv, window=window, seed=window)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_rows_that_see_nothing(qg, kind):
    """Sequences without tokens, without slots, and chunks longer than their context."""
    check(qg, kind, 4, 2, 128, 16, [0, 1, 0, 5, 3], [0, 0, 40, 2, 3])
    check(qg, kind, 4, 2, 64, 16, [0, 100, 300, 40], [10, 30, 0, 40])
    check(qg, kind, 4, 2, 64, 16, [0, 0, 1], [0, 0, 0])


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_long_context_is_split(qg, kind):
    check(qg, kind, 8, 1, 128, 64, [1], [33333])
    check(qg, kind, 4, 2, 256, 64, [1, 1], [20001, 5])
    check(qg, kind, 4, 2, 128, 64, [70], [9000])


def test_many_sequences(qg):
    """More sequences than threads of a block; one of them long."""
    lens = [1 + (37 * i) % 90 for i in range(700)]
    lens[333] = 4000
    check(qg, BF16, 4, 2, 64, 16, [1] * 700, lens)
    check(qg, F16, 4, 2, 128, 16, [1 + i % 40 for i in range(300)], [40 + (i * 31) % 100 for i in range(300)])


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_hint_only_chooses_the_kernel(qg, kind):
    for hint in (0, 1, 1000):
        check(qg, kind, 8, 2, 128, 32, [1, 50, 200], [70, 60, 700], max_new=hint)
        check(qg, kind, 8, 2, 64, 32, [1, 1], [70, 333], max_new=hint)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.25])
def test_scales(qg, scale):
    """Flat, very peaked (scores of hundreds) and negative scales."""
    check(qg, F16, 4, 2, 128, 16, [1, 90], [300, 400], scale=scale)


def test_slots_before_heads(qg):
    for kind in KINDS:
        check(qg, kind, 8, 4, 128, 16, [1, 33], [99, 200], nhd=True)


def test_fp32_out_of_single_tokens_keeps_fp32_accuracy(qg):
    """Probabilities go in as two addends: fp32 outputs are not held to 11 or 8 bits."""
    for kind in (F16, BF16):
        g = gen(5)
        new, kv = [1, 1], [700, 1234]
        q_start, lens, pages, n = tables(new, kv, 32, 1, g)
        k, v, _, _ = make_cache(kind, n, 2, 32, 128, g)
        q = torch.randn((2, 8, 128), generator=g, device="cuda").to(kind)
        out = qg.qg_attn_paged(q, k, v, q_start, lens, pages, out_dtype=F32, max_new=1)
        o, _, A, B = attention(q, k, v, None, None, new, kv, pages, 128 ** -0.5, 0)
        within(out, o, attention_bound(o, A, B, kind, F32, False, exact_p=True), "fp32 out")


def test_fp32_out_of_chunks(qg):
    for kind in KINDS:
        check(qg, kind, 4, 2, 128, 32, [90, 1], [300, 80], out_dtype=F32)


def test_strided_queries_and_interleaved_pools(qg):
    """q as a view of a wider projection; keys and values of one pool, page by page."""
    g = gen(9)
    new, kv = [1, 40], [50, 90]
    q_start, lens, pages, n = tables(new, kv, 16, 1, g)
    pool = torch.randn((n, 2, 2, 16, 128), generator=g, device="cuda").half()
    k, v = pool[:, 0], pool[:, 1]
    wide = torch.randn((41, 4, 2, 128), generator=g, device="cuda").half()
    q = wide[:, :, 0]
    for hint in (1, 40):
        out = qg.qg_attn_paged(q, k, v, q_start, lens, pages, max_new=hint)
        o, _, A, B = attention(q, k, v, None, None, new, kv, pages, 128 ** -0.5, 0)
        within(out, o, attention_bound(o, A, B, F16, F16, False), "strided")


def test_pages_freed_behind_a_window(qg):
    """Page ids of slots that the window has left may be gone (-1) or out of range."""
    g = gen(11)
    for new in ([1], [50]):
        q_start, lens, pages, n = tables(new, [600], 16, 1, g)
        k, v, _, _ = make_cache(F16, n, 2, 16, 128, g)
        q = torch.randn((new[0], 4, 128), generator=g, device="cuda").half()
        full = qg.qg_attn_paged(q, k, v, q_start, lens, pages, window=100, max_new=new[0])
        low = 600 - new[0] - 100 + 1
        gone = pages.clone()
        gone[0, :low // 16] = -1
        gone[0, 0] = 1 << 30
        cut = qg.qg_attn_paged(q, k, v, q_start, lens, gone, window=100, max_new=new[0])
        assert torch.equal(full, cut)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_missing_pages_read_as_zeros(qg, kind):
    g = gen(12)
    q_start, lens, pages, n = tables([1, 20], [40, 70], 16, 1, g)
    k, v, kd, vd = make_cache(kind, n, 2, 16, 128, g)
    q = torch.randn((21, 4, 128), generator=g, device="cuda").to(F16 if kind == "q8" else kind)
    bad = pages.clone()
    bad[0, 1], bad[1, 2] = -5, n + 7
    outs = []
    for hint in (1, 20):
        outs.append(qg.qg_attn_paged(q, k, v, q_start, lens, bad, kd=kd, vd=vd, max_new=hint))
    k2, v2 = k.clone(), v.clone()
    for x in (k2, v2):
        x[int(pages[0, 1])] = 0
        x[int(pages[1, 2])] = 0
    for hint, got in zip((1, 20), outs):
        want = qg.qg_attn_paged(q, k2, v2, q_start, lens, pages, kd=kd, vd=vd, max_new=hint)
        assert torch.equal(got, want)


@pytest.mark.parametrize("hint", [1, 64])
def test_pool_past_32_bit_offsets(qg, hint):
    """Pages whose element offsets pass 2^31, in pools of 8-bit codes."""
    page, H, D = 128, 8, 256
    per = page * H * D
    n = (1 << 31) // per + 40
    g = gen(13)
    k, v = (torch.empty((n, H, page, D), dtype=torch.int8, device="cuda") for _ in range(2))
    kd, vd = (torch.empty((n, H, page, D // 32), dtype=torch.float16, device="cuda") for _ in range(2))
    ids = torch.arange(n - 6, n, device="cuda")
    for x, d in ((k, kd), (v, vd)):
        x[ids] = torch.randint(-127, 128, (6, H, page, D), generator=g, device="cuda").to(torch.int8)
        d[ids] = (torch.rand((6, H, page, D // 32), generator=g, device="cuda") * 0.02 + 0.01).half()
    pages = ids.to(torch.int32)[None].contiguous()
    new, kv = [3], [700]
    q_start, lens = torch.tensor([0, 3], dtype=torch.int32, device="cuda"), torch.tensor(kv, dtype=torch.int32, device="cuda")
    q = torch.randn((3, 16, D), generator=g, device="cuda").half()
    out = qg.qg_attn_paged(q, k, v, q_start, lens, pages, kd=kd, vd=vd, max_new=hint)
    o, _, A, B = attention(q, k, v, kd, vd, new, kv, pages, D ** -0.5, 0)
    within(out, o, attention_bound(o, A, B, F16, F16, True), "far pages")


def test_other_stream_graph_and_determinism(qg):
    g = gen(14)
    new, kv = [1, 1, 60], [5000, 70, 400]
    q_start, lens, pages, n = tables(new, kv, 32, 1, g)
    k, v, _, _ = make_cache(BF16, n, 2, 32, 128, g)
    q = torch.randn((62, 8, 128), generator=g, device="cuda").bfloat16()
    ws = torch.empty(qg.qg_attn_workspace_size(128, 8, 2, 62, 3), dtype=torch.uint8, device="cuda")
    for hint in (1, 60):
        first = qg.qg_attn_paged(q, k, v, q_start, lens, pages, ws=ws, max_new=hint)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        out = torch.zeros_like(first)
        ws.fill_(255)  # whatever the workspace holds
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(5):
                qg.qg_attn_paged(q, k, v, q_start, lens, pages, ws=ws, out=out, max_new=hint)
        side.synchronize()
        assert torch.equal(first, out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qg.qg_attn_paged(q, k, v, q_start, lens, pages, ws=ws, out=out, max_new=hint)
        lens2 = torch.tensor([4000, 33, 90], dtype=torch.int32, device="cuda")  # lengths are read on the device
        want = qg.qg_attn_paged(q, k, v, q_start, lens2, pages, ws=ws, max_new=hint)
        keep = lens.clone()
        lens.copy_(lens2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        lens.copy_(keep)
    assert qg.qg_device_error() == 0


def test_refusals(qg):
    g = gen(15)
    q_start, lens, pages, n = tables([1], [40], 16, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 16, 128, g)
    q = torch.randn((1, 4, 128), generator=g, device="cuda").half()
    with pytest.raises(ValueError):
        qg.qg_attn_paged(q.float(), k, v, q_start, lens, pages)
    with pytest.raises(qg.QGError):
        qg.qg_attn_paged(q.bfloat16(), k, v, q_start, lens, pages)
    with pytest.raises(ValueError):
        qg.qg_attn_paged(q[..., :64], k, v, q_start, lens, pages)
    with pytest.raises(qg.QGError):
        qg.qg_attn_paged(q[:, :3].contiguous(), k, v, q_start, lens, pages)  # 3 heads over 2
    with pytest.raises(ValueError):
        qg.qg_attn_paged(q, k, v, q_start.long(), lens, pages)
    with pytest.raises(ValueError):
        qg.qg_attn_paged(q, k, v.bfloat16(), q_start, lens, pages)
    with pytest.raises(ValueError):
        qg.qg_attn_paged(q, k.to(torch.int8), v.to(torch.int8), q_start, lens, pages)  # no steps
    with pytest.raises(ValueError):
        qg.qg_attn_paged(q.cpu(), k, v, q_start, lens, pages)
    with pytest.raises(qg.QGError) as e:
        qg.qg_attn_paged(q, k, v, q_start, lens, pages, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == qg.QG_EWORKSPACE
    with pytest.raises(qg.QGError):
        qg.qg_attn_paged(q, k[:, :, :8], v[:, :, :8], q_start, lens, pages)  # pages of 8 slots
    with pytest.raises(qg.QGError):
        qg.qg_attn_paged(q, k, v, q_start, lens, pages, window=-1)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,Hk", [(4, 4), (6, 2), (12, 2), (16, 2)])
def test_chunks_of_other_groups_and_signs(qg, kind, D, H, Hk):
    """Row tiles that are no whole tokens, and negative scales, whose queries come another way; several items per CTA."""
    new, past = [130, 1, 300, 45], [0, 700, 500, 90]
    for scale in (None, -D ** -0.5):
        check(qg, kind, H, Hk, D, 16, new, [n + p for n, p in zip(new, past)], scale=scale, window=200, seed=H)
    check(qg, kind, H, Hk, D, 64, [60] * 40, [60 + 13 * i for i in range(40)], seed=H + 1)
