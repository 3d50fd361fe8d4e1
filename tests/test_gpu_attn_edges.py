"""qg_attn_paged where it has gone wrong or could: repeated 8-bit chunks of wide heads."""
import pytest
import torch

from layer_testlib import BF16, F16, UNIT, attention, attention_bound, gen, make_cache, sequence, tables, within
from qg_testlib import qg_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    return qg_module()


@pytest.mark.parametrize("page", [16, 64, 128])
def test_8bit_chunks_of_wide_heads_repeat_bit_for_bit(qg, page):
    """Two warpgroups convert the codes in turn.  Tiles whose later pages are missing or past the end land
    before those that come from memory; whatever the order, the result is one."""
    g = gen(page)
    new, kv = [40, 90, 1, 200, 33] * 6, [40, 700, 129, 1400, 257] * 6
    q_start, lens, pages, n = tables(new, kv, page, 3, g)
    k, v, kd, vd = make_cache("q8", n, 4, page, 256, g)
    q = (2 * torch.randn((sum(new), 24, 256), generator=g, device="cuda")).half()
    call = lambda: qg.qg_attn_paged(q, k, v, q_start, lens, pages, kd=kd, vd=vd, max_new=max(new))  # noqa: E731
    first = call()
    o, _, A, B = attention(q, k, v, kd, vd, new, kv, pages, 256 ** -0.5, 0)
    within(first, o, attention_bound(o, A, B, F16, F16, True), "out")
    cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(40):
        if i % 2:
            cold.fill_(i)  # the cache comes from memory again
        assert torch.equal(first, call())
    assert qg.qg_device_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_steps_of_missing_and_present_pages_in_turn(qg, D):
    """Chunks whose tiles lie on missing pages and on present ones in turn: zeros that the copying warp wrote
    and steps that bulk copies bring follow each other in one place."""
    g = gen(D)
    page, new, kv = 16, [150, 64, 300], [2000, 1500, 900]
    q_start, lens, pages, n = tables(new, kv, page, 3, g)
    k, v, kd, vd = make_cache("q8", n, 2, page, D, g)
    q = (2 * torch.randn((sum(new), 8, D), generator=g, device="cuda")).half()
    holes = pages.clone()
    for b, length in enumerate(kv):
        gone = torch.rand(-(-length // page), generator=g, device="cuda") < 0.4
        holes[b, :gone.numel()] = torch.where(gone, -1, holes[b, :gone.numel()])
        k[pages[b, :gone.numel()][gone].long()] = 0
        v[pages[b, :gone.numel()][gone].long()] = 0
    want = qg.qg_attn_paged(q, k, v, q_start, lens, pages, kd=kd, vd=vd, max_new=300)
    o, _, A, B = attention(q, k, v, kd, vd, new, kv, pages, D ** -0.5, 0)
    within(want, o, attention_bound(o, A, B, F16, F16, True), "out")
    for _ in range(20):
        assert torch.equal(want, qg.qg_attn_paged(q, k, v, q_start, lens, holes, kd=kd, vd=vd, max_new=300))


@pytest.mark.parametrize("kind", [F16, BF16, "q8"], ids=["f16", "bf16", "q8"])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 7, 1 << 30])
def test_widest_windows_over_padded_sequences(qg, kind, window):
    """"No window" as the largest number, where sequences begin with padding: the rows see what they see without."""
    g = gen(3)
    new, kv = [10, 1, 7], [3, 20, 0]
    q_start, lens, pages, n = tables(new, kv, 16, 1, g)
    k, v, kd, vd = make_cache(kind, n, 2, 16, 128, g)
    q = torch.randn((18, 4, 128), generator=g, device="cuda").to(F16 if kind == "q8" else kind)
    for hint in (1, 60):
        lse = [torch.empty((18, 4), device="cuda") for _ in range(2)]
        want, got = (qg.qg_attn_paged(q, k, v, q_start, lens, pages, kd=kd, vd=vd, max_new=hint, window=w, lse=s)
                     for w, s in zip((0, window), lse))
        assert torch.equal(want, got) and torch.equal(*lse)
        assert (got[:7] == 0).all() and (got[7:11] != 0).any(-1).all() and (got[11:] == 0).all()


def test_arguments_beyond_32_bits_are_refused(qg):
    g = gen(4)
    q_start, lens, pages, n = tables([1], [40], 16, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 16, 128, g)
    q = torch.randn((1, 4, 128), generator=g, device="cuda").half()
    for kw in (dict(window=1 << 32), dict(window=(1 << 32) + 8), dict(window=1 << 70), dict(max_new=(1 << 32) + 1)):
        with pytest.raises((ValueError, OverflowError)):
            qg.qg_attn_paged(q, k, v, q_start, lens, pages, **kw)
    with pytest.raises(ValueError):
        qg.qg_norm_residual(torch.empty(((1 << 32) + 1, 1), dtype=F16, device="cuda"), None, None)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", [F16, "q8"], ids=["f16", "q8"])
def test_slots_up_to_the_last_that_counts(qg, kind):
    """Positions next to 2^31 (one page, listed again and again), seen through a window."""
    g = gen(6)
    page, D, window, L = 1 << 20, 64, 200, 2 ** 31 - 256
    k, v, kd, vd = make_cache(kind, 1, 1, page, D, g)
    pages = torch.zeros((1, 1 << 11), dtype=torch.int32, device="cuda")
    q = torch.randn((3, 4, D), generator=g, device="cuda").half()
    q_start = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    near = slice(L % page - 400, L % page)  # the last 400 slots, as a sequence of their own
    short = [None if t is None else t[:, :, near].contiguous() for t in (k, v, kd, vd)]
    for length in (L, 2 ** 31 - 1):  # held to L
        lens = torch.tensor([length], dtype=torch.int32, device="cuda")
        for hint in (1, 60):
            got = qg.qg_attn_paged(q, k, v, q_start, lens, pages, kd=kd, vd=vd, max_new=hint, window=window)
            ids = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
            o, _, A, B = attention(q, *short, [3], [400], ids, D ** -0.5, window)
            within(got, o, attention_bound(o, A, B, F16, F16, kind == "q8"), "far")
    torch.cuda.empty_cache()


def test_q_start_that_decreases_stays_inside_the_arrays(qg):
    """The rows' values are not defined then; every access is, and nothing else is written."""
    g = gen(7)
    batch, T = 3000, 600
    k, v, _, _ = make_cache(F16, 8, 2, 16, 64, g)
    pages = torch.arange(8, dtype=torch.int32, device="cuda").repeat(batch, 1)
    q = torch.randn((T, 8, 64), generator=g, device="cuda").half()
    lens = torch.full((batch,), 100, dtype=torch.int32, device="cuda")
    need = qg.qg_attn_workspace_size(64, 8, 2, T, batch)
    for n in (batch, 700, 5):
        starts = torch.tensor([0, T] * (n // 2) + [0] * (1 + n % 2), dtype=torch.int32, device="cuda")[:n + 1].contiguous()
        for hint in (1, 60):
            need = qg.qg_attn_workspace_size(64, 8, 2, T, n)
            ws = torch.full((need + 4096,), 7, dtype=torch.uint8, device="cuda")
            out = torch.zeros((T + 64, 8, 64), dtype=F16, device="cuda")
            qg.qg_attn_paged(q, k, v, starts, lens[:n], pages[:n], out=out[:T], ws=ws[:need], max_new=hint)
            torch.cuda.synchronize()
            assert (ws[need:] == 7).all() and (out[T:] == 0).all() and torch.isfinite(out).all()
    assert qg.qg_device_error() == 0


@pytest.mark.parametrize("kind", [F16, BF16, "q8"], ids=["f16", "bf16", "q8"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 2, 40])
@pytest.mark.parametrize("batch", [1, 152])
def test_one_dominant_slot_over_a_long_tail(qg, kind, D, new, batch):
    """The first slot 17.4 nats above 33000 others, each of which is 2^-25 of it and all together 1e-3: what the
    sum counts, the products have to see.  One sequence is split over CTAs; 152 (the same one) are not."""
    g = gen(D + new)
    page, L = 64, 33001
    q_start, lens, pages, n = tables([new], [L], page, 1, g)
    k, v, kd, vd = make_cache(kind, n, 1, page, D, g)
    dtype = F16 if kind == "q8" else kind
    q = 0.01 * torch.randn((new, 4, D), generator=g, device="cuda")
    q[..., 0] = 4
    at = 17.4 * D ** 0.5 / 4
    first = int(pages[0, 0])
    k.copy_((k.float() * 0.05).round() if kind == "q8" else k * 0.05)
    k[..., 0] = 0
    k[first, 0, 0] = 0
    k[first, 0, 0, 0] = 127 if kind == "q8" else at
    if kind == "q8":
        kd[first, 0, 0, 0] = at / 127
    v.abs_()  # a tail of one sign
    q = q.to(dtype)
    starts = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * new
    lse = torch.empty((batch * new, 4), device="cuda")
    out = qg.qg_attn_paged(q.repeat(batch, 1, 1), k, v, starts, lens.repeat(batch), pages.repeat(batch, 1), kd=kd, vd=vd,
                           out_dtype=torch.float32, lse=lse, max_new=new)
    o, want_lse, A, B = attention(q, k, v, kd, vd, [new], [L], pages, D ** -0.5, 0)
    chunk = new * 4 > 16
    # P in two addends in the row kernel; in the chunk kernel's fp16 each slot is held to 2^-32 of the largest at worst
    bound = attention_bound(o, A, B, dtype, torch.float32, kind == "q8", exact_p=not chunk)
    if chunk:
        bound = bound + L * 2.0 ** -32 * 5
    for i in range(batch):
        within(out[i * new:(i + 1) * new], o, bound, "out")
    tol = (2.0 ** -18 + (2.0 ** -11 if kind == "q8" and chunk else 0)) * B + 2.0 ** -18 + 2.0 ** -22 * want_lse.abs()
    assert ((lse.double().view(batch, new, 4) - want_lse).abs() <= tol).all()


@pytest.mark.parametrize("kind,spread,scale", [(F16, 60.0, 8.0), (F16, 2000.0, 1.0), (F16, 2000.0, -3.0), (BF16, 1e3, 0.7), (BF16, 1e6, 1.0), (BF16, 3e3, 77.0)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_of_millions_and_more(qg, kind, spread, scale, D):
    """Softmax of such scores is one slot where it leads by more than the scores' own error: that slot's values
    come out, and nothing becomes zero or infinite."""
    g = gen(D)
    new, kv = [150, 4, 1], [700, 333, 90]
    q_start, lens, pages, n = tables(new, kv, 32, 1, g)
    k, v, _, _ = make_cache(kind, n, 2, 32, D, g)
    k.mul_(spread)
    q = (spread * torch.randn((155, 4, D), generator=g, device="cuda")).to(kind)
    o, want_lse, A, B = attention(q, k, v, None, None, new, kv, pages, scale, 0)
    for hint in (1, 150):
        lse = torch.empty((155, 4), device="cuda")
        out = qg.qg_attn_paged(q, k, v, q_start, lens, pages, scale=scale, lse=lse, max_new=hint)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        # |lse - want| within the scores' error dS of the bound's derivation
        assert ((lse.double() - want_lse).abs() <= 2.0 ** -18 * B + 1).all()
        # the weight of the leading slot from the reference: o is one row of v (A = |o|) where it leads by far
        clear = ((A - o.abs()) == 0).all(-1) & lead(q, k, kv, new, pages, scale, 2.0 ** -17 * B + 40)
        assert clear.float().mean() > 0.5
        within(out[clear], o[clear], 3 * UNIT[kind] * o[clear].abs() + 2.0 ** -16, "out")


def lead(q, k, kv, new, pages, scale, least):
    """Rows whose largest visible score leads the next by `least`."""
    out, at = torch.zeros(q.shape[:2], dtype=torch.bool, device=q.device), 0
    for b, (n, L) in enumerate(zip(new, kv)):
        kk = sequence(k, None, pages[b], L).repeat_interleave(q.shape[1] // k.shape[1], 0)
        z = (q[at:at + n].double().transpose(0, 1) @ kk.transpose(1, 2)) * scale
        z = z.masked_fill(torch.arange(L, device=q.device)[None] > torch.arange(L - n, L, device=q.device)[:, None], -float("inf"))
        top = z.topk(2, -1).values
        out[at:at + n] = (top[..., 0] - top[..., 1]).transpose(0, 1) > least[at:at + n]
        at += n
    return out


@pytest.mark.parametrize("kind", [F16, BF16, "q8"], ids=["f16", "bf16", "q8"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,Hk,new", [(8, 2, [1] * 5), (12, 1, [1] * 5), (4, 2, [4, 7, 5, 8, 6]), (5, 1, [3, 1, 2, 3, 3])])
def test_fp32_out_of_few_rows(qg, kind, D, H, Hk, new):
    """Up to 16 rows: probabilities in two addends, 8-bit keys exact; of the roundings to 16 bits only that of
    an 8-bit value is left."""
    g = gen(D + H)
    kv = [7, 100, 999, 2500, 40]
    q_start, lens, pages, n = tables(new, kv, 48, 1, g)
    k, v, kd, vd = make_cache(kind, n, Hk, 48, D, g)
    dtype = F16 if kind == "q8" else kind
    q = (2 * torch.randn((sum(new), H, D), generator=g, device="cuda")).to(dtype)
    out = qg.qg_attn_paged(q, k, v, q_start, lens, pages, kd=kd, vd=vd, out_dtype=torch.float32, max_new=max(new))
    o, _, A, B = attention(q, k, v, kd, vd, new, kv, pages, D ** -0.5, 0)
    within(out, o, attention_bound(o, A, B, dtype, torch.float32, kind == "q8", exact_p=True), "out")


@pytest.mark.parametrize("kind", [F16, BF16, "q8"], ids=["f16", "bf16", "q8"])
@pytest.mark.parametrize("out_dtype", [None, torch.float32], ids=["same", "f32"])
def test_tokens_of_no_sequence_come_out_as_zeros(qg, kind, out_dtype):
    """Rows before the first sequence's and after the last one's, in calls of a fixed size."""
    g = gen(5)
    new, kv = [3, 0, 20], [50, 9, 333]
    q_start, lens, pages, n = tables(new, kv, 16, 1, g)
    k, v, kd, vd = make_cache(kind, n, 2, 16, 64, g)
    for T, lead_in in ((23, 0), (24, 1), (400, 7), (23 + 600, 600)):
        q = torch.randn((T, 6, 64), generator=g, device="cuda").to(F16 if kind == "q8" else kind)
        for hint in (1, 20):
            out = torch.full((T, 6, 64), 3.0, device="cuda").to(out_dtype or q.dtype)
            lse = torch.zeros((T, 6), device="cuda")
            qg.qg_attn_paged(q, k, v, q_start + lead_in, lens, pages, kd=kd, vd=vd, out=out, lse=lse, max_new=hint)
            inside = slice(lead_in, lead_in + 23)
            want_lse = torch.empty((23, 6), device="cuda")
            want = qg.qg_attn_paged(q[inside], k, v, q_start, lens, pages, kd=kd, vd=vd, out_dtype=out_dtype, lse=want_lse, max_new=hint)
            assert torch.equal(out[inside], want) and torch.equal(lse[inside], want_lse)
            rest = torch.ones(T, dtype=torch.bool, device="cuda")
            rest[inside] = False
            assert (out[rest] == 0).all() and (lse[rest] == -float("inf")).all()
    none = torch.zeros_like(q_start)  # no sequence has a token
    assert (qg.qg_attn_paged(q, k, v, none, lens, pages, kd=kd, vd=vd, max_new=0) == 0).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("step", [515.5, 2.0 ** -14, 2.0 ** -24])
def test_8bit_values_at_both_ends_of_their_range(qg, D, step):
    """Codes of +-127 with the largest step whose values fp16 holds, and with the smallest steps there are."""
    g = gen(D)
    new, kv = [1, 2, 60], [100, 33, 400]
    q_start, lens, pages, n = tables(new, kv, 16, 1, g)
    k, v, kd, vd = make_cache("q8", n, 2, 16, D, g)
    k[:, :, ::3] = 127
    v[:, :, 1::3] = -127
    kd.fill_(step)
    vd.fill_(step)
    q = torch.randn((63, 8, D), generator=g, device="cuda").half()
    scale = 0.05 / (60 * step * D ** 0.5)
    o, _, A, B = attention(q, k, v, kd, vd, new, kv, pages, scale, 0)
    for hint in (1, 60):
        out = qg.qg_attn_paged(q, k, v, q_start, lens, pages, kd=kd, vd=vd, scale=scale, out_dtype=torch.float32, max_new=hint)
        # fp16 products below 2^-14 are rounded to multiples of 2^-24
        within(out, o, attention_bound(o, A, B, F16, torch.float32, True) + 2.0 ** -25, "out")


@pytest.mark.parametrize("kind", [F16, "q8"], ids=["f16", "q8"])
@pytest.mark.parametrize("pages,heads", [(6, 1), (1, 2), (1, 1)])
def test_strides_of_dimensions_of_one_element_say_nothing(qg, kind, pages, heads):
    """Pools and steps of one head or one page whose strides there are any."""
    g = gen(8)
    page, D = 32, 64
    k, v, kd, vd = make_cache(kind, pages, heads, page, D, g)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    L = pages * page - 3
    q_start, lens = torch.tensor([0, 2], dtype=torch.int32, device="cuda"), torch.tensor([L], dtype=torch.int32, device="cuda")
    q = torch.randn((2, 4, D), generator=g, device="cuda").half()

    def odd(t, other):
        if t is None:
            return None
        s = list(t.stride())
        for i in (0, 1):
            if t.shape[i] == 1:
                s[i] = other
        return t.as_strided(t.shape, s)
    for hint in (1, 60):
        want = qg.qg_attn_paged(q, k, v, q_start, lens, table, kd=kd, vd=vd, max_new=hint)
        got = qg.qg_attn_paged(q, odd(k, 1), odd(v, 3), q_start, lens, table, kd=odd(kd, 1), vd=odd(vd, 5), max_new=hint)
        assert torch.equal(want, got)


@pytest.mark.parametrize("new,longest", [([1] * 6, 1), ([2] * 6, 2), ([1, 1, 1, 1, 1, 60], 60), ([1, 40, 1], 40), ([300], 300), ([1] * 63 + [130], 130)])
def test_default_of_the_longest_chunk(qg, new, longest):
    """Without max_new the kernel is the one that the longest chunk takes (the two round differently)."""
    g = gen(9)
    kv = [n + 500 + 37 * i for i, n in enumerate(new)]
    q_start, lens, pages, n = tables(new, kv, 16, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 16, 64, g)
    q = torch.randn((sum(new), 8, 64), generator=g, device="cuda").half()
    rows, chunk = (qg.qg_attn_paged(q, k, v, q_start, lens, pages, max_new=m, out_dtype=torch.float32) for m in (1, 300))
    assert not torch.equal(rows, chunk)
    assert torch.equal(qg.qg_attn_paged(q, k, v, q_start, lens, pages, out_dtype=torch.float32), rows if longest * 4 <= 16 else chunk)


def test_one_token_of_rows_at_any_distance(qg):
    """One row of a buffer whose rows are an odd number of elements apart."""
    g = gen(10)
    q_start, lens, pages, n = tables([1], [40], 16, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 16, 64, g)
    wide = torch.randn((3, 8 * 64 + 1), generator=g, device="cuda").half()
    row = wide[:, :512].unflatten(1, (8, 64))[:1]
    assert row.stride(0) == 513
    for hint in (1, 60):
        want = qg.qg_attn_paged(row[:, :4].contiguous(), k, v, q_start, lens, pages, max_new=hint)
        assert torch.equal(qg.qg_attn_paged(row[:, :4], k, v, q_start, lens, pages, max_new=hint), want)
    turns = qg.qg_rope_turns(64)[0].cuda()
    parts = row[:, :4], row[:, 4:6], row[:, 6:]
    want = qg.qg_rope_append(*(p.contiguous() for p in parts), turns, k, v, q_start, lens, pages)
    assert torch.equal(qg.qg_rope_append(*parts, turns, k, v, q_start, lens, pages), want)
