"""qg_rope_append, qg_rope_turns and qg_norm_residual where they have gone wrong or could."""
import pytest
import torch

from layer_testlib import BF16, F16, F32, gen, make_cache, tables, values
from qg_testlib import qg_module
from test_gpu_rope_norm import rope_check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    return qg_module()


@pytest.mark.parametrize("kind", [F16, BF16, "q8"], ids=["f16", "bf16", "q8"])
@pytest.mark.parametrize("D,H,Hk", [(64, 14, 2), (64, 9, 3), (64, 1, 1), (64, 3, 3), (64, 5, 1), (128, 3, 3), (128, 1, 1), (128, 7, 1), (256, 3, 1)])
def test_queries_and_keys_in_one_step_of_a_warp(qg, kind, D, H, Hk):
    """A warp takes 4 heads of 64 or 2 of 128 at once: the last of the queries beside the first of the keys."""
    for pairs in (False, True):
        for norm in (False, True):
            rope_check(qg, kind, F32, D, H, Hk, D, pairs, 16, [1, 6, 2], [1, 30, 17], norm=norm, seed=H)
    rope_check(qg, kind, F32, D, H, Hk, 64, False, 32, [700, 300], [800, 301], seed=H + 1)  # several steps per warp
    rope_check(qg, kind, F32, D, H, Hk, 24, True, 32, [5], [40], seed=H + 2)


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 6])
def test_norm_of_as_many_rows_as_an_int_counts(qg, rows):
    y = torch.arange(2 ** 12, device="cuda").half().repeat(2 ** 19)[:rows].view(rows, 1)
    r, x = qg.qg_norm_residual(y, None, None, alpha=-1.0)
    assert x is None and torch.equal(r, -y)  # as values: 0 + -1 * 0 is +0
    del y, r
    torch.cuda.empty_cache()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("D,rot,pairs", [(64, 64, False), (128, 128, True), (256, 64, False), (128, 0, False), (64, 20, False), (128, 96, False), (256, 30, True)])
def test_8bit_blocks_with_a_value_that_is_not_finite(qg, bad, D, rot, pairs):
    """They read as NaN, as a block of 32 whose step is not finite; the others hold what they held."""
    g = gen(D)
    q_start, lens, pages, n = tables([3], [20], 16, 0, g)
    x = torch.randn((3, 4, D), generator=g, device="cuda")
    turns = qg.qg_rope_turns(rot)[0].cuda() if rot else None
    reads = []
    for poisoned in (False, True):
        k, v, kd, vd = make_cache("q8", n, 1, 16, D, gen(1))
        y = x.clone()
        if poisoned:
            y[1, 2, D - 3] = bad  # the key: its last block, and its partner's where that is rotated
            y[2, 3, 5] = bad      # the value: its first block
        qg.qg_rope_append(y[:, :2], y[:, 2:3], y[:, 3:], turns, k, v, q_start, lens, pages, kd=kd, vd=vd, pairs=pairs)
        reads.append([(values(a, b)[pages[0, 1].long(), 0, 1:4]) for a, b in ((k, kd), (v, vd))])
    (k0, v0), (k1, v1) = reads
    hit = torch.zeros((3, D // 32), dtype=torch.bool, device="cuda")
    hit[1, -1] = True
    if rot == D:
        hit[1, (D - 3 if pairs else D // 2 - 3) // 32] = True
    hit = hit.repeat_interleave(32, -1)
    assert torch.isnan(k1[hit]).all() and torch.equal(k1[~hit], k0[~hit])
    hit = torch.zeros((3, D), dtype=torch.bool, device="cuda")
    hit[2, :32] = True
    assert torch.isnan(v1[hit]).all() and torch.equal(v1[~hit], v0[~hit])


@pytest.mark.parametrize("kind", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("D,rot,pairs", [(64, 0, False), (64, 20, False), (128, 62, True), (128, 96, False), (128, 64, False), (256, 30, False)])
def test_infinities_past_the_rotated_part_pass_through(qg, kind, D, rot, pairs):
    g = gen(D)
    q_start, lens, pages, n = tables([2], [9], 16, 0, g)
    k, v, _, _ = make_cache(kind, n, 1, 16, D, g)
    x = torch.randn((2, 4, D), generator=g, device="cuda")
    x[..., D - 1], x[..., rot] = float("inf"), -float("inf")
    turns = qg.qg_rope_turns(rot)[0].cuda() if rot else None
    q = qg.qg_rope_append(x[:, :2], x[:, 2:3], x[:, 3:], turns, k, v, q_start, lens, pages, pairs=pairs)
    key = k[pages[0, 0].long(), 0, 7:9]
    assert torch.equal(q[..., rot:], x[:, :2, rot:].to(kind)) and torch.equal(key[:, rot:], x[:, 2, rot:].to(kind))
    assert torch.isfinite(q[..., :rot]).all() and torch.isfinite(key[:, :rot]).all()
