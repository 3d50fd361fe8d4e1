"""qg_attn_shaped and qg_attn_tree where fp32 is short: distances between positions that fp32 does not hold."""
import pytest
import torch

from draft_testlib import attention, bounds, intervals
from layer_testlib import BF16, F16, F32, gen, make_cache, within
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
