"""qg_rope_append, qg_rope_turns and qg_norm_residual where they have gone wrong or could."""
import pytest
import torch

from layer_testlib import BF16, F16, F32
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
