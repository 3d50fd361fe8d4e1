"""qg_attn_paged where it has gone wrong or could: repeated 8-bit chunks of wide heads."""
import pytest
import torch

from layer_testlib import F16, attention, attention_bound, gen, make_cache, tables, within
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
