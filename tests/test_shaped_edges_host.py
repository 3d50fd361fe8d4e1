"""What shaped and tree attention refuse of their scores, on the host."""
import pytest

from test_draft_host import EINVAL, EWORKSPACE, attn
from test_layer_host import qg  # noqa: F401  (the module's fixture)


@pytest.mark.parametrize("name", ["shaped", "tree"])
def test_quotients_that_lose_the_scale(qg, name):  # noqa: F811
    """scale / cap below the normal numbers of fp32 has fewer bits than the scale; 0 and the least normal number are as good as any."""
    L = qg.lib()
    for scale, cap in ((1e-6, 1e37), (-1e-6, 1e33), (1e-8, 2e30), (2.0 ** -126, 2.0), (2.0 ** -149, 1.0), (1e-30, 1e30)):
        assert attn(L, name, scale=scale, cap=cap) == EINVAL, (scale, cap)
    for scale, cap in ((0.0, 1e38), (2.0 ** -125, 2.0), (-(2.0 ** -126), 1.0), (1.0, 1e30), (1.0, 8e37)):
        assert attn(L, name, scale=scale, cap=cap, ws=None) == EWORKSPACE, (scale, cap)
