"""qg_rope_turns beyond the usual ranges, on the host."""
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def qg():
    from gguf_block_quantized_quant_gb300 import build
    build.build()
    import gguf_block_quantized_quant_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("rot,base,original,factor", [(128, 10000.0, 65536.0, 8.0), (128, 10000.0, 1048576.0, 40.0), (64, 10000.0, 4096.0, 4.0),
                                                      (64, 500.0, 131072.0, 2.0), (32, 1e6, 32768.0, 16.0), (256, 100.0, 262144.0, 3.0)])
def test_yarn_ramp(qg, rot, base, original, factor):
    """The ramp of the published rule: its upper edge is held to rot - 1, not to the last pair."""
    def edge(turns):
        return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(edge(32.0)), 0), min(math.ceil(edge(1.0)), rot - 1)
    f = np.array([base ** (-2.0 * j / rot) for j in range(rot // 2)])
    ramp = np.clip((np.arange(rot // 2) - lo) / (hi - lo if hi != lo else 1e-3), 0, 1)
    want = f / factor * ramp + f * (1 - ramp)
    turns, _ = qg.qg_rope_turns(rot, base, qg.ROPE_YARN, factor, original)
    got = turns.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    # floor to 2^-64 turns, and a few roundings of the power and the logarithms
    assert np.allclose(got, want, rtol=1e-12, atol=2 * math.pi * 2.0 ** -64)
