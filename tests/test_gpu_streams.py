"""Calls on a stream that is not the current one, with the workspace and the outputs left to them, while
the current stream allocates and writes memory of the same sizes."""
import pytest
import torch

from layer_testlib import BF16, F16, gen, make_cache, tables
from qg_testlib import qg_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    return qg_module()


def crossed(qg, call, sizes):
    """call(stream) gives outputs; sizes: bytes of the memory that it takes for itself."""
    want = [t.clone() for t in call(None) if t is not None]
    side = torch.cuda.Stream()
    for turn in range(3):
        torch.cuda.synchronize()
        # freed on the current stream, whose writes to them are not done
        torch.cuda._sleep(20_000_000)
        old = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes for _ in range(3)]
        del old
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000_000 if turn % 2 else 60_000_000)
        got = [t for t in call(side) if t is not None]
        # handed out again on the current stream while the call has yet to run
        new = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert all(int(t.min()) == 255 for t in new)
    assert qg.qg_device_error() == 0


@pytest.mark.parametrize("hint", [1, 60])
def test_attention(qg, hint):
    g = gen(1)
    new, kv = [1, 1, 60], [5000, 70, 400]
    q_start, lens, pages, n = tables(new, kv, 32, 1, g)
    k, v, _, _ = make_cache(BF16, n, 2, 32, 128, g)
    q = torch.randn((62, 8, 128), generator=g, device="cuda").bfloat16()
    crossed(qg, lambda s: [qg.qg_attn_paged(q, k, v, q_start, lens, pages, max_new=hint, stream=s)],
            [qg.qg_attn_workspace_size(128, 8, 2, 62, 3), q.nbytes])


def test_rope_and_norms(qg):
    g = gen(2)
    q_start, lens, pages, n = tables([40], [100], 16, 1, g)
    k, v, _, _ = make_cache(F16, n, 2, 16, 128, g)
    x = torch.randn((40, 12, 128), generator=g, device="cuda")
    turns = qg.qg_rope_turns(128)[0].cuda()
    crossed(qg, lambda s: [qg.qg_rope_append(x[:, :8], x[:, 8:10], x[:, 10:], turns, k, v, q_start, lens, pages, stream=s)], [40 * 8 * 128 * 2])
    y, w = torch.randn((64, 2048), generator=g, device="cuda"), torch.ones(2048, device="cuda")
    crossed(qg, lambda s: qg.qg_norm_residual(y, y, w, stream=s), [y.nbytes])


def test_projections_and_ffn(qg):
    import synth
    g = synth.rng(5, salt=7)
    N, K, fmt = 512, 1024, qg.Q4_K
    w = lambda n, kk: torch.from_numpy(synth.weights(fmt, n, kk, g)).cuda().reshape(-1)  # noqa: E731
    W, Wg, Wu, Wd = w(N, K), w(512, K), w(512, K), w(K, 512)
    t = gen(3)
    for M in (1, 4, 16):
        x = torch.randn((M, K), generator=t, device="cuda")
        crossed(qg, lambda s: [qg.qg_gemv(fmt, W, x, N, stream=s)], [qg.qg_workspace_size(qg.QG_OP_GEMV, fmt, M, N, K), M * N * 4])
        crossed(qg, lambda s: [qg.qg_ffn_sublayer(fmt, Wg, Wu, Wd, x, 512, stream=s)],
                [qg.qg_workspace_size(qg.QG_OP_FFN_SUBLAYER, fmt, M, K, K, I=512), M * K * 4])
        crossed(qg, lambda s: list(qg.qg_quantize_act(x, stream=s)), [M * K, M * K // 8])
        q = qg.qg_quantize_act(x)
        crossed(qg, lambda s: [qg.qg_gemv_q(fmt, W, *q, N, stream=s)], [max(1, qg.qg_workspace_size(qg.QG_OP_GEMV_Q, fmt, M, N, K)), M * N * 4])
    x = torch.randn((100, K), generator=t, device="cuda")
    crossed(qg, lambda s: [qg.qg_prefill_gemm(fmt, W, x, N, stream=s)], [qg.qg_workspace_size(qg.QG_OP_PREFILL, fmt, 100, N, K), 100 * N * 4])


def test_the_default_stream_given_from_another(qg):
    """The default stream's handle is 0; it is a stream like any other."""
    y, w = torch.randn((64, 2048), generator=gen(4), device="cuda"), torch.ones(2048, device="cuda")
    want = qg.qg_norm_residual(y, y, w)
    q = qg.qg_quantize_act(y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        got = qg.qg_norm_residual(y, y, w, stream=torch.cuda.default_stream())
        again = qg.qg_quantize_act(y, stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, *again), (*want, *q)))
