"""One decoder layer on raw GGUF blocks: the quantized projections with the norms, rotary positions,
paged cache and attention between them, for a prompt's chunks and for single tokens.

    python examples/decoder_layer.py [--cache q8]

Weights are random Q4_K blocks (grouped-query attention with head norms, SwiGLU FFN).  A batch of
prompts goes through in chunks, then every sequence takes single tokens; the time of each and the
agreement with the same layer in plain fp32 torch are printed.
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import gguf_block_quantized_quant_gb300 as qg
import synth


def weights(N, K, g):
    """Raw Q4_K blocks of N x K random weights around zero, standard deviation about K ** -0.5."""
    W = synth.weights(qg.Q4_K, N, K, g).reshape(-1, 144)
    # w = d * scale * code - dmin * min with 6-bit scales and mins and 4-bit codes, all uniform
    d = (g.uniform(0.75, 1.25, W.shape[0]) / (256 * K ** 0.5)).astype(np.float16)
    W[:, 0:2] = d[:, None].view(np.uint8)
    W[:, 2:4] = (7.5 * d.astype(np.float32)).astype(np.float16)[:, None].view(np.uint8)
    return torch.from_numpy(W.reshape(-1)).cuda()


class Layer:
    """hidden -> hidden; 2 norms, qkv and output projections, FFN, all weights Q4_K."""

    def __init__(self, hidden=2048, heads=16, kv_heads=4, dim=128, inter=4096, seed=0):
        self.H, self.h, self.hk, self.D, self.I = hidden, heads, kv_heads, dim, inter
        g = synth.rng(1, salt=seed)
        self.shapes = {"qkv": ((heads + 2 * kv_heads) * dim, hidden), "o": (hidden, heads * dim),
                       "gate": (inter, hidden), "up": (inter, hidden), "down": (hidden, inter)}
        self.W = {n: weights(*s, g) for n, s in self.shapes.items()}
        t = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda n: 1 + 0.1 * torch.randn(n, generator=t, device="cuda")  # noqa: E731
        self.w_attn, self.w_ffn, self.w_out, self.wq, self.wk = w(hidden), w(hidden), w(hidden), w(dim), w(dim)
        turns, self.amp = qg.qg_rope_turns(dim, 10000.0)
        self.turns = turns.cuda()

    def linear(self, name, x):
        n = self.shapes[name][0]
        # up to 16 tokens the GEMV on int8 activations, beyond the tensor-core GEMM
        return qg.qg_gemv(qg.Q4_K, self.W[name], x, n) if x.shape[0] <= 16 else qg.qg_prefill_gemm(qg.Q4_K, self.W[name], x, n)

    def ffn(self, x):
        if x.shape[0] <= 16:
            return qg.qg_ffn_sublayer(qg.Q4_K, self.W["gate"], self.W["up"], self.W["down"], x, self.I)
        h = torch.nn.functional.silu(self.linear("gate", x)).mul_(self.linear("up", x))
        return self.linear("down", h)

    def __call__(self, res, cache, q_start, kv_len, pages, max_new):
        """res (tokens, hidden) fp32 -> (res after the layer, its norm for the next one)."""
        T, h, hk, D = res.shape[0], self.h, self.hk, self.D
        _, x = qg.qg_norm_residual(res, None, self.w_attn)
        qkv = self.linear("qkv", x)
        q, k, v = (t.view(T, -1, D) for t in qkv.split([h * D, hk * D, hk * D], dim=1))
        q = qg.qg_rope_append(q, k, v, self.turns, cache.k, cache.v, q_start, kv_len, pages, kd=cache.kd, vd=cache.vd, amp=self.amp,
                              wq=self.wq, wk=self.wk)
        o = qg.qg_attn_paged(q, cache.k, cache.v, q_start, kv_len, pages, kd=cache.kd, vd=cache.vd, max_new=max_new, out_dtype=torch.float32)
        res, x = qg.qg_norm_residual(self.linear("o", o.view(T, h * D)), res, self.w_ffn)
        return qg.qg_norm_residual(self.ffn(x), res, self.w_out)

    def plain(self, res, lengths):
        """The layer in fp32 torch for whole sequences of the given lengths (rows of res back to back)."""
        if not hasattr(self, "F"):
            self.F = {n: qg.qg_dequant_f16(qg.Q4_K, self.W[n], *s).view(torch.float16).float() for n, s in self.shapes.items()}
        rms = lambda t, w: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
        T, h, hk, D = res.shape[0], self.h, self.hk, self.D
        qkv = rms(res, self.w_attn) @ self.F["qkv"].T
        q, k, v = (t.view(T, -1, D) for t in qkv.split([h * D, hk * D, hk * D], dim=1))
        freq = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") * 2 / D)
        pos = torch.cat([torch.arange(n, device="cuda") for n in lengths])
        ang = pos.double()[:, None] * freq
        c, s = ang.cos().float()[:, None], ang.sin().float()[:, None]

        def turn(t):
            a, b = t[..., :D // 2], t[..., D // 2:]
            return torch.cat((a * c - b * s, b * c + a * s), -1)
        q, k = turn(rms(q, self.wq)), turn(rms(k, self.wk))
        out, at = [], 0
        for n in lengths:
            qq, kk, vv = q[at:at + n].transpose(0, 1), k[at:at + n].transpose(0, 1), v[at:at + n].transpose(0, 1)
            kk, vv = kk.repeat_interleave(h // hk, 0), vv.repeat_interleave(h // hk, 0)
            z = qq @ kk.transpose(1, 2) * D ** -0.5
            z = z.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
            out.append((z.softmax(-1) @ vv).transpose(0, 1).reshape(n, h * D))
            at += n
        res = res + torch.cat(out) @ self.F["o"].T
        x = rms(res, self.w_ffn)
        res = res + (torch.nn.functional.silu(x @ self.F["gate"].T) * (x @ self.F["up"].T)) @ self.F["down"].T
        return res, rms(res, self.w_out)


class Cache:
    """A pool of pages and each sequence's page table."""

    def __init__(self, kind, batch, longest, kv_heads, dim, page=32):
        width = -(-longest // page)
        shape = (batch * width, kv_heads, page, dim)
        dtype = {"f16": torch.float16, "bf16": torch.bfloat16, "q8": torch.int8}[kind]
        self.k, self.v = (torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(2))
        self.kd = self.vd = None
        if kind == "q8":
            self.kd, self.vd = (torch.zeros(shape[:3] + (dim // 32,), dtype=torch.float16, device="cuda") for _ in range(2))
        self.pages = torch.randperm(batch * width, device="cuda").to(torch.int32).view(batch, width)


def run(layer, kind, prompts, steps, chunk=256, seed=1):
    """Prompts of the given lengths in chunks, then `steps` single tokens each.  Returns the layer's
    outputs per sequence, the inputs, and the seconds of both parts."""
    B = len(prompts)
    total = [n + steps for n in prompts]
    g = torch.Generator(device="cuda").manual_seed(seed)
    xs = [torch.randn((n, layer.H), generator=g, device="cuda") for n in total]
    cache = Cache(kind, B, max(total), layer.hk, layer.D)
    outs, done, spent = [[] for _ in range(B)], [0] * B, [0.0, 0.0]
    while any(d < t for d, t in zip(done, total)):
        new = [min(chunk, p - d) if d < p else int(d < t) for d, p, t in zip(done, prompts, total)]
        if any(d < p for d, p in zip(done, prompts)):
            new = [n if d < p else 0 for n, d, p in zip(new, done, prompts)]
        rows = torch.cat([x[d:d + n] for x, d, n in zip(xs, done, new)])
        q_start = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
        kv_len = torch.tensor([d + n for d, n in zip(done, new)], dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        res, x = layer(rows, cache, q_start, kv_len, cache.pages, max(new))
        torch.cuda.synchronize()
        spent[int(max(new) == 1)] += time.perf_counter() - t0
        at = 0
        for b, n in enumerate(new):
            outs[b].append(res[at:at + n])
            at += n
        done = [d + n for d, n in zip(done, new)]
    return [torch.cat(o) for o in outs], xs, spent


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--cache", choices=("f16", "bf16", "q8"), default="f16")
    a = ap.parse_args()
    layer, prompts, steps = Layer(), [1000, 37, 600, 1], 32
    run(layer, a.cache, [40, 3], 2)  # loads the kernels
    outs, xs, (chunks, singles) = run(layer, a.cache, prompts, steps)
    print(f"prompts of {prompts}: {sum(prompts)} tokens in {chunks * 1e3:.2f} ms; {steps} steps of {len(prompts)} tokens: "
          f"{singles / steps * 1e6:.0f} us each")
    want, _ = layer.plain(torch.cat(xs), [x.shape[0] for x in xs])
    got, x = torch.cat(outs), torch.cat(xs)
    print(f"difference from plain fp32 on the layer's change of the residual: {((got - want).norm() / (want - x).norm()).item():.2e}")
    if qg.qg_device_error():
        raise RuntimeError("a kernel reported a bounded-wait timeout")


if __name__ == "__main__":
    main()
