"""Plain 64-bit forms of the decoder-layer operators for the GPU tests (not collected as tests)."""
import math

import numpy as np
import torch

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
# largest relative error of one rounding to the type
UNIT = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make_cache(kind, n_pages, heads, page, dim, g, nhd=False):
    """Pools (k, v, kd, vd) of shape (pages, heads, page, dim); nhd: slots before heads in memory."""
    shape = (n_pages, page, heads, dim) if nhd else (n_pages, heads, page, dim)
    out = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device="cuda")
        if kind == "q8":
            x = (x * 45).round().clamp(-127, 127).to(torch.int8)
        else:
            x = x.to(kind)
        out.append(x.transpose(1, 2) if nhd else x)
    steps = [None, None]
    if kind == "q8":
        steps = [(torch.rand((n_pages, heads, page, dim // 32), generator=g, device="cuda") * 0.02 + 0.012).half() for _ in range(2)]
    return out[0], out[1], steps[0], steps[1]


def tables(new, kv_len, page, spare, g):
    """(q_start, kv_len, pages, n_pages): random distinct pages, -1 where a sequence has none."""
    need = [max(0, -(-n // page)) for n in kv_len]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    width = max(max(need), 1) + 1
    pages = torch.full((len(new), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        pages[b, :n] = order[at:at + n]
        at += n
    starts = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    return starts, torch.tensor(kv_len, dtype=torch.int32, device="cuda"), pages, n_pages


def values(x, steps):
    x = x.double()
    return x if steps is None else x * steps.double().repeat_interleave(32, -1)


def sequence(pool, steps, pages_b, length):
    """(heads, length, dim) values of one sequence in 64 bits."""
    page = pool.shape[2]
    ids = pages_b[:-(-length // page)].long()
    x = values(pool[ids], None if steps is None else steps[ids])
    return x.transpose(0, 1).reshape(pool.shape[1], -1, pool.shape[3])[:, :length]


def attention(q, k, v, kd, vd, new, kv_len, pages, scale, window):
    """(o, lse, A, B): result, natural log of the sums, sum of p |v| and the largest
    scale * sum |q k| of each row (for error bounds)."""
    T, H, D = q.shape
    G = H // k.shape[1]
    o = torch.zeros((T, H, D), dtype=torch.float64, device=q.device)
    A = torch.zeros_like(o)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    B = torch.zeros((T, H), dtype=torch.float64, device=q.device)
    t0 = 0
    for b, (n, L) in enumerate(zip(new, kv_len)):
        if n and L:
            kk, vv = sequence(k, kd, pages[b], L), sequence(v, vd, pages[b], L)
            qq = q[t0:t0 + n].double().transpose(0, 1).reshape(-1, G, n, D)
            z = (qq @ kk[:, None].transpose(-1, -2)) * scale
            mag = (qq.abs() @ kk[:, None].abs().transpose(-1, -2)) * abs(scale)
            pos = torch.arange(L - n, L, device=q.device)[:, None]
            key = torch.arange(L, device=q.device)[None]
            see = key <= pos
            if window:
                see = see & (key > pos - window)
            z = z.masked_fill(~see, -math.inf)
            m = z.amax(-1, keepdim=True)
            p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
            s = p.sum(-1, keepdim=True)
            p = p / torch.where(s == 0, 1.0, s)
            back = lambda x: x.reshape(H, n, -1).transpose(0, 1)  # noqa: E731
            o[t0:t0 + n] = back(p @ vv[:, None])
            A[t0:t0 + n] = back(p @ vv[:, None].abs())
            lse[t0:t0 + n] = back(torch.where(s == 0, -math.inf, m + torch.log(s)))[..., 0]
            B[t0:t0 + n] = back(mag.masked_fill(~see, 0.0).amax(-1, keepdim=True))[..., 0]
        t0 += n
    return o, lse, A, B


def attention_bound(o, A, B, dtype, out_dtype, q8, exact_p=False):
    """Bound of |out - o| per element, u the unit rounding of the type:
      u_out |o|                  the one rounding of the result,
      (u_P + u_V) A              probabilities rounded before the value sum (none where they go in
                                 as two addends: exact_p), 8-bit values rounded to fp16,
      2 dS A                     scores off by dS: p and the normaliser each by a factor 1 +- dS;
                                 dS = 2^-18 B (fp32 sums of up to 256 products and the base-2
                                 exponent's rounding) + 2^-11 B where 8-bit keys are rounded,
      2^-16 A                    exponentials and sums in fp32; two addends of 8 bits leave 2^-16."""
    u_p = 0.0 if exact_p else UNIT[dtype]
    ds = 2.0 ** -18 * B + (2.0 ** -11 * B if q8 and not exact_p else 0.0)
    c = u_p + (UNIT[F16] if q8 else 0.0) + 2.0 ** -16 + 2 * ds[..., None]
    return UNIT[out_dtype] * o.abs() + c * A + 2.0 ** -24


def within(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: {int((~torch.isfinite(got)).sum())} values are not finite"
    ratio = ((got - want).abs() / bound).max().item() if got.numel() else 0.0
    assert ratio <= 1.0, f"{what}: worst error / bound {ratio:.3f}"
    return ratio
