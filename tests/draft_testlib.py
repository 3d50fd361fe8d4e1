"""Plain 64-bit forms of shaped and tree attention and of the logits' penalties (not collected as tests)."""
import math

import torch

from layer_testlib import F16, UNIT, sequence


def intervals(new, kv_len, window=0, prefix=None, first=None):
    """Per sequence (see, distance): which slots each new token sees, and how far they are.  prefix: a list,
    one per sequence; first: a list, one per token."""
    out, t0 = [], 0
    for b, (n, L) in enumerate(zip(new, kv_len)):
        p = torch.arange(L - n, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None]
        last = p if prefix is None else p.clamp(min=prefix[b] - 1)
        see = (j <= last) & (p >= 0)
        if window:
            see &= j > p - window
        if first is not None:
            see &= j >= torch.tensor(first[t0:t0 + n], device="cuda", dtype=torch.long)[:, None]
        out.append((see, (p - j).abs()))
        t0 += n
    return out


def ancestors(parents):
    """(bits of each draft's row as a Python integer, depth) from the parents of one sequence."""
    bits, depth = [], []
    for i, p in enumerate(parents):
        ok = 0 <= p < i
        bits.append((bits[p] if ok else 0) | 1 << i)
        depth.append(depth[p] + 1 if ok else 0)
    return bits, depth


def words_of(bits, words):
    """int32 (rows, words) of rows of bits."""
    rows = [[(b >> 32 * w) & 0xffffffff for w in range(words)] for b in bits]
    return torch.tensor([[x - (1 << 32) if x >> 31 else x for x in r] for r in rows], dtype=torch.int64, device="cuda").int()


def trees(new, kv_len, bits, positions=None, window=0, words=1):
    """As intervals(), for drafts whose rows have these bits (a list, one per token)."""
    out, t0 = [], 0
    for n, L in zip(new, kv_len):
        base = L - n
        see = torch.zeros((n, L), dtype=torch.bool)
        place = torch.arange(L)
        at = [base + i if positions is None else positions[t0 + i] for i in range(n)]
        for i in range(n):
            if base + i < 0:
                continue
            for j in range(min(n, 32 * words)):
                if base + j >= 0:
                    see[i, base + j] = bool(bits[t0 + i] >> j & 1)
            if base > 0:
                see[i, :base] = place[:base] > at[i] - window if window else True
        for j in range(n):
            if base + j >= 0:
                place[base + j] = at[j]
        dist = (torch.tensor(at).view(-1, 1) - place[None]).abs() if n else torch.zeros((0, L))
        out.append((see.cuda(), dist.cuda()))
        t0 += n
    return out


def attention(q, k, v, kd, vd, new, kv_len, pages, scale, views, cap=0.0, slopes=None, q8=False):
    """(o, lse, A, W, D): the result, the logarithm of the sums, sum of p |v|, and what errors of the scores make of a result and
    of the logarithm, to first order: with delta_j the largest error of score j, sum p delta |v| + (sum p delta) A and sum p delta.

    delta: the raw score as in plain attention, 2^-18 of the row's largest sum |q k| scale (and 2^-11 of it where 8-bit
    keys are rounded to fp16; a cap makes neither larger); 2^-19 of the capped score's size (the fit of tanh is off by 7e-7
    relative, 2^-20.4, and the products around it by 2^-24 each; where 1 - 2 / (1 + e) is used the score is at least 0.63 caps
    and 1, 2 r, e and r are off by 2^-24, 2^-22, 2^-22); 2^-21 of the bias (a product, its factor's, a difference); 2^-22 of the
    row's maximum, the exponent's rounding."""
    T, H, D_ = q.shape
    G = H // k.shape[1]
    o = torch.zeros((T, H, D_), dtype=torch.float64, device=q.device)
    A, W = torch.zeros_like(o), torch.zeros_like(o)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    D = torch.zeros((T, H), dtype=torch.float64, device=q.device)
    t0 = 0
    for b, (n, L) in enumerate(zip(new, kv_len)):
        if n and L:
            kk, vv = sequence(k, kd, pages[b], L), sequence(v, vd, pages[b], L)
            qq = q[t0:t0 + n].double().transpose(0, 1).reshape(-1, G, n, D_)
            see, dist = views[b]
            z = (qq @ kk[:, None].transpose(-1, -2)) * scale
            mag = (qq.abs() @ kk[:, None].abs().transpose(-1, -2)) * abs(scale)
            delta = (2.0 ** -18 + (2.0 ** -11 if q8 else 0.0)) * torch.where(see, mag, 0.0).amax(-1, keepdim=True).expand_as(z).clone()
            if cap:
                z = cap * torch.tanh(z / cap)
                delta += 2.0 ** -19 * z.abs()
            if slopes is not None:
                s = slopes.double().view(-1, G, 1, 1) * dist.double()
                z = z - s
                delta += 2.0 ** -21 * s.abs()
            z = z.masked_fill(~see, -math.inf)
            m = z.amax(-1, keepdim=True)
            m0 = torch.where(m == -math.inf, 0.0, m)
            delta += 2.0 ** -22 * m0.abs()
            p = torch.exp(z - m0)
            s = p.sum(-1, keepdim=True)
            p = p / torch.where(s == 0, 1.0, s)
            pd = torch.where(see, p * delta, 0.0)
            back = lambda x: x.reshape(H, n, -1).transpose(0, 1)  # noqa: E731
            vz = vv.nan_to_num(0.0, 0.0, 0.0)[:, None]  # slots that nobody sees may hold anything
            o[t0:t0 + n], A[t0:t0 + n] = back(p @ vz), back(p @ vz.abs())
            D[t0:t0 + n] = back(pd.sum(-1, keepdim=True))[..., 0]
            W[t0:t0 + n] = back(pd @ vz.abs()) + D[t0:t0 + n][..., None] * A[t0:t0 + n]
            lse[t0:t0 + n] = back(torch.where(s == 0, -math.inf, m0 + torch.log(s)))[..., 0]
        t0 += n
    return o, lse, A, W, D


def bounds(o, lse, A, W, D, dtype, out_dtype, q8):
    """Bounds of out and of lse: the result's rounding, probabilities and 8-bit values rounded before their product, 2^-16 for
    exponentials and sums in fp32, and the scores' errors (a tenth more for what first order leaves out)."""
    out = UNIT[out_dtype] * o.abs() + (UNIT[dtype] + (UNIT[F16] if q8 else 0.0) + 2.0 ** -16) * A + 1.1 * W + 2.0 ** -24
    return out, 1.1 * D + 2.0 ** -18 + 2.0 ** -22 * lse.nan_to_num(0.0, 0.0, 0.0).abs()
