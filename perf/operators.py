"""Workloads of the decoder-layer operators beside the quantized projections: attention over a
paged cache, rotary positions with the append to that cache, and the norms around a residual.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes a
case's inputs on the GPU, ``run()`` is one pass (the plain torch form, or the package's kernels
where ``own`` is true), ``work()`` its least bytes and operations and ``exact()`` its result in
64 bits.  A cache is a pool of pages, each ``kv_heads x page x dim``; row b of ``pages`` lists
the pages of sequence b in order, and its new tokens are the last of its ``kv_len[b]`` slots.
"""
import math
import random

import numpy as np
import torch

own = False

F16, BF16, F32 = "f16", "bf16", "f32"
TYPES = {F16: torch.float16, BF16: torch.bfloat16, F32: torch.float32}
SIZE = {F16: 2, BF16: 2, F32: 4}


# ------------------------------------------------------------------------------------- cases
def _attn(name, heads, kv_heads, dim, dtype, cache, page, batch, new, past, window=0, mix=1):
    return {"name": name, "op": "attn", "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "cache": cache,
            "page": page, "batch": batch, "new_lo": new[0], "new_hi": new[1], "past_lo": past[0], "past_hi": past[1],
            "window": window, "mix": mix}


def _rope(name, heads, kv_heads, dim, rot, style, scaling, source, dtype, cache, page, batch, new, past, qk_norm=False, mix=1):
    return {"name": name, "op": "rope", "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "style": style,
            "scaling": scaling, "source": source, "dtype": dtype, "cache": cache, "page": page, "batch": batch,
            "new_lo": new[0], "new_hi": new[1], "past_lo": past[0], "past_hi": past[1], "qk_norm": qk_norm, "mix": mix}


def _norm(name, rows, width, source, stream, out, post, gate):
    return {"name": name, "op": "norm", "rows": rows, "width": width, "source": source, "stream": stream, "out": out,
            "post": post, "gate": gate}


def listed():
    return [
        # one user's token early in a conversation: the latency of the whole call
        _attn("token 1x700 f16", 32, 8, 128, F16, "same", 64, 1, (1, 1), (700, 700)),
        # one user's token after a long document, 8-bit cache: few heads, so the keys are split
        _attn("token 1x32k q8 d256", 16, 2, 256, F16, "q8", 64, 1, (1, 1), (32000, 32000)),
        # a server's decode step: many users, ragged lengths
        _attn("tokens 64 ragged bf16", 32, 8, 128, BF16, "same", 64, 64, (1, 1), (300, 16000)),
        # the same with an 8-bit cache and wide heads
        _attn("tokens 48 ragged q8 d256", 24, 4, 256, F16, "q8", 32, 48, (1, 1), (100, 12000)),
        # a prompt of 2048 tokens from nothing
        _attn("prompt 2048 f16", 32, 8, 128, F16, "same", 64, 1, (2048, 2048), (0, 0)),
        # a chunk of a long prompt after 28 thousand tokens of it
        _attn("chunk 4096 after 28k bf16", 32, 8, 128, BF16, "same", 64, 1, (4096, 4096), (28000, 28000)),
        # a server's mixed step: chunks of several prompts and single tokens, sliding window
        _attn("mixed 12 window d64", 16, 16, 64, BF16, "same", 16, 12, (1, 700), (1, 6000), 1024, 5),
        # a 512-token chunk on an 8-bit cache with wide heads
        _attn("chunk 512 after 8k q8 d256", 24, 4, 256, F16, "q8", 32, 1, (512, 512), (8000, 8000)),
        # a decode step of 16 users: rotate part of each head with head norms, append
        _rope("rope 16 tokens partial", 16, 2, 256, 64, "half", "none", F32, F16, "same", 32, 16, (1, 1), (100, 8000), True),
        # a long prompt's chunk: whole heads, scaled frequencies, 8-bit cache
        _rope("rope 4096 tokens yarn q8", 32, 8, 128, 128, "half", "yarn", F32, F16, "q8", 64, 1, (4096, 4096), (0, 0)),
        # a decode step: residual and next norm of one token
        _norm("norm 1x5120", 1, 5120, F32, F32, F32, False, False),
        # a prompt's chunk: norms before and after the block, gate, bf16 out
        _norm("norm 4096x5120 gated", 4096, 5120, F32, F32, BF16, True, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "norm"])
    mix = rng.randrange(1 << 20)
    if op == "norm":
        rows = _log_int(rng, 1, 6000)
        width = _log_int(rng, 64, 16384)
        source = rng.choice([F32, F32, F16, BF16])
        stream = rng.choice([F32, source])
        c = _norm("", rows, width, source, stream, rng.choice([F32, F16, BF16]), rng.random() < 0.5, rng.random() < 0.3)
        del c["name"]
        return c
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 6, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    dtype = rng.choice([F16, BF16])
    cache = "q8" if dtype == F16 and rng.random() < 0.5 else "same"
    if op == "rope":
        single = rng.random() < 0.5
        batch = _log_int(rng, 1, 128) if single else _log_int(rng, 1, 4)
        new = (1, 1) if single else (1, _log_int(rng, 2, 4000 // batch))
        rot = dim if rng.random() < 0.5 else 2 * _log_int(rng, 4, dim // 2)
        c = _rope("", heads, kv_heads, dim, rot, rng.choice(["half", "pairs"]), rng.choice(["none", "linear", "yarn"]),
                  rng.choice([F32, F32, dtype]), dtype, cache, page, batch, new, (1, _log_int(rng, 10, 2000)), rng.random() < 0.5, mix)
        del c["name"]
        return c
    if rng.random() < 0.5:
        batch = _log_int(rng, 1, 64)
        longest = _log_int(rng, 30, min(40000, 300000 // batch))
        new, past = (1, rng.choice([1, 1, 1, 2, 4])), (max(1, longest // rng.choice([1, 4, 50])), longest)
    else:
        batch = _log_int(rng, 1, 8)
        wide = max(1, heads * dim // 4096)
        longest, after = _log_int(rng, 16, 4000 // (batch * wide)), _log_int(rng, 16, 24000 // batch)
        new, past = (max(1, longest // rng.choice([1, 4, 50])), longest), (max(1, after // rng.choice([1, 4, 50])), after)
    c = _attn("", heads, kv_heads, dim, dtype, cache, page, batch, new, past, rng.choice([0, 0, 0, 128, 1000]), mix)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, slots in use with them) of each sequence: part of the case, not of the seed."""
    r = random.Random(case["mix"])
    span = lambda lo, hi: lo if hi <= lo else _log_int(r, max(1, lo), hi)  # noqa: E731
    new = [span(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    return new, [n + span(case["past_lo"], case["past_hi"]) for n in new]


def _frequencies(case):
    """(radians per position of each rotated pair in 64 bits, factor of the rotated values)."""
    half, base, factor, original = case["rot"] // 2, 10000.0, 8.0, 4096.0
    f = base ** (-np.arange(half, dtype=np.float64) / half)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "yarn":
        edge = lambda turns: half * math.log(original / (turns * 2 * math.pi)) / math.log(base)  # noqa: E731
        lo, hi = max(math.floor(edge(32.0)), 0), min(math.ceil(edge(1.0)), half - 1)
        ramp = np.clip((np.arange(half) - lo) / max(hi - lo, 1e-3), 0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


# ------------------------------------------------------------------------------------ inputs
def _pool(case, kv_len, g, d):
    """Page pool of a cache with a few spare pages, and each sequence's pages in random order."""
    page, need = case["page"], [-(-n // case["page"]) for n in kv_len]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=d, dtype=torch.int32)
    width = max(need)
    at = np.concatenate([[0], np.cumsum(need)[:-1]])[:, None] + np.minimum(np.arange(width)[None], np.array(need)[:, None] - 1)
    pages = order[torch.from_numpy(at).to(d)].contiguous()
    shape = (total, case["kv_heads"], page, case["dim"])
    s = {"pages": pages, "kd": None, "vd": None}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=g, device=d, dtype=torch.float32 if math.prod(shape) < 1 << 28 else torch.float16)
        if case["cache"] == "q8":
            s[name] = x.mul_(45).round_().clamp_(-127, 127).to(torch.int8)
            s[name + "d"] = (torch.rand(shape[:3] + (case["dim"] // 32,), generator=g, device=d) * 0.02 + 0.012).half()
        else:
            s[name] = x.to(TYPES[case["dtype"]])
        del x
    return s


def prepare(case, seed):
    d = torch.device("cuda")
    g = torch.Generator(device=d).manual_seed(seed)
    if case["op"] == "norm":
        rows, width, source, stream = case["rows"], case["width"], TYPES[case["source"]], TYPES[case["stream"]]
        rand = lambda *shape: torch.randn(shape, generator=g, device=d)  # noqa: E731
        return {"case": case, "y": rand(rows, width).to(source), "res": (3 * rand(rows, width)).to(stream),
                "w_pre": 1 + 0.1 * rand(width), "w_post": 1 + 0.1 * rand(width) if case["post"] else None,
                "gate": (0.5 + 0.2 * rand(rows, width)).to(source) if case["gate"] else None}
    new, kv_len = _lengths(case)
    s = _pool(case, kv_len, g, d)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    total = int(starts[-1])
    s.update(case=case, q_start=torch.from_numpy(starts).to(d), kv_len=torch.tensor(kv_len, dtype=torch.int32, device=d),
             total=total, max_new=max(new), max_len=max(kv_len))
    h, hk, dim = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "attn":
        s["q"] = (2 * torch.randn((total, h, dim), generator=g, device=d)).to(TYPES[case["dtype"]])
        return s
    qkv = torch.randn((total, (h + 2 * hk) * dim), generator=g, device=d).to(TYPES[case["source"]])  # one projection's output
    s["q"] = qkv[:, :h * dim].view(total, h, dim)
    s["nk"] = qkv[:, h * dim:(h + hk) * dim].view(total, hk, dim)
    s["nv"] = qkv[:, (h + hk) * dim:].view(total, hk, dim)
    f, s["amp"] = _frequencies(case)
    turns = [int(t / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for t in f.tolist()]  # 2^-64 turns per position
    s["turns"] = torch.from_numpy(np.array(turns, dtype=np.uint64).view(np.int64)).to(d)
    s["wq"] = s["wk"] = None
    if case["qk_norm"]:
        s["wq"], s["wk"] = (1 + 0.1 * torch.randn(dim, generator=g, device=d) for _ in range(2))
    return s


# ---------------------------------------------------------------------------------- one pass
def _whole(s, name):
    """A pool's values in 32 bits."""
    x = s[name].float()
    if s[name + "d"] is None:
        return x
    return (x.view(x.shape[:3] + (-1, 32)) * s[name + "d"].float().unsqueeze(-1)).view(x.shape)


def _stored(codes, steps):
    """An 8-bit pool as the values it stands for."""
    return (codes.view(steps.shape + (32,)) * steps.unsqueeze(-1)).view(codes.shape)


def _token_rows(s):
    """Sequence, place among its new tokens and position of each new token."""
    t = torch.arange(s["total"], device=s["q_start"].device)
    seq = torch.searchsorted(s["q_start"][1:].contiguous(), t, right=True)
    at = t - s["q_start"][seq]
    new = s["q_start"][1:] - s["q_start"][:-1]
    return seq, at, (s["kv_len"] - new)[seq] + at


def _plain_attn(s):
    c = s["case"]
    b, h, hk, dim, n, length = c["batch"], c["heads"], c["kv_heads"], c["dim"], s["max_new"], s["max_len"]
    seq, at, _ = _token_rows(s)
    q = s["q"].new_zeros((b, n, h, dim), dtype=torch.float32)
    q[seq, at] = s["q"].float() * dim ** -0.5
    q = q.view(b, n, hk, h // hk, dim).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, dim)
    k, v = (_whole(s, w)[s["pages"]].transpose(1, 2).reshape(b, hk, -1, dim)[:, :, :length] for w in ("k", "v"))
    scores = (q @ k.transpose(-1, -2)).view(b, hk, h // hk, n, length)
    del k
    new = s["q_start"][1:] - s["q_start"][:-1]
    row = (s["kv_len"] - new)[:, None] + torch.arange(n, device=q.device)
    key = torch.arange(length, device=q.device)
    seen = key <= row[:, :, None]
    if c["window"]:
        seen &= key > row[:, :, None] - c["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hk, -1, length) @ v).view(b, hk, h // hk, n, dim) / torch.where(total == 0, 1.0, total)
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, h, dim)[seq, at].to(s["q"].dtype)


def _plain_turn(x, cos, sin, rot, style):
    a = x[..., :rot]
    even, odd = (a[..., :rot // 2], a[..., rot // 2:]) if style == "half" else (a[..., 0::2], a[..., 1::2])
    cos, sin = cos[:, None], sin[:, None]
    turned = (even * cos - odd * sin, odd * cos + even * sin)
    turned = torch.cat(turned, -1) if style == "half" else torch.stack(turned, -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rope(s):
    c = s["case"]
    seq, _, position = _token_rows(s)
    turn = ((position.long()[:, None] * s["turns"]) >> 32).float() * 2.0 ** -32  # whole turns drop out
    cos, sin = (turn * (2 * math.pi)).cos() * s["amp"], (turn * (2 * math.pi)).sin() * s["amp"]
    q, k, v = s["q"].float(), s["nk"].float(), s["nv"].float()
    if c["qk_norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["wq"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["wk"]
    q, k = (_plain_turn(x, cos, sin, c["rot"], c["style"]) for x in (q, k))
    page, slot = s["pages"][seq, position // c["page"]], position % c["page"]
    pools = []
    for name, x in (("k", k), ("v", v)):
        if c["cache"] == "q8":
            blocks = x.view(x.shape[:2] + (-1, 32))
            step = blocks.abs().amax(-1) / 127
            codes = torch.where(step[..., None] > 0, blocks / step[..., None], 0.0).round().clamp(-127, 127)
            s[name][page, :, slot] = codes.to(torch.int8).view(x.shape)
            s[name + "d"][page, :, slot] = step.half()
            pools.append(_stored(s[name], s[name + "d"]))
        else:
            s[name][page, :, slot] = x.to(s[name].dtype)
            pools.append(s[name])
    return q.to(TYPES[c["dtype"]]), pools[0], pools[1]


def _plain_norm(s):
    c = s["case"]
    rms = lambda x, w: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
    y = s["y"].float()
    if c["post"]:
        y = rms(y, s["w_post"])
    if c["gate"]:
        y = y * s["gate"].float()
    r = s["res"].float() + 0.5 * y
    return r.to(s["res"].dtype), rms(r, s["w_pre"]).to(TYPES[c["out"]])


def run(s):
    c = s["case"]
    if not own:
        return {"attn": _plain_attn, "rope": _plain_rope, "norm": _plain_norm}[c["op"]](s)
    import gguf_block_quantized_quant_gb300 as qg
    if c["op"] == "attn":
        return qg.qg_attn_paged(s["q"], s["k"], s["v"], s["q_start"], s["kv_len"], s["pages"], kd=s["kd"], vd=s["vd"],
                                max_new=s["max_new"], window=c["window"])
    if c["op"] == "rope":
        q = qg.qg_rope_append(s["q"], s["nk"], s["nv"], s["turns"], s["k"], s["v"], s["q_start"], s["kv_len"], s["pages"],
                              kd=s["kd"], vd=s["vd"], pairs=c["style"] == "pairs", amp=s["amp"], wq=s["wq"], wk=s["wk"],
                              eps=1e-6, q_dtype=TYPES[c["dtype"]])
        if c["cache"] == "q8":
            return q, _stored(s["k"], s["kd"]), _stored(s["v"], s["vd"])
        return q, s["k"], s["v"]
    return qg.qg_norm_residual(s["y"], s["res"], s["w_pre"], w_post=s["w_post"], gate=s["gate"], alpha=0.5, eps=1e-6,
                               x_dtype=TYPES[c["out"]])


# ------------------------------------------------------------------------- what it cannot do without
def work(case):
    if case["op"] == "norm":
        per = SIZE[case["source"]] * (2 if case["gate"] else 1) + 2 * SIZE[case["stream"]] + SIZE[case["out"]]
        n = case["rows"] * case["width"]
        return {"bytes": n * per + 4 * case["width"] * (2 if case["post"] else 1), "flops": n * (12 if case["post"] else 7)}
    new, kv_len = _lengths(case)
    h, hk, dim = case["heads"], case["kv_heads"], case["dim"]
    row = hk * (dim * 34 // 32 if case["cache"] == "q8" else dim * 2)  # bytes of one slot's keys, or values
    table = 4 * sum(-(-n // case["page"]) for n in kv_len) + 8 * case["batch"]
    if case["op"] == "rope":
        t = sum(new)
        moved = t * dim * (SIZE[case["source"]] * (h + 2 * hk) + SIZE[case["dtype"]] * h) + 2 * t * row
        return {"bytes": moved + 4 * case["rot"] + 8 * case["batch"] + 4 * case["batch"], "flops": 3 * t * case["rot"] * (h + hk)}
    window = case["window"] or 1 << 60
    slots = sum(n - max(0, n - m - window + 1) for m, n in zip(new, kv_len))
    # a row at position p sees min(p + 1, window) keys
    upto = lambda x: x * (x + 1) // 2 if x <= window else window * (window + 1) // 2 + (x - window) * window  # noqa: E731
    pairs = sum(upto(n) - upto(n - m) for m, n in zip(new, kv_len))
    return {"bytes": 2 * slots * row + 2 * sum(new) * h * dim * SIZE[case["dtype"]] + table, "flops": 4 * dim * h * pairs}


# ------------------------------------------------------------------------------ in 64 bits
def _exact_pool(s, name):
    x = s[name].double()
    if s[name + "d"] is not None:
        x *= s[name + "d"].double().repeat_interleave(32, -1)
    return x


def _exact_attn(case, s):
    starts, lens, group = s["q_start"].tolist(), s["kv_len"].tolist(), case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b, length in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        ids = s["pages"][b, :-(-length // case["page"])].long()
        for j in range(case["kv_heads"]):
            part = {w: s[w][ids, j] for w in ("k", "v")}
            part.update({w + "d": None if s[w + "d"] is None else s[w + "d"][ids, j] for w in ("k", "v")})
            k, v = (_exact_pool(part, w).reshape(-1, case["dim"])[:length] for w in ("k", "v"))
            for first in range(lo, hi, 512):
                rows = torch.arange(first, min(hi, first + 512), device=k.device)
                distance = (length - (hi - rows))[:, None] - torch.arange(length, device=k.device)[None]
                off = distance < 0
                if case["window"]:
                    off |= distance >= case["window"]
                for i in range(group):
                    head = j * group + i
                    z = torch.einsum("td,sd->ts", s["q"][rows, head].double(), k) / math.sqrt(case["dim"])
                    out[rows, head] = torch.softmax(z.masked_fill(off, -math.inf), -1) @ v
    return out


def _exact_rope(case, s):
    f, amp = _frequencies(case)
    f = torch.from_numpy(f).to(s["q"].device)
    starts, lens, rot = s["q_start"].tolist(), s["kv_len"].tolist(), case["rot"]
    first, second = ((slice(0, rot // 2), slice(rot // 2, rot)) if case["style"] == "half" else (slice(0, rot, 2), slice(1, rot, 2)))
    out = s["q"].double()
    pools = [_exact_pool(s, "k"), _exact_pool(s, "v")]
    for b, length in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        position = torch.arange(length - (hi - lo), length, device=out.device)
        angle = position.double()[:, None] * f
        cos, sin = amp * torch.cos(angle)[:, None], amp * torch.sin(angle)[:, None]
        turned = {}
        for name, w in (("q", s["wq"]), ("nk", s["wk"])):
            x = s[name][lo:hi].double()
            if w is not None:
                x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
            z = x.clone()
            z[..., first], z[..., second] = x[..., first] * cos - x[..., second] * sin, x[..., second] * cos + x[..., first] * sin
            turned[name] = z
        out[lo:hi] = turned["q"]
        where = s["pages"][b][position // case["page"]].long()
        for pool, x in zip(pools, (turned["nk"], s["nv"][lo:hi].double())):
            if case["cache"] == "q8":
                blocks = x.reshape(x.shape[0], x.shape[1], -1, 32)
                step = blocks.abs().amax(-1, keepdim=True) / 127
                x = ((blocks / step.clamp_min(1e-300)).round() * step.half().double()).reshape(x.shape)
            pool[where, :, position % case["page"]] = x
    return out, pools[0], pools[1]


def _exact_norm(case, s):
    def rms(x, w):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
    t = s["y"].double()
    t = rms(t, s["w_post"]) if case["post"] else t
    t = t * s["gate"].double() if case["gate"] else t
    r = s["res"].double() + t / 2
    return r, rms(r, s["w_pre"])


def exact(case, seed):
    if work(case)["flops"] > 6e12:  # over 20 seconds in 64 bits
        return None
    return {"attn": _exact_attn, "rope": _exact_rope, "norm": _exact_norm}[case["op"]](case, prepare(case, seed))
