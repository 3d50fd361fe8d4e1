"""Workloads of the operators around drafted tokens and shaped scores: attention over a paged cache
with capped scores, a distance bias, a document or a prefix mask; attention of trees of drafted
tokens; penalties, biases and grammar masks on logits; and the accepted drafts moved together in
the cache.

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
def _shaped(name, heads, kv_heads, dim, dtype, cache, page, batch, new, past, cap=0.0, bias=False, docs=0, prefix=False, window=0, mix=1):
    """docs: documents that a sequence's new tokens hold, each of which sees itself alone, before a last part that
    sees all.  prefix: a first part of each sequence whose tokens see all of it."""
    return {"name": name, "op": "shaped", "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "cache": cache,
            "page": page, "batch": batch, "new_lo": new[0], "new_hi": new[1], "past_lo": past[0], "past_hi": past[1],
            "cap": cap, "bias": bias, "docs": docs, "prefix": prefix, "window": window, "mix": mix}


def _tree(name, heads, kv_heads, dim, dtype, cache, page, batch, new, past, cap=0.0, bias=False, window=0, mix=1):
    return {"name": name, "op": "tree", "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "cache": cache,
            "page": page, "batch": batch, "new_lo": new[0], "new_hi": new[1], "past_lo": past[0], "past_hi": past[1],
            "cap": cap, "bias": bias, "docs": 0, "prefix": False, "window": window, "mix": mix}


def _logits(name, vocab, dtype, out, batch, drafts, history, bias=0, grammar=True, mix=1):
    """drafts: drafted tokens of a sequence, a row of logits each (1: a row per sequence, no tree)."""
    return {"name": name, "op": "logits", "vocab": vocab, "dtype": dtype, "out": out, "batch": batch, "drafts": drafts,
            "hist_lo": history[0], "hist_hi": history[1], "bias": bias, "grammar": grammar, "mix": mix}


def _keep(name, layers, kv_heads, dim, dtype, page, batch, new, kept, past, mix=1):
    return {"name": name, "op": "keep", "layers": layers, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "cache": "same", "page": page,
            "batch": batch, "new_lo": new, "new_hi": new, "kept": kept, "past_lo": past[0], "past_hi": past[1], "mix": mix}


def listed():
    return [
        # one user's token early in a conversation, capped scores and a window: the latency of the whole call
        _shaped("capped token 1x900 f16 d256", 16, 8, 256, F16, "same", 64, 1, (1, 1), (900, 900), cap=50.0, window=4096),
        # a server's decode step with capped scores: many users, ragged lengths
        _shaped("capped tokens 64 ragged bf16", 32, 8, 128, BF16, "same", 64, 64, (1, 1), (300, 16000), cap=50.0),
        # a chunk of a long prompt with capped scores
        _shaped("capped chunk 2048 after 6k bf16", 32, 8, 128, BF16, "same", 64, 1, (2048, 2048), (6000, 6000), cap=50.0),
        # prompts of several users, scores that fall with the distance, a key per head
        _shaped("distance 6 prompts f16", 24, 24, 128, F16, "same", 32, 6, (100, 1500), (1, 500), bias=True),
        # retrieved documents that do not see each other and the question after them, heads of 64, behind a shared prefix
        _shaped("documents 4 x 2000 d64", 16, 4, 64, F16, "same", 64, 4, (1600, 2400), (1, 1), docs=6, prefix=True),
        # one user's 16 drafted tokens: the latency of the whole call
        _tree("tree 1 x 16 after 700 f16", 32, 8, 128, F16, "same", 64, 1, (16, 16), (700, 700)),
        # a server's verification step: 32 users, a tree of 8 to 48 drafts each
        _tree("trees 32 ragged bf16", 32, 8, 128, BF16, "same", 64, 32, (8, 48), (300, 16000)),
        # the same with an 8-bit cache, wide heads and capped scores
        _tree("trees 24 ragged q8 d256 capped", 16, 4, 256, F16, "q8", 32, 24, (4, 24), (100, 12000), cap=30.0),
        # logits of one user's next token with penalties
        _logits("logits 1x32000 f32", 32000, F32, F32, 1, 1, (600, 600), grammar=False),
        # logits of the drafts of 16 users, bf16, with penalties, biases and a grammar for each row
        _logits("logits 16x12 of 131071 bf16", 131071, BF16, F32, 16, 12, (200, 6000), bias=100),
        # one user's accepted drafts in one layer
        _keep("keep 5 of 16, 1 layer f16", 1, 8, 128, F16, 64, 1, 16, 5, (700, 700)),
        # a server's accepted drafts in all layers
        _keep("keep 6 of 48, 32 x 16 layers bf16", 16, 8, 128, BF16, 32, 32, 48, 6, (16, 200)),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["shaped", "shaped", "tree", "tree", "logits", "keep"])
    mix = rng.randrange(1 << 20)
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 6, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    dtype = rng.choice([F16, BF16])
    cache = "q8" if dtype == F16 and rng.random() < 0.4 else "same"
    cap = rng.choice([0.0, 20.0, 30.0, 50.0])
    if op == "logits":
        drafts = rng.choice([1, 1, _log_int(rng, 2, 60)])
        rows = _log_int(rng, 1, 190)
        c = _logits("", _log_int(rng, 900, 131071), rng.choice([F32, F32, F16, BF16]), F32, max(1, rows // drafts), drafts,
                    (1, _log_int(rng, 4, 6000)), rng.choice([0, 3, 100]), rng.random() < 0.6, mix)
        if rng.random() < 0.3:
            c["out"] = c["dtype"]
    elif op == "keep":
        new = _log_int(rng, 2, 48)
        c = _keep("", _log_int(rng, 1, 16), kv_heads, dim, dtype, page, _log_int(rng, 1, 128 // kv_heads), new,
                  rng.randint(1, max(1, min(8, new // 2))), (10, _log_int(rng, 11, 200)), mix)
    elif op == "tree":
        batch = _log_int(rng, 1, 32)
        drafts = _log_int(rng, 2, min(200, 1500 // batch))
        longest = _log_int(rng, 30, 200000 // batch if batch > 12 else 16000)
        c = _tree("", heads, kv_heads, dim, dtype, cache, page, batch, (max(1, drafts // rng.choice([1, 4])), drafts),
                  (max(1, longest // rng.choice([1, 4, 50])), longest), cap, rng.random() < 0.3, rng.choice([0, 0, 500]), mix)
    else:
        style = rng.choice(["cap", "bias", "docs", "prefix", "all"])
        opts = {"cap": cap or 50.0 if style in ("cap", "all") else 0.0, "bias": style in ("bias", "all"),
                "docs": rng.randint(2, 7) if style in ("docs", "all") else 0, "prefix": style in ("prefix", "all"),
                "window": rng.choice([0, 0, 200, 1000])}
        if rng.random() < 0.4 and style != "docs":
            batch = _log_int(rng, 1, 64)
            longest = _log_int(rng, 30, min(20000, 300000 // batch))
            new, past = (1, rng.choice([1, 1, 1, 3])), (max(1, longest // rng.choice([1, 4, 50])), longest)
        else:
            batch = _log_int(rng, 1, 6)
            wide = max(1, heads * dim // 4096)
            longest, after = _log_int(rng, 16, 2000 // (batch * wide)), _log_int(rng, 16, 6000 // batch)
            new, past = (max(1, longest // rng.choice([1, 4, 50])), longest), (max(1, after // rng.choice([1, 4, 50])), after)
        c = _shaped("", heads, kv_heads, dim, dtype, cache, page, batch, new, past, mix=mix, **opts)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, slots in use with them) of each sequence: part of the case, not of the seed."""
    r = random.Random(case["mix"])
    span = lambda lo, hi: lo if hi <= lo else _log_int(r, max(1, lo), hi)  # noqa: E731
    new = [span(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    return new, [n + span(case["past_lo"], case["past_hi"]) for n in new]


def _layout(case):
    """Per sequence: (first slot of each new token's document, length of the prefix)."""
    r = random.Random(case["mix"] + 1)
    firsts, prefixes = [], []
    for n, length in zip(*_lengths(case)):
        base = length - n
        first = [0] * n
        if case["docs"]:
            ends = sorted(r.randrange(n + 1) for _ in range(case["docs"]))
            for lo, hi in zip([0] + ends[:-1], ends):
                first[lo:hi] = [base + lo if lo else 0] * (hi - lo)  # the first one continues what was there
        firsts.append(first)
        prefixes.append(r.randrange(length // 2 + 1) if case["prefix"] else 0)
    return firsts, prefixes


def _parents(case):
    """Per sequence: each drafted token's parent among them (-1: the committed text), breadth first as drafts come."""
    r = random.Random(case["mix"] + 2)
    new = _lengths(case)[0] if case["op"] != "logits" else [case["drafts"]] * case["batch"]
    return [[-1] + [r.randrange(max(0, i - 1 - i // 2), i) for i in range(1, n)] for n in new]


def _slopes(heads):
    return 2.0 ** (-8.0 * np.arange(1, heads + 1) / heads)


# ------------------------------------------------------------------------------------ inputs
def _pool(case, kv_len, g, d, layers=None):
    """Page pool of a cache with a few spare pages, and each sequence's pages in random order."""
    page, need = case["page"], [-(-n // case["page"]) for n in kv_len]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=d, dtype=torch.int32)
    width = max(need)
    at = np.concatenate([[0], np.cumsum(need)[:-1]])[:, None] + np.minimum(np.arange(width)[None], np.array(need)[:, None] - 1)
    shape = ((layers,) if layers else ()) + (total, case["kv_heads"], page, case["dim"])
    s = {"pages": order[torch.from_numpy(at).to(d)].contiguous(), "kd": None, "vd": None}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=g, device=d, dtype=torch.float32 if math.prod(shape) < 1 << 28 else torch.float16)
        if case["cache"] == "q8":
            s[name] = x.mul_(45).round_().clamp_(-127, 127).to(torch.int8)
            s[name + "d"] = (torch.rand(shape[:3] + (case["dim"] // 32,), generator=g, device=d) * 0.02 + 0.012).half()
        else:
            s[name] = x.to(TYPES[case["dtype"]])
        del x
    return s


def _tree_inputs(parents, d):
    """(mask words of each drafted token, its depth) from the parents, as int32 tensors."""
    words = max(-(-len(p) // 32) for p in parents)
    rows, depths = [], []
    for parent in parents:
        bits, depth = [], []
        for i, p in enumerate(parent):
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
            depth.append(depth[p] + 1 if p >= 0 else 0)
        rows += [[b >> 32 * w & 0xffffffff for w in range(words)] for b in bits]
        depths += depth
    return (torch.from_numpy(np.array(rows, dtype=np.uint32).view(np.int32)).to(d),
            torch.tensor(depths, dtype=torch.int32, device=d))


def _prepare_logits(case, g, d):
    r = random.Random(case["mix"] + 3)
    b, n, v = case["batch"], case["drafts"], case["vocab"]
    span = [case["hist_lo"] if case["hist_hi"] <= case["hist_lo"] else _log_int(r, case["hist_lo"], case["hist_hi"]) for _ in range(b)]
    rand = lambda *shape: torch.rand(shape, generator=g, device=d)  # noqa: E731
    ids = lambda *shape: (rand(*shape).square_() * v).int().clamp_(max=v - 1)  # noqa: E731  some ids come often
    s = {"case": case, "x": (3 * torch.randn((b * n, v), generator=g, device=d)).to(TYPES[case["dtype"]]),
         "history": ids(b, max(span)), "history_len": torch.tensor(span, dtype=torch.int32, device=d),
         "prompt_len": torch.tensor([x // 2 for x in span], dtype=torch.int32, device=d),
         "repetition": 1 + 0.5 * rand(b), "frequency": 0.3 * rand(b), "presence": 0.5 * rand(b),
         "seq": None, "q_start": None, "drafts": None, "tree": None, "bias_start": None, "bias_ids": None, "bias": None, "allow": None}
    if n > 1:
        s["seq"] = torch.arange(b, device=d, dtype=torch.int32).repeat_interleave(n)
        s["q_start"] = torch.arange(0, b * n + 1, n, device=d, dtype=torch.int32)
        s["drafts"] = ids(b * n)
        s["tree"], _ = _tree_inputs(_parents(case), d)
    if case["bias"]:
        k = min(case["bias"], v)
        s["bias_start"] = torch.arange(0, b * k + 1, k, device=d, dtype=torch.int32)
        s["bias_ids"] = torch.cat([torch.randperm(v, generator=g, device=d)[:k] for _ in range(b)]).int()
        s["bias"] = 4 * rand(b * k) - 2
    if case["grammar"]:  # a quarter of the ids, at random
        w = torch.randint(-1 << 31, 1 << 31, (2, b * n, -(-v // 32)), generator=g, device=d).int()
        s["allow"] = w[0] & w[1]
    return s


def prepare(case, seed):
    d = torch.device("cuda")
    g = torch.Generator(device=d).manual_seed(seed)
    if case["op"] == "logits":
        return _prepare_logits(case, g, d)
    new, kv_len = _lengths(case)
    s = _pool(case, kv_len, g, d, case.get("layers"))
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    total = int(starts[-1])
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=d)  # noqa: E731
    s.update(case=case, q_start=torch.from_numpy(starts).to(d), kv_len=ints(kv_len), total=total, max_new=max(new), max_len=max(kv_len))
    if case["op"] == "keep":
        # the root and a path below it, whose places lie past the kept ones: a pass can be done again
        m, n = case["kept"], new[0]
        paths = [random.Random(case["mix"] * 131 + b) for b in range(case["batch"])]
        s["keep"] = ints([[0] + sorted(r.sample(range(m, n), m - 1)) for r in paths])
        s["keep_len"] = ints([m - b % 2 if m > 1 else m for b in range(case["batch"])])
        return s
    h, dim = case["heads"], case["dim"]
    s["q"] = (2 * torch.randn((total, h, dim), generator=g, device=d)).to(TYPES[case["dtype"]])
    s["slopes"] = torch.from_numpy(_slopes(h)).float().to(d) if case["bias"] else None
    if case["op"] == "tree":
        s["tree"], depth = _tree_inputs(_parents(case), d)
        base = np.repeat(np.array(kv_len) - np.array(new), new)
        s["positions"] = depth + torch.from_numpy(base.astype(np.int32)).to(d)
    else:
        firsts, prefixes = _layout(case)
        s["first"] = ints(sum(firsts, [])) if case["docs"] else None
        s["prefix"] = ints(prefixes) if case["prefix"] else None
    return s


# ---------------------------------------------------------------------------------- one pass
def _whole(s, name):
    """A pool's values in 32 bits."""
    x = s[name].float()
    if s[name + "d"] is None:
        return x
    return (x.view(x.shape[:3] + (-1, 32)) * s[name + "d"].float().unsqueeze(-1)).view(x.shape)


def _bits(words, count):
    """The first `count` bits of each row of 32-bit words, as truth values."""
    at = torch.arange(count, device=words.device)
    return (words[:, at // 32] >> (at % 32).int() & 1).bool()


def _plain_attn(s):
    c = s["case"]
    b, h, hk, dim, n, length = c["batch"], c["heads"], c["kv_heads"], c["dim"], s["max_new"], s["max_len"]
    t = torch.arange(s["total"], device=s["q"].device)
    seq = torch.searchsorted(s["q_start"][1:].contiguous(), t, right=True)
    at = t - s["q_start"][seq]
    base = s["kv_len"] - (s["q_start"][1:] - s["q_start"][:-1])
    key = torch.arange(length, device=t.device)
    # position of each new token and of each slot, and which slots it sees
    row = (base[seq] + at) if c["op"] == "shaped" else s["positions"]
    column = key.expand(b, length)
    if c["op"] == "tree":
        column = column.clone()
        column[seq, (base[seq] + at).long()] = s["positions"].long()
        own_bits = _bits(s["tree"], n)
        drafted = key - base[seq, None]  # place of the slot among the drafts
        old = drafted < 0
        if c["window"]:
            old &= key > row[:, None] - c["window"]
        seen = old | ((drafted >= 0) & (drafted < n) & own_bits.gather(1, drafted.clamp(0, n - 1).long()))
    else:
        last = row if s["prefix"] is None else torch.maximum(row, s["prefix"][seq] - 1)
        seen = key <= last[:, None]
        if c["window"]:
            seen &= key > row[:, None] - c["window"]
        if s["first"] is not None:
            seen &= key >= s["first"][:, None]
    seen &= key < s["kv_len"][seq, None]
    q = s["q"].new_zeros((b, n, h, dim), dtype=torch.float32)
    q[seq, at] = s["q"].float() * dim ** -0.5
    q = q.view(b, n, hk, h // hk, dim).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, dim)
    k, v = (_whole(s, w)[s["pages"]].transpose(1, 2).reshape(b, hk, -1, dim)[:, :, :length] for w in ("k", "v"))
    scores = (q @ k.transpose(-1, -2)).view(b, hk, h // hk, n, length)
    del k
    if c["cap"]:
        scores.div_(c["cap"]).tanh_().mul_(c["cap"])
    if s["slopes"] is not None:
        far = torch.zeros((b, n, length), device=t.device)
        far[seq, at] = (row[:, None] - column[seq]).abs().float()
        scores -= s["slopes"].view(1, hk, h // hk, 1, 1) * far[:, None, None]
    hidden = torch.ones((b, n, length), dtype=torch.bool, device=t.device)
    hidden[seq, at] = ~seen
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hk, -1, length) @ v).view(b, hk, h // hk, n, dim) / torch.where(total == 0, 1.0, total)
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, h, dim)[seq, at].to(s["q"].dtype)


def _plain_logits(s):
    c = s["case"]
    b, n, v = c["batch"], c["drafts"], c["vocab"]
    d = s["x"].device
    at = torch.arange(s["history"].shape[1], device=d)
    used = at < s["history_len"][:, None]
    ids = s["history"].long()
    said = torch.zeros((b, v), dtype=torch.int32, device=d).scatter_add_(1, ids, used.int())
    count = torch.zeros((b, v), dtype=torch.int32, device=d).scatter_add_(1, ids, (used & (at >= s["prompt_len"][:, None])).int())
    said, count = (x.repeat_interleave(n, 0) for x in (said, count))
    if n > 1:
        path = _bits(s["tree"], n).int()
        drafted = s["drafts"].long().view(b, 1, n).expand(b, n, n).reshape(b * n, n)
        said.scatter_add_(1, drafted, path)
        count.scatter_add_(1, drafted, path)
    x = s["x"].float()
    if s["bias"] is not None:
        add = torch.zeros((b, v), device=d).scatter_(1, s["bias_ids"].long().view(b, -1), s["bias"].view(b, -1))
        x = x + add.repeat_interleave(n, 0)
    rep, freq, pres = (s[w].repeat_interleave(n)[:, None] for w in ("repetition", "frequency", "presence"))
    x = torch.where(said > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - freq * count - pres * (count > 0)
    if s["allow"] is not None:
        x = torch.where(_bits(s["allow"], v), x, -math.inf)
    return x.to(TYPES[c["out"]])


def _plain_keep(s):
    c = s["case"]
    m, page = s["keep"].shape[1], c["page"]
    base = s["kv_len"] - (s["q_start"][1:] - s["q_start"][:-1])
    seq = torch.arange(c["batch"], device=base.device)[:, None].expand(-1, m)
    use = torch.arange(m, device=base.device) < s["keep_len"][:, None]
    src, dst = base[:, None] + s["keep"], base[:, None] + torch.arange(m, device=base.device)
    seq, src, dst = seq[use], src[use], dst[use]
    from_page, to_page = (s["pages"][seq, x // page].long() for x in (src, dst))
    for name in ("k", "v"):
        s[name][:, to_page, :, dst % page] = s[name][:, from_page, :, src % page]
    return s["k"], s["v"], base + s["keep_len"]


def run(s):
    c = s["case"]
    if not own:
        return {"shaped": _plain_attn, "tree": _plain_attn, "logits": _plain_logits, "keep": _plain_keep}[c["op"]](s)
    import gguf_block_quantized_quant_gb300 as qg
    if c["op"] == "shaped":
        return qg.qg_attn_shaped(s["q"], s["k"], s["v"], s["q_start"], s["kv_len"], s["pages"], kd=s["kd"], vd=s["vd"], cap=c["cap"],
                                 slopes=s["slopes"], first=s["first"], prefix=s["prefix"], max_new=s["max_new"], window=c["window"])
    if c["op"] == "tree":
        return qg.qg_attn_tree(s["q"], s["k"], s["v"], s["q_start"], s["kv_len"], s["pages"], s["tree"], positions=s["positions"],
                               kd=s["kd"], vd=s["vd"], cap=c["cap"], slopes=s["slopes"], max_new=s["max_new"], window=c["window"])
    if c["op"] == "logits":
        return qg.qg_logits_adjust(s["x"], out_dtype=TYPES[c["out"]], seq=s["seq"], history=s["history"], history_len=s["history_len"],
                                   prompt_len=s["prompt_len"], repetition=s["repetition"], frequency=s["frequency"],
                                   presence=s["presence"], bias_start=s["bias_start"], bias_ids=s["bias_ids"], bias=s["bias"],
                                   allow=s["allow"], drafts=s["drafts"], tree=s["tree"], q_start=s["q_start"])
    kv_len = qg.qg_cache_keep(s["k"], s["v"], s["q_start"], s["kv_len"], s["pages"], s["keep"], s["keep_len"])
    return s["k"], s["v"], kv_len


# ------------------------------------------------------------------------- what it cannot do without
def _spans(case):
    """Per sequence: (slots that some new token sees, pairs of a new token and a slot it sees)."""
    window = case["window"] or 1 << 60
    new, kv_len = _lengths(case)
    if case["op"] == "tree":
        for parent, length in zip(_parents(case), kv_len):
            base, depth = length - len(parent), []
            for p in parent:
                depth.append(depth[p] + 1 if p >= 0 else 0)
            yield (len(parent) + min(base, window - 1), sum(min(base, max(0, window - 1 - x)) + x + 1 for x in depth))
        return
    for n, length, first, prefix in zip(new, kv_len, *_layout(case)):
        p = np.arange(length - n, length)
        lo = np.maximum(np.array(first), p - window + 1).clip(0)
        hi = np.minimum(np.maximum(p, prefix - 1), length - 1)
        order = np.argsort(lo, kind="stable")
        reach = np.maximum.accumulate(hi[order])
        before = np.concatenate([[-1], reach[:-1]])
        yield (int(np.maximum(0, hi[order] - np.maximum(lo[order] - 1, before)).sum()), int(np.maximum(0, hi - lo + 1).sum()))


def work(case):
    if case["op"] == "logits":
        rows, v = case["batch"] * case["drafts"], case["vocab"]
        r = random.Random(case["mix"] + 3)
        span = [case["hist_lo"] if case["hist_hi"] <= case["hist_lo"] else _log_int(r, case["hist_lo"], case["hist_hi"]) for _ in range(case["batch"])]
        extra = 4 * sum(span) + 8 * case["bias"] * case["batch"] + (rows * 4 * -(-v // 32) if case["grammar"] else 0)
        return {"bytes": rows * v * (SIZE[case["dtype"]] + SIZE[case["out"]]) + extra, "flops": 2 * rows * v}
    new, kv_len = _lengths(case)
    if case["op"] == "keep":
        m = case["kept"]
        moved = sum((m - b % 2 if m > 1 else m) - 1 for b in range(case["batch"]))
        return {"bytes": 4 * moved * case["layers"] * case["kv_heads"] * case["dim"] * SIZE[case["dtype"]] + 4 * case["batch"] * (m + 4), "flops": 0}
    h, hk, dim = case["heads"], case["kv_heads"], case["dim"]
    row = hk * (dim * 34 // 32 if case["cache"] == "q8" else dim * 2)  # bytes of one slot's keys, or values
    spans = list(_spans(case))
    table = 4 * sum(-(-n // case["page"]) for n in kv_len) + 8 * case["batch"]
    if case["op"] == "tree":
        table += 4 * sum(new) * -(-max(new) // 32)
    return {"bytes": 2 * row * sum(x for x, _ in spans) + 2 * sum(new) * h * dim * SIZE[case["dtype"]] + table,
            "flops": 4 * dim * h * sum(x for _, x in spans)}


# ------------------------------------------------------------------------------ in 64 bits
def _exact_attn(case, s):
    new, kv_len = _lengths(case)
    group, window = case["heads"] // case["kv_heads"], case["window"] or 1 << 40
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    slopes, t0 = _slopes(case["heads"]), 0
    if case["op"] == "tree":
        parents = _parents(case)
    else:
        firsts, prefixes = _layout(case)
    for b, (n, length) in enumerate(zip(new, kv_len)):
        # which slots each new token sees, and how far they are, on the host
        base, slot = length - n, np.arange(length)
        if case["op"] == "tree":
            see, depth = np.zeros((n, length), dtype=bool), np.zeros(n, dtype=np.int64)
            for i, p in enumerate(parents[b]):
                if p >= 0:
                    see[i], depth[i] = see[p], depth[p] + 1
                see[i, base + i] = True
                see[i, :base] = slot[:base] > base + depth[i] - window
            place = np.concatenate([slot[:base], base + depth])
            apart = np.abs((base + depth)[:, None] - place[None])
        else:
            p = np.arange(base, length)[:, None]
            see = ((slot <= p) | (slot < prefixes[b])) & (p - slot < window) & (slot >= np.array(firsts[b])[:, None])
            apart = np.abs(p - slot)
        see, apart = torch.from_numpy(see).to(out.device), torch.from_numpy(apart).to(out.device)
        ids = s["pages"][b, :-(-length // case["page"])].long()
        for j in range(case["kv_heads"]):
            part = []
            for w in ("k", "v"):
                x = s[w][ids, j].double()
                if s[w + "d"] is not None:
                    x *= s[w + "d"][ids, j].double().repeat_interleave(32, -1)
                part.append(x.reshape(-1, case["dim"])[:length])
            for head in range(j * group, (j + 1) * group):
                for lo in range(0, n, 512):
                    hi = min(n, lo + 512)
                    z = torch.einsum("td,sd->ts", s["q"][t0 + lo:t0 + hi, head].double(), part[0]) / math.sqrt(case["dim"])
                    if case["cap"]:
                        z = case["cap"] * torch.tanh(z / case["cap"])
                    if case["bias"]:
                        z = z - float(np.float32(slopes[head])) * apart[lo:hi].double()
                    z = z.masked_fill(~see[lo:hi], -math.inf)
                    out[t0 + lo:t0 + hi, head] = torch.nan_to_num(torch.softmax(z, -1)) @ part[1]  # a row that sees nothing: zeros
        t0 += n
    return out


def _exact_logits(case, s):
    x = s["x"].double()
    history, spans, prompts = s["history"].cpu(), s["history_len"].tolist(), s["prompt_len"].tolist()
    drafts = s["drafts"].cpu() if case["drafts"] > 1 else None
    parents = _parents(case)
    for r in range(x.shape[0]):
        b, i = divmod(r, case["drafts"])
        said = history[b, :spans[b]].tolist()
        made = said[prompts[b]:]
        if case["drafts"] > 1:
            while i >= 0:
                made.append(int(drafts[b * case["drafts"] + i]))
                i = parents[b][i]
        said = np.unique(np.array(said + made, dtype=np.int64))
        ids, counts = np.unique(np.array(made, dtype=np.int64), return_counts=True)
        if case["bias"]:
            part = slice(b * len(s["bias_ids"]) // case["batch"], (b + 1) * len(s["bias_ids"]) // case["batch"])
            x[r, s["bias_ids"][part].long()] += s["bias"][part].double()
        said, ids, counts = (torch.from_numpy(a).to(x.device) for a in (said, ids, counts))
        rep, freq, pres = (s[w][b].double() for w in ("repetition", "frequency", "presence"))
        y = x[r, said]
        x[r, said] = torch.where(y > 0, y / rep, y * rep)
        x[r, ids] -= freq * counts + pres
    if s["allow"] is not None:
        words = s["allow"].cpu().numpy().view(np.uint8).reshape(x.shape[0], -1)
        allowed = np.unpackbits(words, axis=1, bitorder="little")[:, :case["vocab"]]
        x[torch.from_numpy(allowed == 0).to(x.device)] = -math.inf
    return x


def _exact_keep(case, s):
    keep, kept = s["keep"].tolist(), s["keep_len"].tolist()
    new, kv_len = _lengths(case)
    pages = s["pages"].tolist()
    where = lambda b, slot: (pages[b][slot // case["page"]], slot % case["page"])  # noqa: E731
    out = [s["k"].double(), s["v"].double()]
    for b in range(case["batch"]):
        base = kv_len[b] - new[b]
        for i in range(kept[b]):
            (p, a), (q, z) = where(b, base + keep[b][i]), where(b, base + i)
            for x in out:
                x[:, q, :, z] = x[:, p, :, a]
    return out[0], out[1], torch.tensor([n - m + t for n, m, t in zip(kv_len, new, kept)], dtype=torch.int32, device=s["k"].device)


def exact(case, seed):
    if work(case)["flops"] > 4e12:  # over 20 seconds in 64 bits
        return None
    s = prepare(case, seed)
    return {"logits": _exact_logits, "keep": _exact_keep}.get(case["op"], _exact_attn)(case, s)
