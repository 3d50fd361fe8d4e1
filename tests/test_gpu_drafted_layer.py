"""A step over drafted trees end to end: rotary positions by depth, tree attention, logits with the drafts' own penalties, accepted
drafts kept in the cache, and a token after them, against the layer in plain fp32 torch for every path of the trees; and a layer
with capped scores."""
import os
import sys

import pytest
import torch

from qg_testlib import qg_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    qg_module()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decoder_layer
    return decoder_layer


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("cap", [0.0, 3.0])
@pytest.mark.parametrize("cache", ["f16", "bf16", "q8"])
def test_drafts_are_what_their_paths_give(ex, cache, cap):
    qg = qg_module()
    layer, head = ex.Layer(hidden=512, heads=8, kv_heads=2, dim=64, inter=512, seed=3, cap=cap), ex.Head(512, 300)
    g = torch.Generator(device="cuda").manual_seed(11)
    prompts, parents = [70, 5, 40], [[-1, 0, 0, 1, 3, 3, 2, 4, 7], [-1, 0, 1, 2], [-1] + [0] * 5 + [3, 6, 7, 8, 9]]
    xs = [torch.randn((n, 512), generator=g, device="cuda") for n in prompts]
    store = ex.Cache(cache, 3, 128, 2, 64)
    q_start = ints([0, 70, 75, 115])
    layer(torch.cat(xs), store, q_start, ints(prompts), store.pages, 70)

    drafts = [torch.randn((len(p), 512), generator=g, device="cuda") for p in parents]
    history = torch.randint(0, 300, (3, 70), generator=g, device="cuda", dtype=torch.int32)
    said = dict(history=history, history_len=ints(prompts), prompt_len=ints([60, 5, 0]), repetition=torch.full((3,), 1.2, device="cuda"),
                frequency=torch.full((3,), 0.3, device="cuda"), presence=torch.full((3,), 0.1, device="cuda"))
    # Ids that the trees do accept: what is likeliest after a draft depends on its own id, so they are found from the root on
    tokens = [[7] * len(p) for p in parents]
    before = [t.clone() for t in (store.k, store.v)]
    for depth in range(6):
        store.k.copy_(before[0])
        store.v.copy_(before[1])
        res, logits, kv_len, keep = ex.verify(layer, head, store, prompts, torch.cat(drafts), parents, tokens, **said)
        best, at = logits.argmax(-1).tolist(), 0
        for t, p in zip(tokens, parents):
            for i in range(1, len(p)):
                t[i] = best[at + p[i]] if i % 2 or p[i] != 0 else (best[at] + 1) % 300
            at += len(p)
    assert qg.qg_device_error() == 0 and max(map(len, keep)) >= 3
    assert kv_len.tolist() == [n + len(k) for n, k in zip(prompts, keep)]

    def close(got, want, x):
        # int8 activations of up to 16 tokens cost 0.6 % per projection, an 8-bit cache as much; see the layer's own test
        assert ((got - want).norm() / (want - x).norm()).item() < 2e-2

    at = 0
    for b, p in enumerate(parents):
        for i in range(len(p)):
            path = [i]
            while p[path[0]] >= 0:
                path.insert(0, p[path[0]])
            rows = torch.cat([xs[b], drafts[b][path]])
            want = layer.plain(rows, [rows.shape[0]])[0]
            close(res[at + i], want[-1], rows[-1])
        at += len(p)

    # one token more on what was kept
    more = torch.randn((3, 512), generator=g, device="cuda")
    got, _ = layer(more, store, ints([0, 1, 2, 3]), kv_len + 1, store.pages, 1)
    for b in range(3):
        rows = torch.cat([xs[b], drafts[b][keep[b]], more[b:b + 1]])
        want = layer.plain(rows, [rows.shape[0]])[0]
        close(got[b], want[-1], rows[-1])


def test_capped_layer(ex):
    layer = ex.Layer(hidden=512, heads=8, kv_heads=2, dim=64, inter=512, seed=3, cap=2.0)
    outs, xs, _ = ex.run(layer, "f16", [70, 1, 33], 5, chunk=48)
    x = torch.cat(xs)
    want, _ = layer.plain(x, [t.shape[0] for t in xs])
    got = torch.cat(outs)
    assert ((got - want).norm() / (want - x).norm()).item() < 2e-2  # as the layer without a cap
    layer.cap = 0.0
    other, _ = layer.plain(x, [t.shape[0] for t in xs])
    assert ((other - want).norm() / (want - x).norm()).item() > 4e-2  # the cap matters here
