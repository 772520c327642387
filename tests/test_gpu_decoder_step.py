"""The decoder operators together, as examples/decode.py runs them: a prompt at
once against the same tokens one by one, replayed graphs against eager calls,
streams other than the default one, and one layer against 64-bit arithmetic."""

import os
import sys

import numpy as np
import pytest
import torch

from oracle import decoder_oracle as O
import q4_weight_only_amd as q4

from decoder_helpers import DEV, dev
from gpu_helpers import say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode  # noqa: E402

pytestmark = pytest.mark.gpu

PROMPTS = [[5, 9, 200, 3] * 9, [7], list(range(40))]


def test_graph_replays_give_the_eager_tokens():
    model = decode.Decoder(vocab=512, seed=1)
    say("generate eager")
    a, za = decode.generate(model, PROMPTS, 40)
    say("generate graph")
    b, zb = decode.generate(model, PROMPTS, 40, graph=True)
    assert a == b and torch.equal(za, zb)
    assert [len(x) for x in a] == [len(p) + 40 for p in PROMPTS]


def test_a_mask_holds_for_every_token():
    model = decode.Decoder(vocab=512, seed=2)
    mask = torch.zeros((3, 16), dtype=torch.int32, device=DEV)
    mask[:, 3] = 0b1010
    ids, z = decode.generate(model, PROMPTS, 5, mask=mask)
    for p, got in zip(PROMPTS, ids):
        assert set(got[len(p):]) <= {97, 99}
    assert torch.isfinite(z).sum(1).tolist() == [2, 2, 2]


def _run(model, ids, chunks):
    """Logits of every row of one sequence, appended in chunks."""
    caches = model.caches(4)
    table = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device=DEV)
    rope = q4.rope_table(128, model.head_dim, device=DEV)
    out, at = [], 0
    for n in chunks:
        lengths = torch.tensor([at + n], dtype=torch.int32, device=DEV)
        out.append(model.forward(torch.tensor(ids[at:at + n], dtype=torch.int32, device=DEV), caches, table, lengths, rope,
                                 max_rows=n, max_length=at + n))
        at += n
    return torch.cat(out), caches


def test_a_prompt_equals_its_tokens_one_by_one():
    """The same rows reach the cache, up to the codes that a growing block
    rounds twice and to roundings of the linears' other kernels: the logits
    agree to a few parts in a hundred of their size (8-bit codes: 2^-4 each)."""
    model = decode.Decoder(vocab=512, seed=3)
    ids = np.random.default_rng(3).integers(0, 512, 75).tolist()
    whole, _ = _run(model, ids, [75])
    for chunks in ([1] * 75, [30, 1, 1, 33, 10]):
        got, _ = _run(model, ids, chunks)
        err = (got - whole).norm(dim=1) / whole.norm(dim=1)
        assert float(err.max()) < 0.15 and float(err.mean()) < 0.05, (float(err.max()), float(err.mean()))


def test_one_layer_against_64_bits():
    """A layer's whole step from dequantized weights in 64 bits, with the
    oracle's append and attention: every rounding on the way is to bf16
    (2^-9), and no sum is longer than 1024, so 2 % of the result's norm is
    several times what they can add up to."""
    m = decode.Decoder(layers=1, vocab=256, seed=4)
    ids = np.random.default_rng(4).integers(0, 256, 50)
    got, _ = _run(m, ids.tolist(), [50])
    W = lambda p: q4.dequant(p).double().cpu().numpy()  # noqa: E731
    L, n = m.layers[0], len(ids)
    r = q4.embed_gguf(m.blocks, 256, m.dim, dev(ids.astype(np.int32))).double().cpu().numpy()
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    _, x = O.add_rmsnorm(r, f(L["attn_norm"]))
    q, k, v = (x @ W(p).T for p in L["qkv"])
    cache = O.Cache.empty(4, m.kv_heads, m.head_dim)
    table, rope = np.array([[3, 0, 2, 1]], dtype=np.int32), q4.rope_table(128, m.head_dim, device="cpu").numpy()
    split = lambda t, h: t.reshape(n, h, m.head_dim).astype(np.float32)  # noqa: E731
    q = O.append(cache, split(q, m.heads), split(k, m.kv_heads), split(v, m.kv_heads), table, [n], rope)
    a, _ = O.attention(cache, q.astype(np.float64), table, [n])
    r, x = O.add_rmsnorm(r, f(L["ffn_norm"]), a.reshape(n, -1) @ W(L["o"]).T)
    g = x @ W(L["gate"]).T
    r, x = O.add_rmsnorm(r, f(m.final_norm), (g / (1 + np.exp(-g)) * (x @ W(L["up"]).T)) @ W(L["down"]).T)
    want = x @ W(m.lm_head).T
    err = np.linalg.norm(f(got) - want) / np.linalg.norm(want)
    assert err < 0.02, err


def test_another_stream():
    """All operators on a stream of their own, behind work that delays it."""
    model = decode.Decoder(vocab=512, seed=5)
    ids = list(range(60))
    want, wc = _run(model, ids, [40, 20])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.randn((4096, 4096), device=DEV)
        for _ in range(5):
            big = (big @ big) * 1e-3
        got, gc = _run(model, ids, [40, 20])
        z = q4.logits_adjust(got)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(z, want)
    assert all(torch.equal(a.data, b.data) for a, b in zip(wc, gc))


def test_each_operator_in_a_graph_on_new_data():
    """Captured once, replayed after the inputs, lengths and tables change."""
    H, G, D, B, V = 2, 4, 128, 3, 1000
    cache = q4.KVCache.empty(B * 40, H, D, DEV)
    table = torch.randperm(B * 40, device=DEV).int().view(B, 40)
    lengths = torch.tensor([1200, 17, 600], dtype=torch.int32, device=DEV)
    rope = q4.rope_table(1280, D, device=DEV)
    x = dict(q=torch.empty((B, H * G * D), device=DEV), k=torch.empty((B, H * D), device=DEV), v=torch.empty((B, H * D), device=DEV),
             r=torch.empty((B, 512), device=DEV), y=torch.empty((B, 512), device=DEV), z=torch.empty((B, V), device=DEV))
    w = torch.rand(512, device=DEV)
    hist, cu = torch.zeros(60, dtype=torch.int32, device=DEV), torch.tensor([0, 20, 40, 60], dtype=torch.int32, device=DEV)

    def work():
        q = q4.kv_append(x["q"], x["k"], x["v"], cache, table, lengths, rope, max_rows=1)
        a = q4.kv_attention(q, cache, table, lengths, max_rows=1, max_length=1280)
        r, n = q4.add_rmsnorm(x["r"], w, x["y"])
        z = q4.logits_adjust(x["z"], history=hist, cu_history=cu, repetition=x["z"][:, 0].abs().contiguous() + 1)
        return q, a, r, n, z

    def fill(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        for t in x.values():
            t.normal_(generator=g)
        hist.random_(0, V, generator=g)
        table.copy_(torch.randperm(B * 40, generator=g, device=DEV).int().view(B, 40))
        codes, exps = cache.planes()
        codes.random_(0, 0x7F, generator=g)
        exps.random_(-8, 2, generator=g)
        lengths.random_(1, 1280, generator=g)

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for seed in range(1, 6):
        fill(seed)
        for o in outs:
            o.fill_(float("nan"))
        say("decoder graph", seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs] + [cache.data.clone()]
        fill(seed)
        want = list(work()) + [cache.data]
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (seed, i)
