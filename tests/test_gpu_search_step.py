"""Beam search, the cache's pages and selected blocks together, as
examples/decode.py runs them: against beams that each have blocks of their own,
against every block selected, as replayed graphs, and on streams other than the default one."""

import os
import sys

import numpy as np
import pytest
import torch

from oracle import decoder_oracle as O
from oracle import search_oracle as S
import q4_weight_only_amd as q4

from decoder_helpers import DEV, assert_close, bf16, dev, device_cache
from gpu_helpers import say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode  # noqa: E402

pytestmark = pytest.mark.gpu

PROMPTS = [[5, 9, 20, 3] * 9, [7], list(range(40))]


def _unshared(model, prompts, steps, beams, eos=-1):
    """The same search with all blocks of every beam its own: after each selection a beam gets copies of all
    of its parent's."""
    n, limit = len(prompts), max(len(p) for p in prompts) + steps
    width = -(-limit // 32)
    rows = n * beams
    stack = q4.KVStack.empty(len(model.layers), rows * width, model.kv_heads, model.head_dim)
    rope = q4.rope_table(4096, model.head_dim)
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.arange(rows * width, **i32).view(rows, width)
    lengths = torch.tensor([len(p) for p in prompts], **i32)
    cu = torch.cat((torch.zeros(1, **i32), lengths.cumsum(0).int()))
    logits = model.forward(torch.tensor(sum(prompts, []), **i32), stack, table[::beams].contiguous(), lengths, rope, cu,
                           max_rows=max(len(p) for p in prompts), max_length=int(lengths.max()), last=(cu[1:] - 1).long())
    scores, finished = np.zeros((n, 1), dtype=np.float32), np.zeros((n, 1))
    seq = [list(p) for p in prompts]
    at = [b * beams for b in range(n)]                       # where the row's blocks are
    for step in range(steps):
        p, t, s = S.beam_select(logits.cpu().numpy(), scores, beams, finished)
        done = finished.reshape(-1)
        seq = [seq[i] + ([] if done[i] else [int(x)]) for i, x in zip(p.reshape(-1), t.reshape(-1))]
        finished = np.array([bool(done[i]) or x == eos for i, x in zip(p.reshape(-1), t.reshape(-1))]).reshape(n, beams)
        scores = s.astype(np.float32)
        if step == steps - 1:
            break
        rows_from = table[[at[i] for i in p.reshape(-1)]].long()
        for c in stack:
            for plane in c.planes():
                plane[table.long()] = plane[rows_from].clone()
        at = list(range(rows))
        lengths = lengths[torch.from_numpy(p.reshape(-1)).to(DEV)] + 1
        logits = model.forward(torch.from_numpy(t.reshape(-1)).to(DEV).int(), stack, table, lengths, rope, max_rows=1, max_length=limit)
    return seq, scores


@pytest.mark.parametrize("beams,eos", [(1, -1), (4, -1), (4, 11), (7, -1)])
def test_shared_blocks_give_what_blocks_of_their_own_give(beams, eos):
    model = decode.Decoder(vocab=64, seed=3)
    say("beam_search", beams, eos)
    seq, lengths, scores = decode.beam_search(model, PROMPTS, 40, beams=beams, eos=eos)
    want, want_scores = _unshared(model, PROMPTS, 40, beams, eos)
    got = [s[:n].tolist() for s, n in zip(seq.reshape(-1, seq.shape[-1]).cpu(), lengths.reshape(-1).tolist())]
    assert got == want
    # a step's score is rounded to fp32 on both sides from values that differ by 1e-9
    assert np.allclose(scores.cpu().numpy(), want_scores, rtol=40 * 2.0 ** -23, atol=1e-7)


def test_every_block_selected_gives_the_same_tokens():
    model = decode.Decoder(vocab=512, seed=4)
    a = decode.beam_search(model, PROMPTS, 20, beams=3)
    b = decode.beam_search(model, PROMPTS, 20, beams=3, keep=4)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_few_blocks_and_the_summaries_that_choose_them():
    """With fewer blocks than there are: after every fork the summaries of all blocks in use are those of their keys."""
    model = decode.Decoder(vocab=512, seed=5)
    prompts = [list(range(200)), [3] * 333]
    seen = []

    def look(stack, table, lengths):
        seen.append((table.cpu().numpy(), lengths.cpu().numpy()))

    decode.beam_search(model, prompts, 40, beams=3, keep=4, each_step=look)
    for table, lengths in seen:
        for row, n in zip(table, lengths):
            ids = row[:-(-n // 32)]
            assert (ids >= 0).all() and len(set(ids)) == len(ids)
        # a partly filled block is in one table only
        ends = [row[(n - 1) // 32] for row, n in zip(table, lengths)]
        for e in ends:
            assert sum((row[:-(-n // 32)] == e).sum() for row, n in zip(table, lengths)) == 1


def test_summaries_follow_append_and_fork():
    rng = np.random.default_rng(6)
    heads, D, blocks = 2, 64, 24
    stack = q4.KVStack.empty(1, blocks, heads, D)
    cache, summary = stack[0], torch.full((1, blocks, heads, 2, D), 5, dtype=torch.int8, device=DEV)
    table, lengths = torch.full((2, 4), -1, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    parents = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    rope = q4.rope_table(200, D)
    for step in range(12):
        grow = int(rng.integers(1, 9))
        f = q4.kv_fork(table, lengths, parents, blocks, grow=grow)
        assert not f.short.any()
        q4.kv_copy_blocks(stack, f.src, f.dst, summaries=summary)
        table, lengths = f.block_table, f.lengths
        rows = table.shape[0] * grow
        q, k, v = (torch.randn((rows, h * D), device=DEV) * 2.0 ** float(rng.integers(-3, 4)) for h in (2 * heads, heads, heads))
        q4.kv_append(q, k, v, cache, table, lengths, rope, max_rows=grow)
        q4.kv_summarize(cache, summary[0], table, lengths, rows=rows, max_rows=grow)
        host = O.Cache(cache.data.cpu().numpy(), blocks, heads, D)
        want = summary[0].cpu().numpy().astype(np.int64)
        got = want.copy()
        t, n = table.cpu().numpy(), lengths.cpu().numpy()
        S.summarize(host, want, t, n, int(n.sum()), np.concatenate([[0], np.cumsum(n)]))   # all blocks in use
        assert np.array_equal(got, want)
        parents = torch.from_numpy(rng.integers(0, table.shape[0], 3)).int().to(DEV)


def test_graph_replays_give_the_eager_step():
    """A step of the search (selection, tokens, tables, copies, append, summaries, blocks, attention) between
    two sets of buffers, recorded and replayed with other logits in between eager calls of the same operators."""
    heads, group, D, blocks, beams, V, width = 2, 4, 64, 200, 4, 5000, 12
    g = torch.Generator(device=DEV).manual_seed(7)
    i32 = dict(dtype=torch.int32, device=DEV)
    rope = q4.rope_table(400, D)

    def start():
        torch.manual_seed(1)
        stack = q4.KVStack.empty(2, blocks, heads, D)
        stack.data.random_(0, 100)
        return dict(stack=stack, summary=torch.zeros((2, blocks, heads, 2, D), dtype=torch.int8, device=DEV),
                    table=torch.arange(2 * beams * width, **i32).view(2 * beams, width), lengths=torch.full((2 * beams,), 250, **i32),
                    scores=torch.zeros((2, beams), device=DEV), seq=torch.zeros((2 * beams, 300), **i32),
                    count=torch.full((2 * beams,), 250, **i32), done=torch.zeros(2 * beams, **i32))

    def step(s, logits, qkv):
        parents, tokens, scores = q4.beam_select(logits, s["scores"], beams, finished=s["done"].view(2, beams))
        seq, count, done = q4.beam_advance(s["seq"], s["count"], parents, tokens, finished=s["done"], eos=3)
        f = q4.kv_fork(s["table"], s["lengths"], parents, blocks)
        q4.kv_copy_blocks(s["stack"], f.src, f.dst, summaries=s["summary"])
        out = []
        for layer, cache in enumerate(s["stack"]):
            q = q4.kv_append(*qkv, cache, f.block_table, f.lengths, rope)
            q4.kv_summarize(cache, s["summary"][layer], f.block_table, f.lengths, rows=2 * beams)
            chosen = q4.kv_select(q, cache, s["summary"][layer], f.block_table, f.lengths, keep=5)
            out.append(q4.kv_attention_blocks(q, cache, chosen, f.block_table, f.lengths))
        for name, x in (("scores", scores), ("seq", seq), ("count", count), ("done", done), ("table", f.block_table), ("lengths", f.lengths)):
            s[name].copy_(x)
        return torch.stack(out)

    logits = torch.empty((2 * beams, V), device=DEV)
    qkv = [torch.empty((2 * beams, h * D), device=DEV) for h in (heads * group, heads, heads)]

    def fresh():
        logits.normal_(generator=g)
        for x in qkv:
            x.normal_(generator=g)

    fresh()
    eager, other = start(), start()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(start(), logits, qkv)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    say("capture")
    with torch.cuda.graph(graph):
        got = step(other, logits, qkv)
    for _ in range(8):
        fresh()
        want = step(eager, logits, qkv)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        for name, x in eager.items():
            y = other[name]
            assert torch.equal(x.data, y.data) if name == "stack" else torch.equal(x, y), name
    assert (other["lengths"] == 258).all()


def test_two_graphs_that_share_a_workspace_in_turn():
    """Graphs replayed one after the other on a stream may have one workspace."""
    z = [torch.randn((6, 9000), device=DEV) for _ in range(2)]
    s = torch.zeros((2, 3), device=DEV)
    want = [q4.beam_select(x, s, 4) for x in z]
    ws = torch.empty(q4.beam_select_workspace(2, 3, 9000), dtype=torch.uint8, device=DEV)
    graphs, got = [torch.cuda.CUDAGraph() for _ in z], []
    for graph, x in zip(graphs, z):
        with torch.cuda.graph(graph):
            got.append(q4.beam_select(x, s, 4, workspace=ws))
    for _ in range(3):
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_other_streams():
    """Calls on two streams at once, each with memory of its own."""
    rng = np.random.default_rng(8)
    c = O.Cache.empty(60, 2, 64)
    O.fill_random(c, rng)
    table, lengths = rng.permutation(60).reshape(2, 30), np.array([900, 955])
    q = bf16(rng.standard_normal((2, 4, 64)))
    host = np.zeros((60, 2, 2, 64), dtype=np.int64)
    S.summarize(c, host, table, lengths, 1855, np.array([0, 900, 1855]))
    chosen = S.select(c, host, q.astype(np.float64), table, lengths, 6, 1, 2)
    want, bound = S.attention_blocks(c, q.astype(np.float64), chosen, table, lengths)
    args = []
    for _ in range(2):
        cache = device_cache(c)
        args.append((dev(q.reshape(2, -1), torch.bfloat16), cache, q4.kv_summary(cache), dev(table, torch.int32), dev(lengths, torch.int32),
                     dev(np.array([0, 900, 1855]), torch.int32)))
    torch.cuda.synchronize()
    streams, out = [torch.cuda.Stream() for _ in range(2)], []
    for stream, (qd, cache, summary, t, n, cu) in zip(streams, args):
        with torch.cuda.stream(stream):
            for _ in range(20):
                q4.kv_summarize(cache, summary, t, n, cu, rows=1855, max_rows=955)
                picked = q4.kv_select(qd, cache, summary, t, n, keep=6)
                o = q4.kv_attention_blocks(qd, cache, picked, t, n, dtype=torch.float32)
            out.append((picked, o))
    torch.cuda.synchronize()
    for picked, o in out:
        assert np.array_equal(picked.cpu().numpy(), chosen)
        assert_close(o.cpu().numpy().reshape(want.shape), want, bound * (1 + 2.0 ** -22) + 2.0 ** -22 * np.abs(want), "attention")
