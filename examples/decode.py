"""A decoder on this library's operators: prompts, then single tokens.

    python examples/decode.py [--steps 16]

Everything between the token ids and the adjusted logits runs in the library:
the 4-bit linears (embedding, fused QKV, O, fused gate/up with SwiGLU, down,
LM head) and, between them, the fused norms, the append to the paged 8-bit
cache, the attention over it and the penalties on the logits.  Weights are
random; the sizes are arguments of Decoder.  Sequences of unequal length share
one batch, blocks are handed out as they are needed.
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import q4_weight_only_amd as q4  # noqa: E402


class Decoder:
    """Random weights of a pre-norm decoder with grouped heads and SwiGLU."""

    def __init__(self, layers=2, dim=512, heads=8, kv_heads=2, head_dim=64, ffn=1024, vocab=2048, window=0,
                 device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):
            return q4.pack(q4.quantize(torch.randn((n, k), generator=g, device=device) * k ** -0.5), n, k)

        def norm():
            return 1.0 + 0.1 * torch.randn(dim, generator=g, device=device)

        self.dim, self.heads, self.kv_heads, self.head_dim, self.window = dim, heads, kv_heads, head_dim, window
        self.vocab, self.device = vocab, device
        qd, kd = heads * head_dim, kv_heads * head_dim
        self.blocks = q4.quantize(torch.randn((vocab, dim), generator=g, device=device))   # the table, GGUF order
        self.lm_head = weight(vocab, dim)
        self.final_norm = norm()
        self.layers = [dict(qkv=[weight(qd, dim), weight(kd, dim), weight(kd, dim)], o=weight(dim, qd), gate=weight(ffn, dim),
                            up=weight(ffn, dim), down=weight(dim, ffn), attn_norm=norm(), ffn_norm=norm())
                       for _ in range(layers)]

    def caches(self, num_blocks):
        return [q4.KVCache.empty(num_blocks, self.kv_heads, self.head_dim, self.device) for _ in self.layers]

    def forward(self, ids, caches, table, lengths, rope, cu_rows=None, *, max_rows, max_length, last=None):
        """Logits [rows or len(last), vocab] of the rows `ids`; `last`: the rows whose logits are wanted."""
        shape = dict(max_rows=max_rows, max_length=max_length)
        r = q4.embed_gguf(self.blocks, self.vocab, self.dim, ids)
        y = None
        for layer, cache in zip(self.layers, caches):
            r, x = q4.add_rmsnorm(r, layer["attn_norm"], y)
            q, k, v = q4.linear_multi(x, layer["qkv"])
            q = q4.kv_append(q, k, v, cache, table, lengths, rope, cu_rows, max_rows=max_rows)
            a = q4.kv_attention(q, cache, table, lengths, cu_rows, window=self.window, **shape)
            r, x = q4.add_rmsnorm(r, layer["ffn_norm"], q4.linear(a, layer["o"]))
            y = q4.linear(q4.linear_swiglu(x, layer["gate"], layer["up"], dtype=torch.bfloat16), layer["down"])
        _, x = q4.add_rmsnorm(r, self.final_norm, y)
        return q4.linear(x if last is None else x[last], self.lm_head)


def generate(model, prompts, steps, *, repetition=1.2, presence=0.1, mask=None, positions=4096, graph=False):
    """Greedy continuations of the prompts (lists of ids): one prompt pass, then
    one token a step for the whole batch, as a replayed graph where asked.
    Returns (ids [batch][prompt + steps], the last step's adjusted logits)."""
    dev, n = model.device, len(prompts)
    need = [-(-(len(p) + steps) // q4.KV_BLOCK) for p in prompts]
    table = torch.full((n, max(need)), -1, dtype=torch.int32)
    for b, at in enumerate(torch.tensor([0] + need[:-1]).cumsum(0).tolist()):
        table[b, :need[b]] = torch.arange(at, at + need[b])
    table = table.to(dev)
    caches = model.caches(sum(need))
    rope = q4.rope_table(positions, model.head_dim, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    lengths = torch.tensor([len(p) for p in prompts], **i32)
    cu = torch.cat((torch.zeros(1, **i32), lengths.cumsum(0).int()))
    limit = max(len(p) for p in prompts) + steps
    # the histories, with room for the answers
    history = torch.zeros((n, limit), **i32)
    for b, p in enumerate(prompts):
        history[b, :len(p)] = torch.tensor(p, **i32)
    prompt_lengths, row = lengths.clone(), torch.arange(n, device=dev)
    rho, pres = (torch.full((n,), x, device=dev) for x in (repetition, presence))

    def pick(logits):
        live = torch.arange(limit, device=dev) < lengths[:, None]
        # one list of ids with bounds: unused places hold an id outside the vocabulary
        ids = torch.where(live, history, -1).reshape(-1)
        bounds = torch.arange(n + 1, **i32) * limit
        z = q4.logits_adjust(logits, history=ids, cu_history=bounds, prompt_lengths=prompt_lengths, repetition=rho,
                             presence=pres, mask=mask)
        return z, z.argmax(-1).int()

    logits = model.forward(torch.cat([history[b, :len(p)] for b, p in enumerate(prompts)]), caches, table, lengths, rope, cu,
                           max_rows=int(prompt_lengths.max()), max_length=int(lengths.max()), last=(cu[1:] - 1).long())
    z, ids = pick(logits)

    def step():
        history[row, lengths.long()] = ids
        lengths.add_(1)
        out, best = pick(model.forward(ids, caches, table, lengths, rope, max_rows=1, max_length=limit))
        z.copy_(out)
        ids.copy_(best)

    todo = steps - 1
    if graph and todo > 1:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()               # the library's and torch's one-time work, and one of the steps
        torch.cuda.current_stream().wait_stream(side)
        recorded = torch.cuda.CUDAGraph()
        with torch.cuda.graph(recorded):
            step()
        for _ in range(todo - 1):
            recorded.replay()
    else:
        for _ in range(todo):
            step()
    history[row, lengths.long()] = ids
    torch.cuda.synchronize()
    ends = (prompt_lengths + steps).tolist()
    return [h[:e].tolist() for h, e in zip(history.cpu(), ends)], z


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    model = Decoder()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g).tolist() for n in (70, 5, 33)]
    for graph in (False, True):
        generate(model, prompts, a.steps, graph=graph)
        t = time.perf_counter()
        ids, _ = generate(model, prompts, a.steps, graph=graph)
        print(f"{'graph' if graph else 'eager'}: {len(prompts)} sequences, {a.steps} tokens each in "
              f"{(time.perf_counter() - t) * 1e3:.1f} ms")
    for p, i in zip(prompts, ids):
        print(len(p), "->", i[len(p):])


if __name__ == "__main__":
    main()
