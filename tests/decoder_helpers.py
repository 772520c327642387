"""Shared plumbing for the decoder operators' GPU tests."""

from __future__ import annotations

import numpy as np
import torch

from oracle import decoder_oracle as O
import q4_weight_only_amd as q4

DEV = "cuda:0"


def dev(a, dtype=None):
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def bf16(x: np.ndarray) -> np.ndarray:
    """fp32 values rounded to bf16 (nearest even), as fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().float().numpy()


def device_cache(c: O.Cache) -> q4.KVCache:
    return q4.KVCache(dev(c.data), c.blocks, c.heads, c.D)


def random_table(rng, lengths, blocks, extra=1):
    """Block ids in no order, each used once; unused entries are -1."""
    need = [-(-max(int(n), 0) // 32) for n in lengths]
    assert sum(need) <= blocks
    order = rng.permutation(blocks)
    table = np.full((len(lengths), max(max(need), 1) + extra), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def assert_close(got, want, bound, what):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaNs differ at {np.argwhere(np.isnan(got) != nan)[:5]}"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    fine = ~nan & ~inf
    err, b = np.abs(got[fine] - want[fine]), np.broadcast_to(bound, want.shape)[fine]
    if err.size:
        i = int(np.argmax(err - b))
        assert np.all(err <= b), f"{what}: error {err[i]:.3g} over {b[i]:.3g}"
