"""Sizes of attention's workspace, and the launches that sizes choose: host code."""

import ctypes
import itertools
import os
import subprocess
import sys

import pytest

import q4_weight_only_amd as q4
from q4_weight_only_amd import _decoder as D


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(q4.library_path()):
        subprocess.run([sys.executable, "-m", "q4_weight_only_amd.build"], check=True)
    return D.decoder_lib()


def _structs(heads, head_dim, batch, rows, max_rows, max_length):
    return (D._Cache(0x10000, 1 << 20, heads, head_dim),
            D._Batch(0x10000, 0x10000, 0x10000, 1 << 20, batch, rows, max_rows, max_length))


def _workspace(L, heads, group, head_dim, batch, max_rows, max_length):
    c, b = _structs(heads, head_dim, batch, max(max_rows, batch), max_rows, max_length)
    return L.q4_kv_attention_workspace(ctypes.byref(c), ctypes.byref(b), heads * group)


@pytest.mark.parametrize("head_dim", [64, 128])
def test_workspace_is_bounded(L, head_dim):
    """Whatever the sizes: 2^16 rows of head_dim sums and two more, in fp32."""
    lengths = (1, 700, 704, 705, 2048, 8192, 8193, 131072, 1 << 20, 1 << 25)
    rows = (1, 2, 5, 16, 17, 33, 400, 512, 1024, 2048, 3900, 4096, 1 << 15, 1 << 20)
    for heads, group in ((1, 1), (1, 64), (8, 4), (20, 1), (7, 3), (256, 64)):
        for batch, most, length in itertools.product((1, 2, 31, 64, 500, 65535), rows, lengths):
            n = _workspace(L, heads, group, head_dim, batch, most, length)
            assert 0 <= n <= (1 << 18) * (head_dim + 2), (heads, group, batch, most, length, n)
            assert n % 16 == 0


def test_long_contexts_are_split_while_few_rows_share_them(L):
    for batch, most, splits in ((1, 1, 32), (2, 1, 16), (64, 1, 16), (1, 512, 4)):
        rows = batch * most * 32
        assert _workspace(L, 8, 4, 128, batch, most, 131072) == rows * splits * 130 * 4
    # 2048 rows of 32 heads fill the chip many times over
    assert _workspace(L, 8, 4, 128, 1, 2048, 131072) == 0
    assert _workspace(L, 8, 4, 128, 1, 2048, 1 << 20) == 0


class _Sizes:
    """What kv_attention_plan reads of a cache and a block table."""

    def __init__(self, heads, head_dim, batch, width=1 << 20):
        self.num_blocks, self.kv_heads, self.head_dim = 1 << 20, heads, head_dim
        self.shape = (batch, width)


def _plan(heads, group, head_dim, batch, rows, length, window=0):
    s = _Sizes(heads, head_dim, batch)
    return q4.kv_attention_plan(s, s, batch * rows, heads * group, max_rows=rows, max_length=length, window=window)


def test_plans_of_ordinary_sizes(L):
    assert _plan(8, 4, 128, 1, 1, 1505) == (16, 4, 12)
    assert _plan(8, 4, 128, 32, 1, 8191) == (16, 4, 1)
    assert _plan(8, 4, 128, 2, 1, 131072) == (16, 4, 16)
    assert _plan(8, 4, 128, 1, 2048, 2048) == (32, 2, 1)
    assert _plan(20, 1, 64, 1, 1505, 6020, 750) == (32, 2, 1)
    assert _plan(20, 1, 64, 1, 700, 3600, 750) == (16, 4, 1)
    assert _plan(20, 1, 64, 1, 900, 3600, 750) == (32, 4, 1)
    assert _plan(8, 4, 128, 1, 512, 16384) == (32, 4, 2)


def test_plan_refuses_what_a_call_refuses(L):
    c, b = _structs(2, 64, 2, 2, 1, 64)
    out = (ctypes.c_int32 * 3)()
    at = [ctypes.addressof(out) + 4 * i for i in range(3)]

    def call(c=c, b=b, heads=4, window=0, at=at):
        return L.q4_kv_attention_plan(ctypes.byref(c) if c else None, ctypes.byref(b) if b else None, heads, window, *at)

    assert call() == 0 and out[0] == 16 and out[1] == 4 and out[2] == 1
    assert call(c=None) == 1 and call(b=None) == 1 and call(at=[None, at[1], at[2]]) == 1 and call(at=[at[0], at[1], None]) == 1
    assert call(heads=5) == 6 and call(heads=0) == 6 and call(window=-1) == 6 and call(window=2**30 + 1) == 6
    assert call(c=_structs(2, 80, 2, 2, 1, 64)[0]) == 6 and call(b=_structs(2, 64, 2, 2, 0, 64)[1]) == 6


def test_workspace_holds_the_parts_of_every_window(L):
    """What a launch writes of partial results fits the workspace, which is the
    same for every window."""
    import random

    rng = random.Random(1)
    split = 0
    for _ in range(20000):
        heads, group = rng.choice(((8, 4), (1, 1), (20, 1), (7, 3), (2, 8), (1, 64), (64, 1)))
        head_dim, batch = rng.choice((64, 128)), int(2 ** rng.uniform(0, 10))
        most, length = int(2 ** rng.uniform(0, 15)), int(2 ** rng.uniform(0, 25))
        window = rng.choice((0, 1, 750, int(2 ** rng.uniform(0, 25))))
        c, b = _structs(heads, head_dim, batch, most, most, length)
        out = (ctypes.c_int32 * 3)()
        at = [ctypes.addressof(out) + 4 * i for i in range(3)]
        assert L.q4_kv_attention_plan(ctypes.byref(c), ctypes.byref(b), heads * group, window, *at) == 0
        tile, waves, parts = out
        assert (tile, waves) in ((16, 4), (32, 4), (32, 2)) and parts >= 1
        if parts == 1:
            continue
        split += 1
        rows = most * group
        partial = -(-rows // tile) * min(rows, tile) * heads * batch * parts
        need = ((partial * 2 + 3) // 4 * 4 + partial * head_dim) * 4
        assert need <= L.q4_kv_attention_workspace(ctypes.byref(c), ctypes.byref(b), heads * group), (heads, group, batch, most, length, window)
    assert split > 1000
