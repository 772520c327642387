"""q4_kv_attention in every launch it has -- 16 or 32 rows a workgroup, two or
four waves, whole or in parts -- with and without a window.  max_rows and
max_length are chosen for the launch, which kv_attention_plan has to confirm;
they change a result by its rounding alone."""

import itertools

import numpy as np
import pytest
import torch

import q4_weight_only_amd as q4

import test_gpu_kv_attention as base

pytestmark = pytest.mark.gpu

WHOLE, PARTS = "whole", "parts"
LAUNCHES = [(16, 4, WHOLE), (16, 4, PARTS), (32, 4, WHOLE), (32, 4, PARTS), (32, 2, WHOLE)]


class _Sizes:
    def __init__(self, heads, head_dim, batch, width):
        self.num_blocks, self.kv_heads, self.head_dim = 1 << 16, heads, head_dim
        self.shape = (batch, width)


def hints(launch, heads, group, D, lengths, rows, window):
    """max_rows and max_length that give the launch, the real length if there are
    such; for parts, ones that leave a row's tokens in three of them at least."""
    longest = max(lengths)
    s = _Sizes(heads, D, len(lengths), -(-longest // 32) + 1)
    reach = min(longest, window + 32) if window else longest
    for length, most in itertools.product((longest, longest * 2, 64, 4096, 1 << 14, 1 << 17, 1 << 19, 1 << 25),
                                          (max(rows), *(n * 2 ** k for k in range(6, 18) for n in (4, 5, 6, 7)))):
        plan = q4.kv_attention_plan(s, s, sum(rows), heads * group, max_rows=most, max_length=length, window=window)
        if plan[:2] != launch[:2] or (plan[2] > 1) != (launch[2] == PARTS):
            continue
        if launch[2] == PARTS:       # tokens of a part, at most
            blocks = -(-length // 32)
            if window:
                blocks = min(blocks, (window + plan[0] // group + 32) // 32 + 1)
            if -(-blocks // plan[2]) * 32 * 2 >= reach:
                continue
        return dict(max_rows=most, max_length=length)
    raise AssertionError(f"no sizes choose {launch} for {heads} x {group} heads of {D}, window {window}")


def _all(launch, D, lengths, rows, window, heads=2, group=3, **kw):
    return base._check(lengths, rows, heads=heads, group=group, D=D, window=window,
                       **hints(launch, heads, group, D, lengths, rows, window), **kw)


SIZES = {WHOLE: ((1100, 0, 33, 700), (45, 1, 33, 6), 300), PARTS: ((24700, 90, 0, 700), (24, 33, 1, 6), 20000)}


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("launch", LAUNCHES)
def test_ragged_batches(launch, D, cut):
    """Two tiles of rows with tokens in every part, an idle slot, sequences of
    fewer blocks than parts, and a group of heads that does not divide a tile."""
    lengths, rows, window = SIZES[launch[2]]
    _all(launch, D, lengths, rows, window if cut else 0, seed=40)
    _all(launch, D, lengths, rows, window if cut else 0, seed=41, dtype=torch.bfloat16, heads=1, group=4)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("launch", LAUNCHES)
def test_windows_smaller_than_a_block_and_larger_than_the_sequence(launch, D):
    lengths, rows, windows = (((24700, 40), (40, 40), (24690,)) if launch[2] == PARTS else
                              ((900, 40), (70, 40), (1, 20, 32, 65, 2000)))
    for window in windows:
        _all(launch, D, lengths, rows, window, seed=42)


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("launch", LAUNCHES)
def test_values_that_are_not_numbers_and_missing_blocks(launch, cut):
    """In the first and the last part, in blocks that rows see part of, and in a
    token that the window passes while the rows go on."""
    lengths, rows, window = SIZES[launch[2]]
    window = window if cut else 0
    n, r = lengths[0], rows[0]
    first = max(0, n - r - window + 1 if window else 0)     # that the first row sees
    at = (first + 3, n - 2, n // 2 + 9)

    def change(c, table, q):
        for j, t in enumerate(at):
            i = table[0, t // 32]
            codes = c.block_codes(i, 0, 1).copy()
            codes[t % 32, 5 + j] = 0x7F
            c.put(i, 0, 1, codes, c.exps[i, 0, 1])
        return table, q

    got = _all(launch, 64, lengths, rows, window, change=change, seed=43)
    last = got[:r, 0]
    assert np.isfinite(last[:, 4]).all() and np.isnan(last[-1, 6]) and np.isfinite(last[0, 6]) and np.isnan(last[0, 5])
    if cut:
        assert np.isfinite(last[-1, 5])

    def missing(c, table, q):
        table = table.copy()
        table[0, (first + 3) // 32] = -1
        return table, q

    got = _all(launch, 64, lengths, rows, window, change=missing, seed=43)
    assert np.isnan(got[0]).all() and np.isfinite(got[r:]).all()


@pytest.mark.parametrize("launch", LAUNCHES)
def test_more_rows_and_tokens_than_the_launch_is_shaped_for(launch):
    """Hints of shorter sequences: what they have no room for is not cut short."""
    lengths, rows, window = SIZES[launch[2]]
    kw = hints(launch, 2, 3, 64, lengths, rows, 0)
    base._check([lengths[0] + 7000, 700], [rows[0] + 40, 90], heads=2, group=3, seed=44, **kw)
