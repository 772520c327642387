"""kv_attention_blocks against the oracle in 64 bits, within the bound that the
oracle derives for the kernels' arithmetic plus the output's rounding (fp32
results: 4 roundings; bf16: 2^-8 of the value at the bound's edge)."""

import numpy as np
import pytest
import torch

from oracle import decoder_oracle as O
from oracle import search_oracle as S
import q4_weight_only_amd as q4

from decoder_helpers import DEV, assert_close, bf16, dev, device_cache, random_table
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _setup(lengths, rows, heads, group, D, keep, seed):
    rng = np.random.default_rng(seed)
    c = O.Cache.empty(sum(-(-max(n, 0) // 32) for n in lengths) + 2, heads, D)
    O.fill_random(c, rng)
    table = random_table(rng, lengths, c.blocks)
    for b, n in enumerate(lengths):      # slots after a sequence's last token hold anything
        if n > 0 and n % 32:
            for h in range(heads):
                for which in range(2):
                    i = table[b, (n - 1) // 32]
                    codes = c.block_codes(i, h, which).copy()
                    codes[n % 32:] = rng.choice([0x7F, 0xFF, 0x7E, 0xFE], codes[n % 32:].shape)
                    c.put(i, h, which, codes, c.exps[i, h, which])
    q = bf16(rng.standard_normal((sum(rows), heads * group, D)) * 1.5)
    chosen = np.full((sum(rows), heads, keep), -1)
    row = 0
    for n, length in zip(rows, lengths):
        for t in range(n):
            count = max(0, (length - n + t) // 32 + 1) if length - n + t >= 0 else 0
            for h in range(heads):
                some = np.sort(rng.permutation(count)[:keep])
                if count and count - 1 not in some and t % 2:     # the row's own block, mostly
                    some[-1:] = count - 1
                chosen[row, h, :len(some)] = some
            row += 1
    return rng, c, table, q, chosen


def _check(lengths, rows, *, heads=2, group=2, D=64, keep=6, scale=None, seed=0, dtype=torch.float32, cu=True, change=None, **kw):
    rng, c, table, q, chosen = _setup(lengths, rows, heads, group, D, keep, seed)
    if change:
        change(rng, c, table, q, chosen)
    bounds = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32) if cu is True else cu
    say("kv_attention_blocks", lengths, rows, heads, group, D, keep, dtype)
    got = q4.kv_attention_blocks(dev(q.reshape(q.shape[0], -1), torch.bfloat16), device_cache(c), dev(chosen, torch.int32), dev(table),
                                 dev(np.array(lengths, dtype=np.int32)), dev(bounds), dtype=dtype, scale=scale, **kw)
    got = got.double().cpu().numpy().reshape(q.shape)
    want, bound = S.attention_blocks(c, q.astype(np.float64), chosen, table, lengths, bounds, scale)
    round_off = 2.0 ** -22 if dtype == torch.float32 else 2.0 ** -8
    assert_close(got, want, bound * (1 + round_off) + round_off * np.abs(want), "kv_attention_blocks")
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lengths", [[1], [2], [31], [32], [33], [129], [1505], [1, 300, 32]])
def test_one_token(D, dtype, lengths):
    _check(lengths, [1] * len(lengths), D=D, group=4, dtype=dtype, seed=1)


@pytest.mark.parametrize("heads,group", [(1, 1), (8, 4), (3, 5), (1, 16), (1, 17), (1, 64), (20, 1), (2, 33)])
@pytest.mark.parametrize("rows", [1, 5])
def test_head_layouts(heads, group, rows):
    _check([300, rows], [rows, rows], heads=heads, group=group, seed=2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("keep", [1, 2, 3, 4, 5, 8, 9, 26, 63, 64, 65, 200, 300])
def test_lists_of_every_length(keep, D):
    """From one entry, through those that are split, to more than a wave has at once."""
    _check([9600], [1], D=D, heads=1, group=3, keep=keep, seed=3)
    _check([9600, 70], [1, 1], D=D, heads=1, group=1, keep=keep, seed=4, dtype=torch.bfloat16)


@pytest.mark.parametrize("lengths,rows", [([9], [9]), ([100], [33]), ([31, 200, 97], [31, 100, 1]), ([130, 130], [129, 70])])
@pytest.mark.parametrize("D", [64, 128])
def test_chunks(lengths, rows, D):
    _check(lengths, rows, D=D, seed=5)
    _check(lengths, rows, D=D, seed=5, max_rows=1)


def test_many_sequences():
    _check([50 + 31 * i for i in range(40)], [1] * 40, heads=8, group=4, D=128, seed=6, dtype=torch.bfloat16)
    _check([50 + 31 * i for i in range(40)], [1] * 40, heads=8, group=4, D=128, keep=40, seed=6)


@pytest.mark.parametrize("keep", [5, 100])
def test_entries_in_no_order_negative_and_past_the_row(keep):
    def change(rng, c, table, q, chosen):
        for row in chosen.reshape(-1, keep):
            rng.shuffle(row)
        chosen[rng.random(chosen.shape) < 0.2] = -7
        chosen[rng.random(chosen.shape) < 0.2] = 2 ** 30
        chosen[0, 0] = -1                      # nothing at all
        chosen[1, 1] = 10 ** 6

    got = _check([4000, 5000], [3, 2], keep=keep, change=change, seed=7)
    assert (got[0, :2] == 0).all() and (got[1, 2:] == 0).all()


@pytest.mark.parametrize("keep", [8, 60, 300])
@pytest.mark.parametrize("length", [40, 700, 1500])
def test_lists_longer_than_the_table(length, keep):
    """Blocks anywhere in a list that is longer than the table is wide, each many times."""
    def change(rng, c, table, q, chosen):
        chosen[...] = rng.integers(-1, length // 32 + 1, chosen.shape)
        chosen[0, 0, : keep // 2] = -1          # only behind the table's width

    _check([length], [1], heads=2, group=4, keep=keep, change=change)


def test_a_block_named_twice_counts_twice():
    def change(rng, c, table, q, chosen):
        chosen[:, :, 3:] = chosen[:, :, :3]

    _check([500], [2], change=change, seed=8)


def test_rows_without_a_position_and_idle_slots():
    got = _check([2, 0, 100], [4, 2, 3], seed=9)
    assert (got[:2] == 0).all() and (got[4:6] == 0).all()
    _check([64, 0, 100], [3, 3, 3], cu=None, seed=9)


def test_rows_behind_the_last_sequence_stay():
    rng, c, table, q, chosen = _setup([100], [5], 1, 2, 64, 4, 10)
    for keep in (4, 200):
        out = torch.full((5, 128), 7.0, device=DEV)
        lists = np.full((5, 1, keep), -1)
        lists[:, :, :4] = chosen
        q4.kv_attention_blocks(dev(q.reshape(5, -1), torch.bfloat16), device_cache(c), dev(lists, torch.int32), dev(table),
                               dev(np.array([100], dtype=np.int32)), dev(np.array([1, 3], dtype=np.int32)), out=out, dtype=torch.float32)
        assert (out[[0, 3, 4]] == 7).all() and (out[1:3] != 7).all()


@pytest.mark.parametrize("keep", [6, 120])
def test_what_is_not_a_number_reaches_who_sees_it(keep):
    def change(rng, c, table, q, chosen):
        for which, place, slot, d in ((0, 3, 5, 7), (1, 5, 31, 40), (1, 0, 0, 1)):
            codes = c.block_codes(table[0, place], 0, which).copy()
            codes[slot, d] = 0x7F
            c.put(table[0, place], 0, which, codes, 2)
        chosen[:, 0] = -1
        chosen[0, 0, :2], chosen[1, 0, :2], chosen[2, 0, :3], chosen[3, 0, :2] = [1, 3], [2, 5], [0, 1, 2], [6, 7]

    got = _check([3900], [4], keep=keep, change=change, seed=11)
    assert np.isnan(got[0, :2]).all() and np.isnan(got[1, :2]).any() and not np.isnan(got[3]).any()


@pytest.mark.parametrize("keep", [6, 120])
def test_unknown_blocks_are_not_numbers(keep):
    def change(rng, c, table, q, chosen):
        table[0, 2], table[0, 3] = -1, c.blocks
        chosen[:, :] = -1
        chosen[0, 0, :2], chosen[0, 1, :1], chosen[1, 0, :2] = [1, 2], [3], [0, 1]

    got = _check([3900], [2], keep=keep, change=change, seed=12)
    assert np.isnan(got[0]).all() and not np.isnan(got[1]).any()


@pytest.mark.parametrize("scale", [0.0, 1e-30, 3.0, -0.5, -40.0, 1e30])
def test_scales(scale):
    def change(rng, c, table, q, chosen):
        if abs(scale) > 100:
            q[:] = 0

    _check([400, 900], [1, 3], scale=scale, change=change, seed=13)
    _check([4000], [1], keep=100, scale=scale, change=change, seed=13)


def test_exponents_at_their_ends():
    def change(rng, c, table, q, chosen):
        c.exps[:, :, 0] = rng.choice([-3, 0, 2], c.exps[:, :, 0].shape)
        c.exps[:, :, 1] = rng.choice([-32, 32, 0], c.exps[:, :, 1].shape)

    _check([900, 5000], [2, 2], keep=10, change=change, seed=14)


def test_all_blocks_are_attention():
    """With every block in the list, and rows that choose alike, kv_attention's result up to the rounding of sums in
    another order; with its blocks in the waves' order, equal bit for bit."""
    rng, c, table, q, chosen = _setup([700, 300], [1, 1], 2, 4, 128, 22, 15)
    chosen[:] = np.arange(22)
    args = dev(q.reshape(2, -1), torch.bfloat16), device_cache(c)
    rest = dev(table), dev(np.array([700, 300], dtype=np.int32))
    a = q4.kv_attention(*args, *rest, dtype=torch.float32, max_length=700)
    b = q4.kv_attention_blocks(*args, dev(chosen, torch.int32), *rest, dtype=torch.float32)
    assert torch.equal(a, b)


def test_outputs_and_workspace_of_the_caller():
    rng, c, table, q, chosen = _setup([9000], [1], 2, 4, 64, 200, 16)
    qd, cache, list_, tab, n = dev(q.reshape(1, -1), torch.bfloat16), device_cache(c), dev(chosen, torch.int32), dev(table), dev(np.array([9000], dtype=np.int32))
    need = q4.kv_attention_blocks_workspace(cache, tab, 1, 8, 200)
    assert need > 0
    want = q4.kv_attention_blocks(qd, cache, list_, tab, n)
    ws, out = torch.full((need,), 255, dtype=torch.uint8, device=DEV), torch.empty_like(want)
    for _ in range(3):
        got = q4.kv_attention_blocks(qd, cache, list_, tab, n, out=out, workspace=ws)
        assert torch.equal(got, want) and got.data_ptr() == out.data_ptr()


def test_refusals():
    c = q4.KVCache.empty(5, 2, 64)
    t, n = torch.zeros((1, 4), dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    q, l = torch.zeros((1, 256), dtype=torch.bfloat16, device=DEV), torch.zeros((1, 2, 3), dtype=torch.int32, device=DEV)
    for bad in (lambda: q4.kv_attention_blocks(q.float(), c, l, t, n), lambda: q4.kv_attention_blocks(q, c, l.long(), t, n),
                lambda: q4.kv_attention_blocks(q, c, l[:, :1].contiguous(), t, n), lambda: q4.kv_attention_blocks(q, c, l[0], t, n),
                lambda: q4.kv_attention_blocks(q, c, l[:, :, :0], t, n), lambda: q4.kv_attention_blocks(q, c, l.cpu(), t, n),
                lambda: q4.kv_attention_blocks(q[:, :192].contiguous(), c, l, t, n),
                lambda: q4.kv_attention_blocks(q, c, l, t, n, scale=float("nan")),
                lambda: q4.kv_attention_blocks(q, c, l, t, n, dtype=torch.float16),
                lambda: q4.kv_attention_blocks(q, c, l, t, n, out=torch.empty((1, 128), dtype=torch.bfloat16, device=DEV))):
        with pytest.raises(ValueError):
            bad()


def test_outputs_that_overlap_are_refused():
    c = q4.KVCache.empty(5, 2, 64)
    t, n = torch.zeros((1, 4), dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    q, l = torch.zeros((1, 256), dtype=torch.bfloat16, device=DEV), torch.zeros((1, 2, 3), dtype=torch.int32, device=DEV)
    for bad in (lambda: q4.kv_attention_blocks(q, c, l, t, n, out=q),
                lambda: q4.kv_select(q, c, q4.kv_summary(c), t, n, keep=3, out=q.view(torch.int32)[:, :6].view(1, 2, 3))):
        with pytest.raises(ValueError, match="overlap"):
            bad()


def test_the_example_has_no_window_over_selected_blocks():
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decode
    with pytest.raises(ValueError, match="window"):
        decode.beam_search(decode.Decoder(vocab=64, window=40), [[1, 2, 3]], 4, beams=2, keep=4)
