"""q4_kv_attention against the oracle in 64 bits, within the bound that the
oracle derives for the kernels' arithmetic plus the output's rounding (fp32
results: 4 roundings; bf16: 2^-8 of the value at the bound's edge)."""

import sys

import numpy as np
import pytest
import torch

from oracle import decoder_oracle as O
import q4_weight_only_amd as q4

from decoder_helpers import DEV, assert_close, bf16, dev, device_cache, random_table
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=["chosen", "32 rows", "32 rows, split", "32 rows, two waves"])
def kernel(request, monkeypatch):
    """Every test runs with the kernel that its sizes choose, and with those for
    more rows: max_rows and max_length, which shape a launch, change no result."""
    monkeypatch.setattr(sys.modules[__name__], "KERNEL", request.param)


KERNEL = "chosen"


def _hint(sets, group):
    """max_rows and max_length that bring a launch of `sets` sequences x kv heads
    to the kernel (without a window)."""
    return {"32 rows": (1 << 19, 1 << 25), "32 rows, split": (1100 // (sets * group) + 17, 1 << 20),
            "32 rows, two waves": (1 << 19, 64)}[KERNEL]


def _setup(lengths, rows, heads, group, D, seed, garbage=True, blocks=None):
    rng = np.random.default_rng(seed)
    need = sum(-(-max(n, 0) // 32) for n in lengths)
    c = O.Cache.empty(blocks or need + 2, heads, D)
    O.fill_random(c, rng)
    table = random_table(rng, lengths, c.blocks)
    if garbage:      # slots after a sequence's last token hold anything
        for b, n in enumerate(lengths):
            if n > 0 and n % 32:
                i = table[b, (n - 1) // 32]
                for h in range(heads):
                    for which in range(2):
                        codes = c.block_codes(i, h, which).copy()
                        codes[n % 32:] = rng.choice([0x7F, 0xFF, 0x7E, 0xFE], codes[n % 32:].shape)
                        c.put(i, h, which, codes, c.exps[i, h, which])
    q = bf16(rng.standard_normal((sum(rows), heads * group, D)) * 1.5)
    return c, table, q


def _call(c, table, q, lengths, rows, *, cu=True, dtype=torch.float32, **kw):
    bounds = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32) if cu is True else cu
    if not {"max_rows", "max_length"} & kw.keys() and KERNEL != "chosen":
        kw["max_rows"], kw["max_length"] = _hint(c.heads * len(lengths), q.shape[1] // c.heads)
    out = q4.kv_attention(dev(q.reshape(q.shape[0], -1), torch.bfloat16), device_cache(c), dev(table),
                          dev(np.array(lengths, dtype=np.int32)), dev(bounds), dtype=dtype, **kw)
    return out.double().cpu().numpy().reshape(q.shape)


def _check(lengths, rows, *, heads=2, group=2, D=64, window=0, scale=None, seed=0, dtype=torch.float32, cu=True,
           change=None, **kw):
    c, table, q = _setup(lengths, rows, heads, group, D, seed)
    if change:
        table, q = change(c, table, q) or (table, q)
    say("attention", lengths, rows, heads, group, D, window, dtype, kw)
    got = _call(c, table, q, lengths, rows, dtype=dtype, window=window, scale=scale, cu=cu, **kw)
    bounds = np.concatenate([[0], np.cumsum(rows)]) if cu is True else cu
    want, bound = O.attention(c, q.astype(np.float64), table, lengths, bounds, window, scale)
    round_off = 2.0 ** -22 if dtype == torch.float32 else 2.0 ** -8
    assert_close(got, want, bound * (1 + round_off) + round_off * np.abs(want), "attention")
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lengths", [[1], [2], [31], [32], [33], [63], [129], [1505], [1, 300, 32]])
def test_one_token(D, dtype, lengths):
    _check(lengths, [1] * len(lengths), D=D, heads=2, group=4, dtype=dtype, seed=1)


@pytest.mark.parametrize("heads,group", [(1, 1), (8, 4), (3, 5), (1, 16), (1, 17), (1, 64), (20, 1), (2, 7)])
@pytest.mark.parametrize("rows", [1, 2, 5])
def test_head_layouts(heads, group, rows):
    _check([70, rows], [rows, rows], heads=heads, group=group, seed=2)


@pytest.mark.parametrize("lengths,rows", [([9], [9]), ([64], [64]), ([65], [65]), ([100], [33]), ([128], [128]),
                                          ([31, 200, 97], [31, 100, 1]), ([257], [250]), ([130, 130], [129, 70])])
@pytest.mark.parametrize("D", [64, 128])
def test_prompts_and_chunks(lengths, rows, D):
    _check(lengths, rows, D=D, heads=2, group=2, seed=3)


@pytest.mark.parametrize("group", [1, 3, 4])
def test_prompt_of_bf16_rows(group):
    _check([190], [190], D=128, heads=1, group=group, seed=4, dtype=torch.bfloat16)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 64, 100, 1000])
@pytest.mark.parametrize("rows", [1, 3, 150])
def test_windows(window, rows):
    _check([260], [rows], window=window, seed=5)


def test_windows_that_leave_each_kernel():
    """A window that cuts, and yet chooses the launch as the hints do."""
    _check([900, 700], [200, 90], window=600, heads=1, group=3, D=128, seed=26)
    _check([3400], [70], window=3000, heads=2, group=2, D=64, seed=26)


def test_windows_of_a_prompt_with_many_heads():
    _check([300], [300], window=70, heads=3, group=1, D=64, seed=6)
    _check([300], [200], window=70, heads=1, group=5, D=128, seed=6)


def test_sizes_that_choose_the_kernels_for_many_rows():
    """By their own number: 2565, 576, 800 and 289 groups of 32 rows, and 32 whose
    blocks are many."""
    if KERNEL != "chosen":
        return
    _check([150] * 9, [150] * 9, heads=19, group=3, seed=21)
    _check([65] * 8, [65] * 8, heads=24, group=1, D=128, seed=21)
    _check([40, 33], [33, 33], heads=8, group=48, D=128, seed=21)
    _check([90], [90], heads=17, group=6, D=128, seed=21)
    _check([21000], [64], heads=1, group=16, D=128, max_length=21000, seed=21)


def test_scale():
    _check([77], [2], scale=0.5, seed=7)
    _check([77], [2], scale=0.0, seed=7)
    _check([77], [2], scale=-0.3, seed=7)


def test_large_scores():
    """One token takes nearly all the weight, and scores in the hundreds."""
    def change(c, table, q):
        return table, bf16(q * 40)

    _check([200], [3], seed=8, change=change)
    _check([200], [100], seed=8, change=change)


def test_scores_that_rise_from_block_to_block():
    """Each block's keys outweigh the last's by more than the running maximum's slack."""
    def change(c, table, q):
        for j in range(6):
            c.exps[table[0, j], :, 0] = j - 2
        return table, q

    _check([180], [1], seed=9, change=change)
    _check([180], [90], seed=9, change=change)


def test_value_scales_that_differ_widely():
    def change(c, table, q):
        for j in range(5):
            c.exps[table[0, j], :, 1] = (-32, 20, 0, -20, 32)[j]
        return table, q

    _check([150], [1], seed=10, change=change)
    _check([150], [150], seed=10, change=change)


def test_key_scales_at_their_limits():
    def change(c, table, q):
        for j in range(3):
            c.exps[table[0, j], :, 0] = (-32, -3, -32)[j]
        return table, q

    _check([96], [2], seed=11, change=change)
    _check([96], [96], seed=11, change=change)


def test_rows_without_tokens_are_zero():
    got = _check([0, 40, 3, 0], [1, 1, 5, 0], seed=12)
    assert not got[0].any() and not got[2:4].any()
    _check([0], [1], seed=12, cu=None)
    _check([10], [70], seed=12)
    _check([-5, 10], [1, 1], seed=12)


def test_nan_values_reach_the_rows_that_see_them_only():
    """Not a number at one token of V: rows before it (and rows whose window
    has passed it) are untouched, in its dimension the others are not a number."""
    def plant(at, dims, which):
        def change(c, table, q):
            for t in at:
                i = table[0, t // 32]
                for h in range(c.heads):
                    codes = c.block_codes(i, h, which).copy()
                    codes[t % 32, dims] = 0x7F if t % 2 else 0xFF
                    c.put(i, h, which, codes, c.exps[i, h, which])
        return change

    for rows in (1, 2, 40, 100):
        got = _check([100], [rows], seed=13, change=plant([70], [3, 40], 1))
        if rows == 100:
            assert np.isfinite(got[:70]).all() and np.isnan(got[70:, :, 3]).all() and np.isfinite(got[70:, :, 4]).all()
        _check([100], [rows], seed=13, change=plant([98, 64], [0, 63], 1))
        _check([100], [rows], seed=13, window=20, change=plant([70, 85], [17], 1))
        _check([100], [rows], seed=13, change=plant([99, 71], [5], 0))
        _check([100], [rows], seed=13, window=9, change=plant([71], [5], 0))
    _check([140], [140], D=128, heads=1, group=4, seed=13, change=plant([3, 100, 139], [0, 100], 1))


def test_queries_that_are_not_finite():
    def change(c, table, q):
        q = q.copy()
        q[0, 0, 0], q[1, 1, 2] = np.nan, np.nan
        return table, q

    _check([50], [3], seed=14, change=change)
    _check([90], [80], seed=14, change=change)


def test_blocks_outside_the_cache_are_nan():
    def change(c, table, q):
        table = table.copy()
        table[0, 1], table[1, 0] = c.blocks, -1
        return table, q

    for rows in (1, 50):
        _check([64 + rows, 20 + rows], [rows, rows], seed=15, change=change)
    # rows before the tokens of such a block are not touched by it
    def far(c, table, q):
        table = table.copy()
        table[0, 1] = -3
        return table, q

    got = _check([70, 20], [70, 1], seed=15, change=far)
    assert np.isfinite(got[:32]).all() and np.isnan(got[32:70]).all()
    _check([70, 20], [70, 1], seed=15, change=far, window=12)
    _check([40, 20], [12, 1], seed=15, change=far, group=1)
    # past the table's width
    for rows in (1, 50):
        c, table, q = _setup([100], [rows], 2, 2, 64, 15)
        got = _call(c, np.ascontiguousarray(table[:, :2]), q, [100], [rows])
        assert np.isnan(got[max(0, rows - 36):]).all()
        want, bound = O.attention(c, q.astype(np.float64), np.ascontiguousarray(table[:, :2]), [100], None)
        assert_close(got, want, bound + 2.0 ** -22 * np.abs(want), "short table")


def test_row_bounds_out_of_range_are_held():
    _check([40, 30], [10, 10], cu=np.array([-5, 10, 99], dtype=np.int32), seed=16)
    _check([40, 20], [10, 10], cu=None, seed=16)


@pytest.mark.parametrize("rows", [1, 6, 80])
def test_small_hints_change_nothing_that_matters(rows):
    """More rows and longer sequences than the launch was shaped for."""
    _check([700, 90], [rows, 3], seed=17, max_rows=1, max_length=1)
    _check([700, 90], [rows, 3], seed=17, max_rows=1, max_length=128)
    _check([700, 90], [rows, 3], seed=17, max_rows=rows, max_length=300)
    _check([700, 90], [rows, 3], seed=17, max_rows=1, max_length=700)
    _check([700, 90], [rows, 3], seed=17, max_rows=4096, max_length=1 << 25)


def test_long_cache():
    _check([20000, 77], [1, 1], heads=1, group=2, seed=18)
    _check([20001], [3], heads=1, group=4, D=128, window=5000, seed=18)


@pytest.mark.parametrize("rows", [1, 6, 40])
def test_split_caches_with_small_hints(rows):
    """Caches that are split, with more rows, tokens or both than the launch was
    shaped for, and a sequence that fewer splits have blocks of."""
    _check([3000, 90], [rows, 3], seed=22, max_rows=1, max_length=2000)
    _check([3000, 90], [rows, 3], seed=22, max_rows=rows, max_length=2000)
    _check([3000, 90, 0], [rows, 3, 1], seed=22, max_rows=rows, max_length=4096)
    _check([3000, 90], [rows, 3], seed=22, max_rows=1, max_length=3000, window=1700)


def test_split_caches_with_nans_and_missing_blocks():
    def nan_value(c, table, q):
        for t, which in ((100, 1), (2998, 1), (1500, 0)):
            i = table[0, t // 32]
            codes = c.block_codes(i, 1, which).copy()
            codes[t % 32, 7] = 0x7F
            c.put(i, 1, which, codes, c.exps[i, 1, which])

    got = _check([3000], [5], seed=23, change=nan_value)
    assert np.isfinite(got[:, :2]).all() and np.isnan(got[:, 2:]).all()

    def missing(c, table, q):
        table = table.copy()
        table[0, 93] = -1
        return table, q

    got = _check([3000], [40], seed=23, change=missing)
    assert np.isfinite(got[:16]).all() and np.isnan(got[16:]).all()


def test_offsets_past_32_bits():
    """Blocks whose bytes lie past 2^32 in the cache."""
    heads, D = 8, 128
    blocks = (1 << 32) // (heads * 2 * 32 * D) + 40
    small, table, q = _setup([90, 33], [40, 1], heads, 1, D, 19)
    data = torch.zeros(q4.kv_cache_bytes(blocks, heads, D), dtype=torch.uint8, device=DEV)
    cache = q4.KVCache(data, blocks, heads, D)
    codes, exps = cache.planes()
    shift = blocks - small.blocks
    codes[shift:].copy_(dev(small.codes))
    exps[shift:].copy_(dev(small.exps))
    far = np.where(table >= 0, table + shift, table).astype(np.int32)
    say("attention far blocks")
    got = q4.kv_attention(dev(q.reshape(41, -1), torch.bfloat16), cache, dev(far), dev(np.array([90, 33], dtype=np.int32)),
                          dev(np.array([0, 40, 41], dtype=np.int32)), dtype=torch.float32)
    want, bound = O.attention(small, q.astype(np.float64), table, [90, 33], [0, 40, 41])
    assert_close(got.double().cpu().numpy().reshape(q.shape), want, bound + 2.0 ** -22 * np.abs(want), "far")
    # and appended there
    rng = np.random.default_rng(19)
    k, v = (rng.standard_normal((2, heads, D)).astype(np.float32) for _ in range(2))
    say("append far blocks")
    q4.kv_append(*(dev(x.reshape(2, -1)) for x in (k, k, v)), cache, dev(far), dev(np.array([91, 34], dtype=np.int32)), None)
    O.append(small, k, k, v, table, [91, 34], None)
    nan = np.isnan(O.VALUES[small.codes])
    assert np.array_equal(O.VALUES[codes[shift:].cpu().numpy()][~nan], O.VALUES[small.codes][~nan])
    assert np.array_equal(exps[shift:].cpu().numpy(), small.exps)
    assert not codes[:shift].any()


def test_repeats_bit_for_bit_with_a_kept_workspace():
    c, table, q = _setup([3000, 500], [2, 2], 2, 4, 128, 20)
    cache = device_cache(c)
    qd, td, ld = dev(q.reshape(4, -1), torch.bfloat16), dev(table), dev(np.array([3000, 500], dtype=np.int32))
    need = q4.kv_attention_workspace(cache, td, 4, 8, max_rows=2, max_length=3000)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device=DEV)
    say("attention workspace", need)
    a = q4.kv_attention(qd, cache, td, ld, max_rows=2, max_length=3000, workspace=ws)
    b = q4.kv_attention(qd, cache, td, ld, max_rows=2, max_length=3000, workspace=ws)
    d = q4.kv_attention(qd, cache, td, ld, max_rows=2, max_length=3000)
    assert torch.equal(a, b) and torch.equal(a, d)


def test_refusals():
    cache = q4.KVCache.empty(2, 2, 64, DEV)
    t = torch.zeros((1, 2), dtype=torch.int32, device=DEV)
    n = torch.ones(1, dtype=torch.int32, device=DEV)
    q = torch.zeros((1, 256), dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: q4.kv_attention(q.float(), cache, t, n), lambda: q4.kv_attention(q[:, :200], cache, t, n),
                lambda: q4.kv_attention(q, cache, t.long(), n), lambda: q4.kv_attention(q, cache, t[0], n),
                lambda: q4.kv_attention(q, cache, t, n, n), lambda: q4.kv_attention(q, cache, t, n, dtype=torch.float16),
                lambda: q4.kv_attention(q, cache, t, n, out=torch.empty((1, 128), dtype=torch.bfloat16, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q4.kv_attention(q[:, :192].contiguous(), cache, t, n), lambda: q4.kv_attention(q, cache, t, n, window=-1),
                lambda: q4.kv_attention(q, cache, t, n, scale=float("nan"))):
        with pytest.raises(q4.Q4Error):
            bad()
    wide = torch.zeros((1, 4096), dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        q4.kv_attention(q, cache, wide, n, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
