"""kv_summarize and kv_select: whole numbers, equal to the oracle's."""

import numpy as np
import pytest
import torch

from oracle import decoder_oracle as O
from oracle import search_oracle as S
import q4_weight_only_amd as q4

from decoder_helpers import DEV, bf16, dev, device_cache, random_table
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _bounds_of(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


def _cache(lengths, heads, D, seed, blocks=None):
    rng = np.random.default_rng(seed)
    c = O.Cache.empty(blocks or sum(-(-max(n, 0) // 32) for n in lengths) + 2, heads, D)
    O.fill_random(c, rng)
    return rng, c, random_table(rng, lengths, c.blocks)


# -------------------------------------------------------------- summarize
def _summarize(c, table, lengths, rows, cu=True, **kw):
    rng = np.random.default_rng(9)
    want = rng.integers(-128, 128, (c.blocks, c.heads, 2, c.D))    # the bounds of other blocks stay
    got = dev(want, torch.int8)
    bounds = _bounds_of(rows) if cu else None
    say("kv_summarize", c.blocks, c.heads, c.D, lengths, rows)
    q4.kv_summarize(device_cache(c), got, dev(table, torch.int32), dev(np.array(lengths), torch.int32), dev(bounds), rows=sum(rows), **kw)
    S.summarize(c, want, table, lengths, sum(rows), bounds)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [1, 4, 5])
@pytest.mark.parametrize("lengths,rows", [([1], [1]), ([16], [16]), ([17], [1]), ([31, 32, 33], [1, 1, 1]), ([200, 64], [77, 64]),
                                          ([0, 50, 9], [1, 3, 12]), ([130, 7], [0, 2])])
def test_summarize(lengths, rows, heads, D):
    rng, c, table = _cache(lengths, heads, D, 1)
    _summarize(c, table, lengths, rows)
    _summarize(c, table, lengths, rows, max_rows=1)           # as for one row; the others follow
    _summarize(c, table, lengths, rows, max_rows=5000)


def test_summarize_what_is_not_a_number():
    rng, c, table = _cache([100], 2, 64, 2)
    for b in range(c.blocks):
        for h in range(2):
            codes = c.block_codes(b, h, 0).copy()
            codes[rng.random(codes.shape) < 0.01] = 0x7F
            codes[rng.random(codes.shape) < 0.01] = 0xFF
            c.put(b, h, 0, codes, 3)
    codes = c.block_codes(table[0, 3], 0, 0).copy()
    codes[4:] = 0x7F                                          # slots behind the last token hold anything
    c.put(table[0, 3], 0, 0, codes, -5)
    _summarize(c, table, [100], [100])


def test_summarize_every_code():
    """Blocks of one code each, of zeros of both signs and of pairs."""
    c = O.Cache.empty(256, 1, 64)
    for i in range(256):
        codes = np.full((32, 64), i, dtype=np.uint8)
        codes[1, 1], codes[2, 2] = 0x80, 0x00
        c.put(i, 0, 0, codes, 0)
    _summarize(c, np.arange(256)[None], [256 * 32], [256 * 32])


def test_summarize_ids_outside_the_cache_and_rows_of_equal_number():
    rng, c, table = _cache([90, 70], 3, 64, 3)
    table[0, 1], table[1, 2] = -1, c.blocks
    _summarize(c, table, [90, 70], [90, 70])
    _summarize(c, table[:, :2], [90, 70], [90, 70])           # past the table
    _summarize(c, table, [90, 70], [7, 7], cu=False)


# ------------------------------------------------------------------ select
def _select(c, table, q, lengths, rows, keep, first, recent, cu=True, summary=None, max_blocks=None, **kw):
    if summary is None:
        summary = np.zeros((c.blocks, c.heads, 2, c.D), dtype=np.int64)
        for i in range(c.blocks):
            for h in range(c.heads):
                summary[i, h] = S.bounds(c.block_codes(i, h, 0))
    bounds = _bounds_of(rows) if cu else None
    say("kv_select", c.heads, c.D, q.shape, lengths, rows, keep, first, recent)
    got = q4.kv_select(dev(q.reshape(q.shape[0], -1), torch.bfloat16), device_cache(c), dev(summary, torch.int8), dev(table, torch.int32),
                       dev(np.array(lengths), torch.int32), dev(bounds), keep=keep, first=first, recent=recent, **kw)
    want = S.select(c, summary, q.astype(np.float64), table, lengths, keep, first, recent, bounds,
                    *([] if max_blocks is None else [max_blocks]))
    # rows of no sequence are not written
    inside = slice(0, q.shape[0]) if bounds is None else slice(bounds[0], bounds[-1])
    assert np.array_equal(got.cpu().numpy()[inside], want[inside])
    return want


def _queries(rng, rows, heads, D):
    return bf16(rng.standard_normal((rows, heads, D)) * np.exp(rng.standard_normal((rows, 1, 1)) * 3))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (3, 7), (1, 64), (20, 1)])
@pytest.mark.parametrize("lengths,rows", [([1], [1]), ([700], [1]), ([700, 33, 1000], [1, 1, 1]), ([900, 300], [5, 19])])
def test_select(lengths, rows, heads, group, D):
    rng, c, table = _cache(lengths, heads, D, 1)
    q = _queries(rng, sum(rows), heads * group, D)
    _select(c, table, q, lengths, rows, 8, 1, 2, max_rows=max(rows), max_length=max(lengths))
    _select(c, table, q, lengths, rows, 8, 1, 2)


@pytest.mark.parametrize("keep,first,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (3, 1, 2), (5, 0, 0), (7, 7, 0), (20, 3, 4), (21, 0, 21), (22, 1, 1),
                                               (23, 1, 2), (64, 1, 2), (300, 10, 100)])
def test_keep_first_and_recent(keep, first, recent):
    rng, c, table = _cache([700, 690, 1], 2, 64, 2)
    q = _queries(rng, 6, 4, 64)
    _select(c, table, q, [700, 690, 1], [3, 2, 1], keep, first, recent)


@pytest.mark.parametrize("count", [1023, 1024, 1025, 1500, 4096, 4097, 9000, 16384, 16385, 40000])
def test_many_blocks(count):
    """Every size of the workgroups that choose.  A table may name a block many times, so that many scores are equal."""
    rng = np.random.default_rng(count)
    c = O.Cache.empty(40, 1, 64)
    O.fill_random(c, rng)
    table = rng.integers(0, 40, (1, count))
    q = _queries(rng, 2, 2, 64)
    n = count * 32 - 5
    _select(c, table, q, [n], [2], 100, 2, 3, max_rows=2)


def test_chunks_of_many_rows():
    rng, c, table = _cache([1200, 40], 2, 128, 3)
    q = _queries(rng, 140, 4, 128)
    _select(c, table, q, [1200, 40], [100, 40], 12, 1, 1, max_rows=100, max_length=1200)
    _select(c, table, q, [1200, 40], [100, 40], 12, 1, 1, max_rows=1, max_length=1200)


@pytest.mark.parametrize("group", [1, 3])
@pytest.mark.parametrize("top", [0.75, 1.5, 3.0, 6.0, 12.0])
def test_sums_halfway_between_two_whole_numbers(top, group):
    """Q in steps of 2^(E - 13), and many halves of them: these go to the even one, whatever the power of two."""
    rng, c, table = _cache([25000, 20000], 2, 64, 22)
    q = np.zeros((40, 2 * group, 64))
    step = 2.0 ** (np.frexp(top)[1] - 13)
    q[:, ::group] = (2 * rng.integers(-120, 120, (40, 2, 64)) + 1) * step / 2     # odd halves, within 8 bits
    q[:, :, 0] = 0
    q[:, ::group, 0] = top
    assert np.array_equal(bf16(q), q)
    _select(c, table, q, [25000, 20000], [20, 20], 30, 1, 2)


@pytest.mark.parametrize("count", [66, 67, 130, 250, 1000, 3000])
@pytest.mark.parametrize("spread", [3, 30])
def test_scores_that_are_far_apart(count, spread):
    """A few blocks whose exponents are far above the others', so that these fall into one bin, or a few."""
    rng = np.random.default_rng(count)
    c = O.Cache.empty(count, 1, 64)
    O.fill_random(c, rng)
    for b in range(count):
        c.put(b, 0, 0, c.block_codes(b, 0, 0), 20 if b % 97 == 5 else int(rng.integers(-spread, 1)))
    table = rng.permutation(count)[None]
    q = _queries(rng, 3, 4, 64)
    for keep in (4, 20, 40):
        _select(c, table, q, [32 * count - 1], [3], keep, 1, 2)


@pytest.mark.parametrize("max_length", [639, 640, 641, 672, 5000])
def test_as_many_as_there_are(max_length):
    """keep of 20, which is all blocks up to 640 tokens."""
    rng, c, table = _cache([600, 33, 640], 2, 64, 21)
    q = _queries(rng, 6, 4, 64)
    q[0] = np.nan                      # no score is looked at
    _select(c, table, q, [600, 33, 640], [3, 1, 2], 20, 1, 2, max_length=max_length)


def test_positions_past_max_length_have_no_blocks():
    rng, c, table = _cache([300, 90], 1, 64, 4)
    q = _queries(rng, 2, 1, 64)
    want = _select(c, table, q, [300, 90], [1, 1], 4, 1, 1, max_length=96, max_blocks=3)
    assert (want[0] == -1).all() and (want[1] >= 0).any()


def test_rows_without_a_position_and_idle_slots():
    rng, c, table = _cache([2, 0, 100], 2, 64, 5)
    q = _queries(rng, 9, 2, 64)
    want = _select(c, table, q, [2, 0, 100], [4, 2, 3], 3, 1, 1)
    assert (want[:2] == -1).all() and (want[4:6] == -1).all()
    q = _queries(rng, 6, 2, 64)
    _select(c, table, q, [2, 0, 100], [2, 2, 2], 3, 1, 1, cu=False)


def test_rows_behind_the_last_sequence_stay():
    rng, c, table = _cache([100], 1, 64, 6)
    q = _queries(rng, 5, 1, 64)
    out = torch.full((5, 1, 2), 77, dtype=torch.int32, device=DEV)
    cu = np.array([1, 3], dtype=np.int32)
    q4.kv_select(dev(q.reshape(5, -1), torch.bfloat16), device_cache(c), q4.kv_summary(device_cache(c)), dev(table, torch.int32),
                 dev(np.array([100]), torch.int32), dev(cu), keep=2, first=0, recent=1, out=out)
    assert (out[[0, 3, 4]] == 77).all() and (out[1:3] != 77).all()


def test_unknown_blocks_and_scores_that_are_equal():
    rng, c, table = _cache([600], 1, 64, 7)
    table[0, [3, 9, 10]] = [-1, c.blocks, -5]
    q = _queries(rng, 1, 3, 64)
    _select(c, table, q, [600], [1], 17, 1, 1)               # more than there are known ones
    _select(c, table, q, [600], [1], 6, 1, 1)
    _select(c, table[:, :12], q, [600], [1], 13, 1, 1, max_length=600)     # blocks past the table are unknown
    assert (_select(c, table[:, :12], q, [600], [1], 13, 1, 1, max_blocks=12) == -1).all()   # as far as the table reaches
    _select(c, table, q, [600], [1], 6, 1, 1, summary=np.ones((c.blocks, 1, 2, 64), dtype=np.int64))


def test_queries_of_every_size():
    """Zeros, what is not finite, the largest and the smallest numbers; rows of q that are alike but for a power of two
    choose alike."""
    rng, c, table = _cache([800], 2, 64, 8)
    q = _queries(rng, 8, 4, 64)
    q[0], q[1, 0, 3], q[2, 3, 60], q[3] = 0, np.nan, np.inf, -0.0
    q[4] = q[5] * np.float32(2.0 ** 100)
    q[6] *= np.float32(2.0 ** -120)
    q[7, :, 10] = 3.3e38
    q = bf16(q)
    want = _select(c, table, q, [800], [8], 9, 1, 1)
    assert np.array_equal(want[4], want[5])


def test_bounds_at_their_ends():
    """Sums as large as they get: every bound 127 or -127, every query of one sign and size."""
    rng, c, table = _cache([500], 1, 128, 9)
    summary = rng.choice([127, -127], (c.blocks, 1, 2, 128))
    for sign in (1, -1):
        q = np.full((1, 2, 128), sign * 1.9921875, dtype=np.float32)
        _select(c, table, q, [500], [1], 6, 0, 1, summary=summary)
    for i in range(c.blocks):
        c.exps[i, 0, 0] = (-32, 32, 0)[i % 3]
    _select(c, table, q, [500], [1], 6, 0, 1, summary=summary)


def test_outputs_and_workspace_of_the_caller():
    rng, c, table = _cache([900], 2, 64, 10)
    q, cache, lengths, tab = dev(_queries(rng, 1, 4, 64).reshape(1, -1), torch.bfloat16), device_cache(c), dev(np.array([900]), torch.int32), dev(table, torch.int32)
    summary = q4.kv_summary(cache)
    q4.kv_summarize(cache, summary, tab, dev(np.array([900]), torch.int32), rows=900)
    want = q4.kv_select(q, cache, summary, tab, lengths, keep=7, max_length=900)
    ws = torch.full((q4.kv_select_workspace(cache, tab, 1, max_length=900),), 255, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(want)
    got = q4.kv_select(q, cache, summary, tab, lengths, keep=7, max_length=900, out=out, workspace=ws)
    assert torch.equal(got, want) and got.data_ptr() == out.data_ptr()


def test_refusals():
    c = q4.KVCache.empty(5, 2, 64)
    s, t, n = q4.kv_summary(c), torch.zeros((1, 4), dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    q = torch.zeros((1, 256), dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: q4.kv_summarize(c, s.float(), t, n, rows=1), lambda: q4.kv_summarize(c, s[:4].contiguous(), t, n, rows=1),
                lambda: q4.kv_summarize(c, s, t.long(), n, rows=1), lambda: q4.kv_summarize(c, s, t, n, rows=-1),
                lambda: q4.kv_select(q.float(), c, s, t, n, keep=3), lambda: q4.kv_select(q[:, :200], c, s, t, n, keep=3),
                lambda: q4.kv_select(q[:, :192].contiguous(), c, s, t, n, keep=3), lambda: q4.kv_select(q, c, s, t, n, keep=0),
                lambda: q4.kv_select(q, c, s, t, n, keep=2), lambda: q4.kv_select(q, c, s, t, n, keep=3, first=-1),
                lambda: q4.kv_select(q, c, s, t, n, keep=2**16 + 1), lambda: q4.kv_select(q, c, s.view(-1)[:-1], t, n, keep=3),
                lambda: q4.kv_select(q, c, s, t, n, keep=3, workspace=torch.empty(4, dtype=torch.uint8, device=DEV)),
                lambda: q4.kv_select(q, c, s, t, n, keep=3, out=torch.empty((1, 2, 4), dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            bad()
