"""q4_kv_attention at the edges of its arithmetic: weights that are small beside
another token's, factors that underflow in a join, scores that are infinite,
huge or all equal.  Each with the launch that its sizes choose, split and not,
and with two tiles of rows a wave."""

import numpy as np
import pytest
import torch

from oracle import decoder_oracle as O
import q4_weight_only_amd as q4

from decoder_helpers import assert_close, bf16, dev, device_cache, random_table
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _setup(length, rows, heads, group, D, seed):
    rng = np.random.default_rng(seed)
    c = O.Cache.empty(-(-length // 32) + 1, heads, D)
    O.fill_random(c, rng)
    table = random_table(rng, [length], c.blocks)
    return c, table, bf16(rng.standard_normal((rows, heads * group, D)))


def _call(c, table, q, length, **kw):
    say("attention values", q.shape, length, kw)
    out = q4.kv_attention(dev(q.reshape(q.shape[0], -1), torch.bfloat16), device_cache(c), dev(table),
                          dev(np.array([length], dtype=np.int32)), dtype=torch.float32, **kw)
    return out.double().cpu().numpy().reshape(q.shape)


def _put(c, table, token, which, codes, exponent=None):
    """Codes [heads, D] of a token, and its block's exponent."""
    i = table[0, token // 32]
    for h in range(c.heads):
        all_codes = c.block_codes(i, h, which).copy()
        all_codes[token % 32] = codes[h]
        c.put(i, h, which, all_codes, c.exps[i, h, which] if exponent is None else exponent)


def _check(c, table, q, length, **kw):
    got = _call(c, table, q, length, **kw)
    want, bound = O.attention(c, q.astype(np.float64), table, [length], None, kw.get("window", 0), kw.get("scale"))
    assert_close(got, want, bound * (1 + 2.0 ** -22) + 2.0 ** -22 * np.abs(want), "attention")
    return got


# the launch that the sizes choose (split for the long lengths here), an unsplit one, and two tiles of rows a wave
HINTS = [{}, dict(max_length=32), dict(max_rows=1 << 15, max_length=32)]


@pytest.mark.parametrize("hints", HINTS)
@pytest.mark.parametrize("rows", [1, 9])
def test_nan_value_in_a_part_whose_weights_underflow(rows, hints):
    """Later keys score some hundred higher, so that 2^(m - top) of the blocks
    before is 0 in fp32; 0 times what is not a number is not a number all the same."""
    c, table, q = _setup(3000, rows, 2, 2, 64, 30)
    i = table[0, 2000 // 32]
    c.exps[i, :, 0] += 10
    codes = np.stack([c.block_codes(table[0, 3], h, 1)[4] for h in range(2)])
    codes[:, 7] = 0x7F
    _put(c, table, 100, 1, codes)
    got = _check(c, table, q, 3000, **hints)
    assert np.isnan(got[:, :, 7]).all() and np.isfinite(got[:, :, 8]).all()


@pytest.mark.parametrize("hints", HINTS)
@pytest.mark.parametrize("D,rows,lead", [(64, 1, 17.5), (128, 2, 17.5), (64, 40, 17.5), (128, 40, 14.0), (64, 1, 20.0)])
def test_one_leading_token_over_a_long_tail(D, rows, lead, hints):
    """Token 5 leads the others by `lead` nats and has values of zero: what is
    left is the sum of 20000 weights of about 2^-25 of its own."""
    length = 20000
    c, table, q = _setup(length, rows, 1, 2, D, 31)
    rng = np.random.default_rng(32)
    q = np.broadcast_to(q[:1, :1], q.shape).copy()     # one query, so that one key leads all of them
    q[...] = bf16(np.sign(q) * 0.5)
    for b in range(table.shape[1] - 1):     # values with a common mean, so that the tail does not cancel
        c.put(table[0, b], 0, 1, O.encode(1.0 + 0.25 * rng.standard_normal((32, D))), 0)
        c.put(table[0, b], 0, 0, O.encode(0.5 * rng.standard_normal((32, D))), 0)
    key = O.encode(np.sign(q[0, 0]) * lead / (0.5 * D ** 0.5))
    _put(c, table, 5, 0, key[None])
    _put(c, table, 5, 1, np.zeros((1, D), dtype=np.uint8))
    got = _check(c, table, q, length, **hints)
    assert (got > 0).all()


@pytest.mark.parametrize("hints", HINTS)
@pytest.mark.parametrize("length,rows", [(1, 1), (40, 3), (40, 40), (3000, 2)])
def test_scores_that_are_all_minus_infinity(length, rows, hints):
    """exp(-inf - -inf) is not a number; only a row that sees nothing gives 0."""
    c, table, q = _setup(length, rows, 1, 2, 64, 33)
    for b in range(-(-length // 32)):
        codes = c.block_codes(table[0, b], 0, 0).copy()
        codes[:, 3] = 0x30 + rng_bits(b)
        c.put(table[0, b], 0, 0, codes, c.exps[table[0, b], 0, 0])
    q[0, 0, 3] = -np.inf
    got = _check(c, table, q, length, **hints)
    assert np.isnan(got[0, 0]).all() and np.isfinite(got[0, 1]).all()
    empty = _call(c, table, q, 0, **hints)
    assert not empty.any()


def rng_bits(b):
    return np.random.default_rng(b).integers(0, 16, 32).astype(np.uint8)


@pytest.mark.parametrize("hints", HINTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [12, 20, 26, 30, 60])
def test_huge_scores(power, sign, D, hints):
    """Scores of about 2^power.  A row that sees one token gives its value, and
    one whose tokens' scores lie far apart the value of the largest: here they
    are 1, 2, .. 80 times one score (or, negative, the first token's is the
    largest)."""
    rows = 80
    c, table, q = _setup(rows, rows, 1, 1, D, 34)
    q[...] = bf16(np.full(q.shape, 2.0 ** (power / 2)))
    for b in range(3):
        n = np.arange(32 * b + 1, 32 * b + 33)
        for j in range(32):      # sum over d of codes with the value n: exact in e4m3 as a sum of two
            codes = np.zeros(D)
            codes[0], codes[1] = n[j] // 8 * 8, n[j] % 8
            c_codes = c.block_codes(table[0, b], 0, 0).copy()
            c_codes[j] = O.encode(sign * codes)
            c.put(table[0, b], 0, 0, c_codes, power // 2)
    got = _call(c, table, q, rows, **hints)
    k = np.array([O.VALUES[c.block_codes(table[0, t // 32], 0, 0)[t % 32]].sum() for t in range(rows)])
    assert np.array_equal(k, sign * np.arange(1, rows + 1))
    v = np.array([O.VALUES[c.block_codes(table[0, t // 32], 0, 1)[t % 32]] * 2.0 ** int(c.exps[table[0, t // 32], 0, 1])
                  for t in range(rows)])
    want = v if sign > 0 else np.broadcast_to(v[:1], v.shape)
    # the next weight is 2^-(2^power / sqrt(D)) of the largest, none that fp32 holds; what is left is the
    # weight's rounding to fp16, which the sum does not have, and two roundings
    assert_close(got[:, 0], want, (2.0 ** -11 + 2.0 ** -22) * np.abs(want), "huge scores")


@pytest.mark.parametrize("hints", HINTS)
@pytest.mark.parametrize("rows", [1, 50])
def test_scale_of_zero_weighs_all_alike(rows, hints):
    """Also where q . k is large."""
    c, table, q = _setup(70, rows, 2, 2, 64, 35)
    _check(c, table, bf16(q * 2.0 ** 60), 70, scale=0.0, **hints)
