"""Pins of the oracle for beam search, the cache's pages and selected blocks:
worked by hand, or counted another way."""

import itertools
import math

import numpy as np
import pytest

from oracle import decoder_oracle as O
from oracle import search_oracle as S


def test_beam_select_by_hand():
    # two beams of four tokens: probabilities 1/2 1/4 1/8 1/8, and 1/4 each
    z = np.log(np.array([[4, 2, 1, 1], [1, 1, 1, 1]], dtype=np.float64)).astype(np.float32)
    scores = np.array([[math.log(0.4), 0.0]], dtype=np.float32)
    p, t, s = S.beam_select(z, scores, 5)
    # the second beam's equal tokens in their order, then 0.4 / 2
    assert p.tolist() == [[1, 1, 1, 1, 0]] and t.tolist() == [[0, 1, 2, 3, 0]]
    np.testing.assert_allclose(s[0], np.log([0.25, 0.25, 0.25, 0.25, 0.2]), atol=1e-6)


def test_beam_select_finished_masked_and_short():
    z = np.array([[0, -np.inf, 0], [1, 2, 3], [np.nan, 0, 0], [np.inf, 0, 0]], dtype=np.float32)
    scores = np.array([[-1, -0.5], [-0.1, -0.1]], dtype=np.float32)
    p, t, s = S.beam_select(z, scores, 4, finished=np.array([[0, 1], [0, 0]]), pad=7)
    assert p[0].tolist() == [1, 0, 0, -1] and t[0].tolist() == [7, 0, 2, -1]
    np.testing.assert_allclose(s[0, :3], [-0.5, -1 - math.log(2), -1 - math.log(2)])
    assert p[1].tolist() == [-1] * 4 and np.isneginf(s[1]).all()     # neither row has a probability


def test_beam_select_against_every_candidate():
    rng = np.random.default_rng(0)
    z = rng.integers(0, 4, (6, 50)).astype(np.float32)     # many ties
    scores = rng.integers(-2, 1, (2, 3)).astype(np.float32)
    p, t, s = S.beam_select(z, scores, 9)
    for g in range(2):
        every = sorted(((-(scores[g, b] + (z[3 * g + b, v] - np.log(np.exp(z[3 * g + b].astype(np.float64)).sum()))), b, v)
                        for b, v in itertools.product(range(3), range(50))))[:9]
        assert [(x // 1 - 3 * g, y) for x, y in zip(p[g], t[g])] == [(b, v) for _, b, v in every]


def test_beam_advance_by_hand():
    seq = np.array([[1, 2, 9, 9], [3, 4, 5, 6], [7, 0, 0, 0]])
    out, n, done = S.beam_advance(seq, [2, 4, 1], [0, 1, 2, -1, 0], [5, 5, 8, 3, 8], finished=[0, 0, 1], eos=8, pad=-9)
    assert out.tolist() == [[1, 2, 5, -9], [3, 4, 5, 6], [7, -9, -9, -9], [-9] * 4, [1, 2, 8, -9]]
    assert n.tolist() == [3, 4, 1, 0, 3] and done.tolist() == [0, 1, 1, 1, 1]


def test_fork_by_hand():
    # row 0: 40 tokens in blocks 5, 3; row 1: 64 tokens in 5, 1
    table, lengths = np.array([[5, 3, -1], [5, 1, -1]]), [40, 64]
    f = S.kv_fork(table, lengths, [0, 0, 1, -1], 8, 1)
    # the first continuation of row 0 copies block 3, the last keeps it; row 1's needs a new block
    assert f["block_table"].tolist() == [[5, 0, -1], [5, 3, -1], [5, 1, 2], [-1, -1, -1]]
    assert f["src"].tolist() == [3, -1, -1, -1] and f["dst"].tolist() == [0, -1, -1, -1]
    assert f["lengths"].tolist() == [41, 41, 65, 0] and f["refs"].tolist() == [1, 1, 1, 1, 0, 3, 0, 0]
    # a store that holds block 3 as well, and one block left
    held = [0, 0, 1, 1, 1, 0, 1, 1]
    f = S.kv_fork(table, lengths, [0, 0], 8, 1, held)
    assert f["src"].tolist() == [3, 3] and f["dst"].tolist() == [0, 1]
    f = S.kv_fork(table, lengths, [0, 1, 0], 8, [1, 0, 1], held)
    assert f["dst"].tolist() == [0, -1, -1] and f["short"].tolist() == [0, 0, 1] and f["block_table"][2].tolist() == [5, -1, -1]


def test_compact_by_hand():
    table, lengths = np.array([[6, 0, 3], [6, 7, -1]]), [70, 50]
    c = S.kv_compact(table, lengths, 9)
    assert c["live"].tolist() == [4] and c["src"].tolist() == [6, 7, -1, -1] and c["dst"].tolist() == [1, 2, -1, -1]
    assert c["block_table"].tolist() == [[1, 0, 3], [1, 2, -1]]
    c = S.kv_compact(table, lengths, 9, held=[0, 0, 0, 0, 0, 0, 0, 1, 1])
    assert c["live"].tolist() == [5] and c["src"].tolist() == [6, -1, -1, -1] and c["block_table"].tolist() == [[1, 0, 3], [1, 7, -1]]


def test_bounds_hold_for_every_code():
    codes = np.arange(256, dtype=np.uint8)[:, None]
    hi, lo = S.bounds(codes[~np.isnan(O.VALUES[codes[:, 0]])])
    assert (hi[0], lo[0]) == (112, -112)
    for c in range(256):
        v = O.VALUES[c]
        hi, lo = S.bounds(np.array([[c]], dtype=np.uint8))
        assert (hi[0], lo[0]) == (127, -127) if np.isnan(v) else 4 * lo[0] <= v <= 4 * hi[0] and hi[0] - lo[0] <= 1


def test_scores_bound_the_products():
    """With the quantization of q (half a step of 2^(E - 13) for each of 2 D sums) the
    score is no less than the largest sum of q . k of the block."""
    rng = np.random.default_rng(1)
    D, group = 64, 3
    c = O.Cache.empty(4, 1, D)
    O.fill_random(c, rng)
    q = rng.standard_normal((1, group, D)).astype(np.float32)
    summary = np.zeros((4, 1, 2, D), dtype=np.int64)
    S.summarize(c, summary, np.array([[0, 1, 2, 3]]), [128], 128)
    up, down = np.maximum(q[0], 0).sum(0), np.minimum(q[0], 0).sum(0)
    e = math.frexp(max(up.max(), -down.min()))[1]
    for i in range(4):
        whole = np.rint(np.concatenate((up, down)) * 2.0 ** (13 - e)).astype(np.int64)
        scale = 4 * 2.0 ** (e - 13 + int(c.exps[i, 0, 0]))
        score = scale * int(whole @ summary[i, 0].reshape(-1))
        k = O.VALUES[c.block_codes(i, 0, 0)] * 2.0 ** int(c.exps[i, 0, 0])
        assert score + scale * 0.5 * np.abs(summary[i, 0]).sum() >= (q[0] @ k.T).sum(0).max()


def test_select_takes_the_first_of_equal_scores_and_the_forced_ones():
    c = O.Cache.empty(9, 1, 64)
    table = np.arange(9)[None]
    summary = np.zeros((9, 1, 2, 64), dtype=np.int64)
    q = np.ones((1, 1, 64))
    assert S.select(c, summary, q, table, [280], 5, 1, 2)[0, 0].tolist() == [0, 1, 2, 7, 8]
    summary[5, 0, 0, 3] = 1
    assert S.select(c, summary, q, table, [280], 4, 1, 2)[0, 0].tolist() == [0, 5, 7, 8]
    assert S.select(c, summary, q, table, [60], 4, 1, 2)[0, 0].tolist() == [0, 1, -1, -1]
    table[0, 5] = 99
    assert S.select(c, summary, q, table, [280], 4, 1, 2)[0, 0].tolist() == [0, 1, 7, 8]


@pytest.mark.parametrize("D,group", [(64, 1), (128, 3)])
def test_attention_over_all_blocks_is_attention(D, group):
    rng = np.random.default_rng(2)
    c = O.Cache.empty(5, 2, D)
    O.fill_random(c, rng)
    q = rng.standard_normal((4, 2 * group, D))
    table, lengths = np.array([[3, 1, -1], [0, 4, 2]]), [40, 96]
    chosen = np.broadcast_to(np.array([2, 0, -1, 1]), (4, 2, 4))
    got, _ = S.attention_blocks(c, q, chosen, table, lengths)
    want, _ = O.attention(c, q, table, lengths)
    np.testing.assert_allclose(got, want, rtol=1e-12, atol=1e-14)


def test_planted_mistakes_are_caught():
    """The hand-worked pins tell these slips from the definitions."""
    table, lengths = np.array([[5, 3, -1], [5, 1, -1]]), [40, 64]
    right = S.kv_fork(table, lengths, [0, 0, 1, -1], 8, 1)
    wrong = S.kv_fork(table, [64, 64], [0, 0, 1, -1], 8, 1)          # a partly filled block taken for a full one
    assert wrong["src"].tolist() != right["src"].tolist()
    z = np.log(np.array([[4, 2, 1, 1], [1, 1, 1, 1]])).astype(np.float32)
    p, t, _ = S.beam_select(z, np.array([[0.0, 0.0]], dtype=np.float32), 5)   # the beams' scores left out
    assert p.tolist() != [[1, 1, 1, 1, 0]]
