"""beam_select and beam_advance against the oracle in 64 bits.  What is selected is
equal; a score is off by its rounding to fp32, half a step (2^-24 of it), and by the
kernels' exponentials, 3e-10 of the sum whose logarithm it has, so 1e-9."""

import numpy as np
import pytest
import torch

from oracle import search_oracle as S
import q4_weight_only_amd as q4

from decoder_helpers import DEV, dev
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _check(z, scores, keep, finished=None, pad=0):
    say("beam_select", z.shape, scores.shape, keep)
    z, scores = z.astype(np.float32), scores.astype(np.float32)
    p, t, s = q4.beam_select(dev(z), dev(scores), keep, finished=dev(finished, torch.int32), pad=pad)
    wp, wt, ws = S.beam_select(z, scores, keep, finished, pad)
    assert np.array_equal(p.cpu().numpy(), wp)
    assert np.array_equal(t.cpu().numpy(), wt)
    with np.errstate(over="ignore"):
        none = np.isinf(ws.astype(np.float32))    # there is none, or its score is beyond fp32
    got = s.double().cpu().numpy()
    assert np.array_equal(got[none], ws.astype(np.float32)[none])
    assert np.array_equal(np.isinf(got), none)
    assert (np.abs(got[~none] - ws[~none]) <= 2.0 ** -24 * np.abs(ws[~none]) + 1e-9).all()
    return wp


def _random(groups, beams, V, seed):
    rng = np.random.default_rng(seed)
    return rng, rng.standard_normal((groups * beams, V)) * 3, -5 * rng.random((groups, beams))


@pytest.mark.parametrize("groups,beams,V,keep", [
    (1, 1, 1, 1), (1, 1, 1, 8), (2, 4, 5, 8), (3, 2, 31, 2), (2, 3, 32, 6), (2, 3, 33, 3), (1, 4, 1000, 4), (5, 1, 4099, 5), (7, 5, 32003, 5),
    (1, 64, 300, 128), (4, 2, 257, 128), (2, 8, 131072, 16), (1, 4, 131072, 4), (1, 1, 1048577, 64)])
def test_shapes(groups, beams, V, keep):
    _, z, scores = _random(groups, beams, V, 1)
    _check(z, scores, keep)


@pytest.mark.parametrize("groups,beams,V", [(4, 8, 32000), (16, 4, 40001), (32, 8, 40000), (64, 8, 20000)])
def test_many_rows(groups, beams, V):
    """Rows and tokens that take every number of loads of a lane."""
    _, z, scores = _random(groups, beams, V, 2)
    _check(z, scores, beams)


@pytest.mark.parametrize("V", [100, 5000, 70001])
def test_finished_masked_and_dead_beams(V):
    rng, z, scores = _random(6, 4, V, 3)
    z[rng.random(z.shape) < 0.9] = -np.inf
    z[5] = -np.inf
    scores[0, 1:] = -np.inf            # the first step: one beam counts
    scores[2, 3], scores[2, 0] = np.nan, np.inf
    finished = np.zeros((6, 4))
    finished[3] = 1                    # a whole group
    finished[4, 1:3] = 2
    finished[0, 2] = 1                 # with a score of -inf
    _check(z, scores, 6, finished, pad=V + 7)


def test_rows_that_are_not_numbers():
    _, z, scores = _random(4, 2, 3000, 4)
    z[0, 17], z[3, 2999], z[4, 5], z[5, :] = np.nan, np.inf, -np.inf, -np.inf
    z[6, 100:200], z[7, 0] = np.nan, np.nan
    p = _check(z, scores, 5)
    assert p[0].tolist() == [1] * 5 and p[1].tolist() == [2] * 5 and p[3].tolist() == [-1] * 5


@pytest.mark.parametrize("V", [33, 40000, 200000])
@pytest.mark.parametrize("keep", [1, 16, 128])
def test_equal_logits(V, keep):
    """All logits are equal, in beams that are alike and in ones that are not: the first tokens of the first beam."""
    z, scores = np.full((6, V), 0.25), np.array([[0, 0, -1], [-2, -1, -2]])
    p = _check(z, scores, keep)
    assert (p[1, :min(keep, V)] == 4).all()


@pytest.mark.parametrize("at", [0, 1000, 36863])
def test_what_counts_lies_together(at):
    """A grammar that allows one run of tokens, as many as a workgroup's threads, in places next to each other."""
    rng, z, scores = _random(2, 3, 40000, 5)
    z[:, :at] = -np.inf
    z[:, at + 3137:] = -np.inf
    _check(z, scores, 100)


@pytest.mark.parametrize("V", [1000, 32003, 70000])
@pytest.mark.parametrize("keep", [1, 5, 16, 17, 64, 100, 128])
def test_one_beam_with_a_score(V, keep):
    """A search's first step: the other beams are at -inf."""
    rng, z, scores = _random(3, 8, V, keep)
    scores[:, 1:] = -np.inf
    scores[1] = np.roll(scores[1], 5)
    _check(z, scores, keep)
    z[:, V // 2:] = -np.inf      # and half of the tokens are not allowed
    _check(z, scores, keep)


@pytest.mark.parametrize("groups,beams,V,keep", [(3, 7, 1941, 7), (2, 6, 2497, 6), (4, 5, 4477, 10), (2, 64, 600, 128), (1, 40, 10000, 128),
                                                 (1, 64, 1000, 17), (2, 8, 3000, 100), (2, 2, 1500, 128), (2, 1, 4096, 128), (1, 1, 4097, 128)])
def test_few_parts_and_few_segments(groups, beams, V, keep):
    """A beam has few parts, or a group hardly more segments than are kept; also where one beam has all candidates,
    and where most tokens are held at the type's lowest value, which is a number."""
    rng, z, scores = _random(groups, beams, V, V)
    _check(z, scores, keep)
    z[:, rng.permutation(V)[: V - 3]] = np.finfo(np.float32).min
    _check(z, scores, keep)
    z, scores = _random(groups, beams, V, V + 1)[1:]
    scores[:, 1:] = -np.inf
    _check(z, scores, keep)


def test_few_values_many_ties():
    rng, _, _ = _random(1, 1, 1, 6)
    z, scores = rng.integers(0, 3, (8, 50000)), -np.array([[0.0, 0.3, 0.7, 1.1], [0.9, 0.2, 0.0, 0.1]])
    _check(z, scores, 100)


def test_large_and_small_logits():
    """Logits far from 0, far from each other and below fp32's normal numbers."""
    rng, z, scores = _random(4, 2, 9999, 7)
    z[0:2] += 1e6
    z[2:4] *= 1e30
    z[4:6] *= 1e-41
    z[6:8] -= 3e38
    for g in range(4):
        _check(z[2 * g:2 * g + 2], scores[g:g + 1], 3)


def test_lse_is_summed_in_64_bits():
    """Two beams whose scores differ by less than a sum in 32 bits is off by: the second one's
    tokens come first by 2e-7."""
    V = 131072
    z = np.zeros((2, V), dtype=np.float32)
    z[0, 5] = z[1, 5] = 1.0
    z[0, 1000:1100] = 2.6e-4       # the first row's sum is larger by 0.026 of 131073.7
    p, t, s = q4.beam_select(dev(z), dev(np.zeros((1, 2), dtype=np.float32)), 2)
    assert p.tolist() == [[1, 0]] and t.tolist() == [[5, 5]]
    _check(z, np.zeros((1, 2)), 2)


def test_outputs_and_workspace_of_the_caller():
    _, z, scores = _random(2, 3, 5000, 8)
    zd, sd = dev(z.astype(np.float32)), dev(scores.astype(np.float32))
    want = q4.beam_select(zd, sd, 4)
    out = tuple(torch.empty_like(x) for x in want)
    ws = torch.full((q4.beam_select_workspace(2, 3, 5000) + 16,), 255, dtype=torch.uint8, device=DEV)
    got = q4.beam_select(zd, sd, 4, out=out, workspace=ws)
    assert all(torch.equal(a, b) and a.data_ptr() == c.data_ptr() for a, b, c in zip(got, want, out))


def test_no_groups():
    p, t, s = q4.beam_select(torch.empty((0, 7), device=DEV), torch.empty((0, 3), device=DEV), 2)
    assert p.shape == t.shape == s.shape == (0, 2)


# ---------------------------------------------------------------- advance
def _advance(rows, width, n, seed, eos=3, dense=False):
    rng = np.random.default_rng(seed)
    seq = rng.integers(-5, 100, (rows, width))
    lengths = rng.integers(0, width + 1, rows) if not dense else np.full(rows, width - 1)
    parents, tokens = rng.integers(-2, rows + 2, n), rng.integers(-1, 6, n)
    finished = rng.integers(0, 2, rows)
    if rows > 2:
        lengths[0], lengths[1], lengths[2] = -7, width + 9, width
    for f in (finished, None):
        say("beam_advance", rows, width, n)
        got = q4.beam_advance(*(dev(x, torch.int32) for x in (seq, lengths, parents, tokens)), finished=dev(f, torch.int32), eos=eos, pad=77)
        want = S.beam_advance(seq, lengths, parents, tokens, f, eos, 77)
        for a, b in zip(got, want):
            assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("rows,width,n", [(1, 1, 1), (3, 2, 5), (4, 7, 9), (8, 1023, 8), (8, 1024, 16), (5, 1025, 3), (7, 4097, 6), (2, 40, 70000)])
def test_advance(rows, width, n):
    _advance(rows, width, n, 1)
    _advance(rows, width, n, 2, eos=-1, dense=True)


def test_advance_without_parents_or_rows():
    out, n, done = q4.beam_advance(torch.empty((0, 5), dtype=torch.int32, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV),
                                   dev(np.array([0, -1]), torch.int32), dev(np.array([4, 4]), torch.int32), pad=9)
    assert out.tolist() == [[9] * 5] * 2 and n.tolist() == [0, 0] and done.tolist() == [1, 1]


# ----------------------------------------------------------------- refusals
def test_refusals():
    z, s = torch.zeros((6, 10), device=DEV), torch.zeros((2, 3), device=DEV)
    for bad in (lambda: q4.beam_select(z.cpu(), s, 2), lambda: q4.beam_select(z, s.cpu(), 2), lambda: q4.beam_select(z.double(), s, 2),
                lambda: q4.beam_select(z, s[:, :2].contiguous(), 2), lambda: q4.beam_select(z[:, ::2], s, 2),
                lambda: q4.beam_select(z, s, 0), lambda: q4.beam_select(z, s, 129), lambda: q4.beam_select(z, s, 2, pad=-1),
                lambda: q4.beam_select(z, s, 2, finished=torch.zeros((2, 3), device=DEV)),
                lambda: q4.beam_select(z, s, 2, finished=torch.zeros((3, 2), dtype=torch.int32, device=DEV)),
                lambda: q4.beam_select(z, s, 2, workspace=torch.empty(8, dtype=torch.uint8, device=DEV)),
                lambda: q4.beam_select(z, s, 2, out=(z,)),
                lambda: q4.beam_select(torch.zeros((65, 4), device=DEV), torch.zeros((1, 65), device=DEV), 2)):
        with pytest.raises(ValueError):
            bad()
    i = torch.zeros((4, 8), dtype=torch.int32, device=DEV)
    for bad in (lambda: q4.beam_advance(i.float(), i[:, 0].contiguous(), i[0], i[0]), lambda: q4.beam_advance(i, i[0], i[0], i[0]),
                lambda: q4.beam_advance(i, i[0, :4], i[0], i[0, :4]), lambda: q4.beam_advance(i, i[0, :4], i[0], i[0], finished=i[0]),
                lambda: q4.beam_advance(i, i[0, :4], i[0], i[0], eos=2**40)):
        with pytest.raises(ValueError):
            bad()


def test_scores_as_large_as_numbers_get():
    """Where sums in fp32 would not be finite, with fewer candidates than are kept, and with more."""
    z = np.full((4, 700), -np.inf)
    z[:, [3, 500]] = [[1, 2], [3.4e38, -3.4e38], [-3e38, -3.3e38], [0, 1]]
    scores = np.array([[3.3e38, -3.4e38], [-3.2e38, 1e31]])
    _check(z, scores, 7)
    rng = np.random.default_rng(9)
    z = rng.standard_normal((4, 700)) * 1e38
    _check(z, scores, 7, finished=np.array([[0, 1], [0, 0]]))


def test_outputs_that_overlap_are_refused():
    z, s, i = torch.zeros((6, 10), device=DEV), torch.zeros((2, 3), device=DEV), torch.zeros((2, 3), dtype=torch.int32, device=DEV)
    j, seq = torch.zeros((2, 3), dtype=torch.int32, device=DEV), torch.zeros((4, 8), dtype=torch.int32, device=DEV)
    n, p = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    for bad in (lambda: q4.beam_select(z, s, 3, out=(None, None, s)), lambda: q4.beam_select(z, s, 3, out=(i, i, None)),
                lambda: q4.beam_select(z, s, 3, finished=i, out=(None, i, None)),
                lambda: q4.beam_advance(seq, n, p, p, out=(seq, None, None)), lambda: q4.beam_advance(seq, n, p, p, out=(None, n, None)),
                lambda: q4.beam_advance(seq, n, p, p, out=(None, None, p))):
        with pytest.raises(ValueError, match="overlap"):
            bad()
    got = q4.beam_select(z, s, 3, out=(i, j, None))
    assert got[0].data_ptr() == i.data_ptr() and got[1].data_ptr() == j.data_ptr()


@pytest.mark.parametrize("byte", [0, 255, 127])
@pytest.mark.parametrize("V", [100, 32003, 131072])
def test_what_a_workspace_held_does_not_matter(V, byte):
    """The rows of beams that have ended are not read, and nothing is written for them."""
    rng, z, scores = _random(3, 4, V, 11)
    z, scores = z.astype(np.float32), scores.astype(np.float32)
    finished = np.array([[0, 1, 0, 0], [1, 1, 1, 1], [1, 0, 1, 1]])
    want = S.beam_select(z, scores, 6, finished, 5)
    ws = torch.full((q4.beam_select_workspace(3, 4, V),), byte, dtype=torch.uint8, device=DEV)
    p, t, s = q4.beam_select(dev(z), dev(scores), 6, finished=dev(finished, torch.int32), pad=5, workspace=ws)
    assert np.array_equal(p.cpu().numpy(), want[0]) and np.array_equal(t.cpu().numpy(), want[1])
