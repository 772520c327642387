"""q4_logits_adjust against the oracle in 64 bits: masked tokens exactly -inf,
the others within 8 roundings of the magnitudes that were added (a division or
product, the count's product, two subtractions, the biases' sum and its
addition; a list of n biases of one token adds n)."""

import numpy as np
import pytest
import torch

from oracle import decoder_oracle as O
import q4_weight_only_amd as q4

from decoder_helpers import DEV, assert_close, dev
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _case(M, V, rng, history=30, bias=5, mask="random"):
    n = rng.integers(0, history + 1, M) if history else np.zeros(M, dtype=int)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    nb = rng.integers(0, bias + 1, M) if bias else np.zeros(M, dtype=int)
    cub = np.concatenate([[0], np.cumsum(nb)]).astype(np.int32)
    words = (V + 31) // 32
    m = None
    if mask == "random":
        m = rng.integers(0, 1 << 32, (M, words), dtype=np.uint64).astype(np.uint32).view(np.int32)
    elif mask == "none":
        m = np.zeros((M, words), dtype=np.int32)
    f = lambda *s: rng.random(s).astype(np.float32)  # noqa: E731
    return dict(z=(rng.standard_normal((M, V)) * 4).astype(np.float32),
                history=(V * rng.random(cu[-1]) ** 3).astype(np.int32), cu=cu,
                prompt=np.array([rng.integers(0, k + 1) for k in n], dtype=np.int32),
                rho=1 + f(M), frequency=f(M), presence=f(M),
                bias_ids=rng.integers(0, V, cub[-1]).astype(np.int32), bias=(f(cub[-1]) - 0.5) * 20, cu_bias=cub, mask=m)


def _check(c, what, out=None):
    keep = {k: c[k] for k in ("prompt", "rho", "frequency", "presence")}
    want, size = O.logits_adjust(c["z"], c["history"], c["cu"], *keep.values(), c["bias_ids"], c["bias"], c["cu_bias"],
                                 None if c["mask"] is None else c["mask"].view(np.uint32))
    say("logits", c["z"].shape, what)
    z = dev(c["z"])
    got = q4.logits_adjust(z, history=dev(c["history"]), cu_history=dev(c["cu"]), prompt_lengths=dev(c["prompt"]),
                           repetition=dev(c["rho"]), frequency=dev(c["frequency"]), presence=dev(c["presence"]),
                           bias_ids=dev(c["bias_ids"]), bias=dev(c["bias"]), cu_bias=dev(c["cu_bias"]), mask=dev(c["mask"]),
                           out=z if out == "z" else None)
    assert (got.data_ptr() == z.data_ptr()) == (out == "z")
    repeats = 0 if c["bias_ids"] is None or not len(c["bias_ids"]) else np.bincount(np.clip(c["bias_ids"], 0, None)).max()
    assert_close(got.cpu().numpy(), want, (8 + repeats) * 2.0 ** -24 * size, what)


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 100, 2047, 2048, 2049, 5001, 32000, 131072])
@pytest.mark.parametrize("M", [1, 3])
def test_sizes(M, V):
    _check(_case(M, V, np.random.default_rng([1, M, V])), "sizes")
    _check(_case(M, V, np.random.default_rng([2, M, V]), mask=None), "no mask", out="z")


def test_many_rows():
    _check(_case(40, 3001, np.random.default_rng(3), history=500, bias=100), "rows")
    _check(_case(257, 260, np.random.default_rng(3), history=90, bias=3), "rows")


def test_long_history():
    _check(_case(2, 20000, np.random.default_rng(4), history=30000, bias=3000), "long")


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 127, 511, 512, 513, 999, 1000, 1001, 2047, 2048, 2049, 4099, 8191, 8192, 8193, 8195,
                               16387])
def test_history_of(n):
    rng = np.random.default_rng([41, n])
    for M, V, prompt in ((1, 5003, n // 2), (2, 131, n), (3, 4098, 0)):
        c = _case(M, V, rng, bias=7)
        c["cu"] = (np.arange(M + 1) * n).astype(np.int32)
        c["history"] = rng.integers(0, V, M * n).astype(np.int32)
        c["prompt"] = np.full(M, prompt, dtype=np.int32)
        _check(c, f"history of {n}")


@pytest.mark.parametrize("n", [1, 127, 128, 129, 511, 512, 513, 2047, 2048, 2049, 4100])
@pytest.mark.parametrize("history", [10, 3000])
def test_biases_of(n, history):   # of different tokens, and with one that is there twice
    rng = np.random.default_rng([42, n, history])
    for repeated in (False, True):
        c = _case(2, 9001, rng, history=history, bias=0)
        c["cu_bias"] = np.array([0, n, 2 * n], dtype=np.int32)
        c["bias_ids"] = np.concatenate([rng.permutation(9001)[:n], rng.permutation(9001)[:n]]).astype(np.int32)
        if repeated:
            c["bias_ids"][n - 1] = c["bias_ids"][n // 2]
        c["bias"] = rng.standard_normal(2 * n).astype(np.float32) * 5
        _check(c, f"biases of {n}")


def test_everything_masked():
    c = _case(2, 5000, np.random.default_rng(5), mask="none")
    _check(c, "masked")
    got = q4.logits_adjust(dev(c["z"]), mask=dev(c["mask"]))
    assert torch.isneginf(got).all()


def test_nothing_given_is_a_copy():
    z = torch.randn((3, 777), device=DEV)
    assert torch.equal(q4.logits_adjust(z), z)


@pytest.mark.parametrize("part", ["rho", "frequency", "presence", "prompt", "history", "bias_ids"])
def test_each_part_may_be_missing(part):
    c = _case(3, 3000, np.random.default_rng(6))
    c[part] = None
    if part == "history":
        c["cu"] = None
    if part == "bias_ids":
        c["bias"] = c["cu_bias"] = None
    _check(c, part)


def test_empty_lists():
    c = _case(2, 300, np.random.default_rng(7), history=0, bias=0)
    _check(c, "empty")


def test_a_token_with_many_biases_and_counts():
    rng = np.random.default_rng(8)
    c = _case(2, 4000, rng)
    c["history"], c["cu"] = np.full(5000, 17, dtype=np.int32), np.array([0, 3000, 5000], dtype=np.int32)
    c["prompt"] = np.array([10, 2000], dtype=np.int32)
    c["bias_ids"] = np.concatenate([np.full(600, 17), np.full(3, 2049)]).astype(np.int32)
    c["bias"] = rng.standard_normal(603).astype(np.float32)
    c["cu_bias"] = np.array([0, 600, 603], dtype=np.int32)
    _check(c, "repeats")


def test_repeated_biases_add_in_their_order():
    z = torch.zeros((1, 64), device=DEV)
    vals = [1.0, 2.0 ** 24, -(2.0 ** 24), 0.25]      # in this order 0.25, in others 1.25
    got = q4.logits_adjust(z, bias_ids=dev(np.full(4, 9, dtype=np.int32)), bias=dev(np.array(vals, dtype=np.float32)),
                           cu_bias=dev(np.array([0, 4], dtype=np.int32)))
    want = np.float32(0)
    for v in vals:
        want = np.float32(want + np.float32(v))
    assert float(got[0, 9]) == float(want)


def test_ids_out_of_range_are_passed_over():
    c = _case(2, 300, np.random.default_rng(9))
    c["history"] = np.array([-1, 300, 5, 2**31 - 1, -2**31, 299], dtype=np.int32)
    c["cu"], c["prompt"] = np.array([0, 4, 6], dtype=np.int32), np.array([0, 1], dtype=np.int32)
    c["bias_ids"], c["bias"] = np.array([300, -5, 7, 2**31 - 1], dtype=np.int32), np.ones(4, dtype=np.float32)
    c["cu_bias"] = np.array([0, 3, 4], dtype=np.int32)
    _check(dict(c, bias_ids=c["bias_ids"]), "out of range")


def test_row_bounds_out_of_range_are_held():
    c = _case(3, 300, np.random.default_rng(10))
    c["history"] = np.arange(10, dtype=np.int32)
    c["cu"], c["prompt"] = np.array([-4, 3, 99, 2], dtype=np.int32), np.zeros(3, dtype=np.int32)
    c["bias_ids"], c["bias"] = np.arange(6, dtype=np.int32), np.ones(6, dtype=np.float32)
    c["cu_bias"] = np.array([2, 1, 50, -3], dtype=np.int32)
    _check(c, "bounds")


def test_logits_that_are_not_finite():
    c = _case(1, 200, np.random.default_rng(11), mask=None)
    c["z"][0, :4] = [np.inf, -np.inf, np.nan, 0.0]
    c["history"], c["cu"], c["prompt"] = np.array([0, 1, 2, 3], dtype=np.int32), np.array([0, 4], dtype=np.int32), np.array([4], dtype=np.int32)
    _check(c, "not finite")
    c["mask"] = np.zeros((1, 7), dtype=np.int32)
    _check(c, "not finite, masked")


def test_refusals():
    z = torch.zeros((2, 100), device=DEV)
    i = torch.zeros(4, dtype=torch.int32, device=DEV)
    for bad in (lambda: q4.logits_adjust(z.half()), lambda: q4.logits_adjust(z[0]), lambda: q4.logits_adjust(z.t()),
                lambda: q4.logits_adjust(z, history=i), lambda: q4.logits_adjust(z, history=i, cu_history=i),
                lambda: q4.logits_adjust(z, bias_ids=i, cu_bias=i[:3]), lambda: q4.logits_adjust(z, mask=i),
                lambda: q4.logits_adjust(z, repetition=torch.ones(3, device=DEV)), lambda: q4.logits_adjust(z, out=z[:1])):
        with pytest.raises(ValueError):
            bad()
