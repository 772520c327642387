"""q4_add_rmsnorm against the oracle in 64 bits.

Tolerance, with E = 2^-24 and a row of C elements: a mean of squares summed in
fp32 by at most 16 or so terms a thread and a tree is within (C / 256 + 24) E
of itself, its root and reciprocal half of that and a few roundings more; r'
takes the roundings of its four operations on magnitudes that its parts bound,
x the relative errors of r' and of the root and three roundings; bf16 results
add 2^-8 of the value."""

import numpy as np
import pytest
import torch

from oracle import decoder_oracle as O
import q4_weight_only_amd as q4

from decoder_helpers import DEV, assert_close, dev
from gpu_helpers import say

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


def _check(M, C, *, y=True, post=False, gate=0, mod=0, scale=1.0, eps=1e-5, rd=torch.float32, yd=torch.float32,
           xd=torch.float32, seed=0, change=None, inplace=False):
    rng = np.random.default_rng([seed, M, C])

    def rand(*shape):
        return rng.standard_normal(shape).astype(np.float32)

    res, yy = dev(rand(M, C) * 2).to(rd), dev(rand(M, C)).to(yd) if y else None
    if change:
        change(res, yy)
    w = 1 + 0.2 * rand(C)
    pw = 1 + 0.2 * rand(C) if post else None
    g = 0.5 + 0.3 * rand(gate, C) if gate else None
    md = 0.3 * rand(mod, C) if mod else None
    want_r, want_x = O.add_rmsnorm(res.double().cpu().numpy(), w, yy.double().cpu().numpy() if y else None, pw, g, scale, md, eps)
    parts = np.abs(res.double().cpu().numpy()) + (np.abs(want_r - res.double().cpu().numpy()) if y else 0)
    say("norm", M, C, y, post, gate, mod, rd, yd, xd)
    r, x = q4.add_rmsnorm(res, dev(w), yy, post_weight=dev(pw), gate=dev(g), scale=scale, modulation=dev(md), eps=eps, dtype=xd,
                          residual_out=res if inplace else None)
    rel = (C / 256 + 40) * E
    rms = np.sqrt((want_r ** 2).mean(1, keepdims=True) + eps)
    size_x = np.abs(w) / rms * (1 + (np.repeat(np.abs(md), M // mod, 0) if mod else 0))
    with np.errstate(invalid="ignore"):
        bound_r = rel * parts + (2.0 ** -8 * np.abs(want_r) if rd == torch.bfloat16 else 0) + 1e-38
        bound_x = size_x * rel * (parts + np.abs(want_r)) + (2.0 ** -8 * np.abs(want_x) if xd == torch.bfloat16 else 0) + 1e-38
        if y:
            assert_close(r.double().cpu().numpy(), want_r, bound_r, "residual")
        else:
            assert r is res
        assert_close(x.double().cpu().numpy(), want_x, bound_x, "x")
    assert r.dtype == rd and x.dtype == xd
    return r, x


@pytest.mark.parametrize("C", [32, 64, 96, 992, 1024, 1056, 1280, 2048, 3072, 4096, 5120, 8192, 8224, 9216, 40000])
@pytest.mark.parametrize("M", [1, 2, 5, 33])
def test_sizes(M, C):
    _check(M, C, post=True, gate=1, mod=1, scale=0.7)
    _check(M, C, xd=torch.bfloat16)


@pytest.mark.parametrize("M", [300, 1505])
@pytest.mark.parametrize("C", [96, 1280, 3072])
def test_many_rows(M, C):
    _check(M, C, post=True, gate=M, mod=M, scale=0.5)
    _check(M, C, rd=torch.bfloat16, xd=torch.bfloat16)


@pytest.mark.parametrize("M,C", [(4, 256), (4, 288), (2047, 512), (2050, 288), (2051, 512), (4097, 32), (511, 3072), (513, 3104),
                                 (3, 8224), (3, 12320), (3, 16384), (3, 16416)])
def test_sizes_at_which_the_launch_changes(M, C):
    _check(M, C, post=True, gate=1, mod=M, scale=0.5)
    _check(M, C, rd=torch.bfloat16, xd=torch.bfloat16, inplace=True)


@pytest.mark.parametrize("rd", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("yd", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("xd", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [6, 600])
def test_types(rd, yd, xd, M):
    for C in (320, 3072, 9216):
        _check(M, C, rd=rd, yd=yd, xd=xd, post=True, gate=2, mod=3, seed=1)
        _check(M, C, rd=rd, yd=yd, xd=xd, seed=2, inplace=True)


@pytest.mark.parametrize("gate,mod", [(0, 0), (1, 0), (0, 1), (3, 4), (12, 6), (2, 12)])
def test_shared_gates_and_modulations(gate, mod):
    _check(12, 160, gate=gate, mod=mod, scale=-1.5, seed=3)
    _check(12, 160, gate=gate, mod=mod, post=True, seed=3)


def test_norm_alone():
    for M in (1, 40, 700):
        _check(M, 3072, y=False, mod=1)
        _check(M, 9216, y=False, xd=torch.bfloat16, rd=torch.bfloat16)


def test_in_place():
    for C in (64, 3072, 9216):
        for M in (5, 600):
            _check(M, C, inplace=True, post=True, gate=M)


def test_rows_of_zeros():
    def change(res, y):
        res[0] = 0
        y[0] = 0
        y[1] = 0

    _check(3, 96, post=True, change=change)
    _check(3, 96, post=True, change=lambda r, y: (r.fill_(0), y.fill_(0)))
    r, x = q4.add_rmsnorm(torch.zeros((2, 64), device=DEV), torch.ones(64, device=DEV), torch.zeros((2, 64), device=DEV), eps=0.0,
                          dtype=torch.float32)
    assert not r.any() and torch.isnan(x).all()       # 0 / 0


def test_rows_that_are_not_finite_stay_apart():
    def change(res, y):
        y[1, 7], res[3, 0] = float("nan"), float("inf")

    r, x = _check_finite_rows(change)
    assert torch.isnan(x[1]).all() and torch.isnan(x[3, 0]) and not x[3, 1:].any()


def _check_finite_rows(change):
    rng = np.random.default_rng(5)
    res, y = (dev(rng.standard_normal((6, 320)).astype(np.float32)) for _ in range(2))
    change(res, y)
    w = torch.ones(320, device=DEV)
    r, x = q4.add_rmsnorm(res, w, y, dtype=torch.float32)
    keep = [0, 2, 4, 5]
    r2, x2 = q4.add_rmsnorm(res[keep].contiguous(), w, y[keep].contiguous(), dtype=torch.float32)
    assert torch.equal(r[keep], r2) and torch.equal(x[keep], x2) and torch.isfinite(x2).all()
    return r, x


def test_large_and_small_values():
    _check(4, 320, change=lambda r, y: r.mul_(1e15))
    _check(4, 320, change=lambda r, y: (r.mul_(1e-12), y.mul_(1e-12)), eps=0.0)


def test_empty():
    r, x = q4.add_rmsnorm(torch.empty((0, 64), device=DEV), torch.ones(64, device=DEV), torch.empty((0, 64), device=DEV))
    assert tuple(x.shape) == (0, 64)


def test_refusals():
    r, w = torch.zeros((4, 64), device=DEV), torch.ones(64, device=DEV)
    for bad in (lambda: q4.add_rmsnorm(r.half(), w), lambda: q4.add_rmsnorm(r.t(), w), lambda: q4.add_rmsnorm(r, w[:32]),
                lambda: q4.add_rmsnorm(r, w, gate=w), lambda: q4.add_rmsnorm(r, w, r[:2]), lambda: q4.add_rmsnorm(r, w.bfloat16()),
                lambda: q4.add_rmsnorm(r, w, r, gate=torch.ones((3, 64), device=DEV)), lambda: q4.add_rmsnorm(r, w.cpu()),
                lambda: q4.add_rmsnorm(r, w, dtype=torch.float16), lambda: q4.add_rmsnorm(r, w, residual_out=r)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(q4.Q4Error):
        q4.add_rmsnorm(torch.zeros((4, 48), device=DEV), torch.ones(48, device=DEV))
    with pytest.raises(q4.Q4Error):
        q4.add_rmsnorm(r, w, eps=-1.0)
