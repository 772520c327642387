"""The decoder operators' oracle against what its definitions say elsewhere:
torch's e4m3 type, brute force, and invariants of the operators."""

import math

import numpy as np
import pytest
import torch

from oracle import decoder_oracle as O


def test_e4m3_values_and_rounding_match_the_type():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(O.VALUES), np.isnan(want))
    assert np.array_equal(O.VALUES[~np.isnan(want)], want[~np.isnan(want)])
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 9, 20000), [0.0, -0.0, 448.0, -448.0]])
    mids = (O.VALUES[:126] + O.VALUES[1:127]) / 2     # every tie
    x = np.concatenate([x, mids, -mids]).astype(np.float32).clip(-448, 448)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.encode(x), got)


def test_exponent_is_the_smallest_that_holds():
    assert O.exponent(0.0) == -32 and O.exponent(448.0) == 0 and O.exponent(448.0 * (1 + 1e-9)) == 1
    assert O.exponent(224.0) == -1 and O.exponent(1e30) == 32 and O.exponent(1e-30) == -32


@pytest.mark.parametrize("D", [64, 128])
def test_layout_is_a_permutation(D):
    at = O.addresses(D)
    for which in range(2):
        assert sorted(at[which].reshape(-1).tolist()) == list(range(32 * D))


@pytest.mark.parametrize("D", [64, 128])
def test_layout_is_what_a_wave_reads(D):
    """K: lane (g, r) of 64 reading 16 bytes has token r of a half block and 16
    dimensions from 64 h + 16 g; V: tokens 4 g .. and 16 + 4 g .. of dimensions
    r and 16 + r of a run of 32."""
    at = O.addresses(D)
    k = np.empty((32 * D, 2), dtype=int)
    v = np.empty((32 * D, 2), dtype=int)
    for s in range(32):
        for d in range(D):
            k[at[0][s, d]] = v[at[1][s, d]] = -1
    for s in range(32):
        for d in range(D):
            k[at[0][s, d]] = (s, d)
            v[at[1][s, d]] = (s, d)
    for chunk in range(D // 32):
        for lane in range(64):
            g, r = lane // 16, lane % 16
            byte = (chunk * 64 + lane) * 16
            tt, h = divmod(chunk, D // 64)
            assert [tuple(x) for x in k[byte:byte + 16]] == [(16 * tt + r, 64 * h + 16 * g + j) for j in range(16)]
            assert [tuple(x) for x in v[byte:byte + 16]] == [
                (16 * jj + 4 * g + j, 32 * chunk + 16 * half + r) for half in range(2) for jj in range(2) for j in range(4)]


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(2)
    x = rng.standard_normal(64).astype(np.float32)
    ang = rng.uniform(0, 6, 16)
    cs = np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    for inter in (False, True):
        y = O.rotate(x, cs, 32, inter)
        assert np.array_equal(y[32:], x[32:])
        z = np.array([complex(x[2 * i], x[2 * i + 1]) if inter else complex(x[i], x[i + 16]) for i in range(16)])
        w = z * np.exp(1j * ang)
        got = np.array([complex(y[2 * i], y[2 * i + 1]) if inter else complex(y[i], y[i + 16]) for i in range(16)])
        assert np.abs(got - w).max() < 1e-6


def _two_ways(lengths_then, rng):
    """The same tokens appended one at a time and at once."""
    D, H = 64, 2
    n = lengths_then
    q = rng.standard_normal((n, 4, D)).astype(np.float32)
    k = rng.standard_normal((n, H, D)).astype(np.float32)
    v = rng.standard_normal((n, H, D)).astype(np.float32)
    table = np.array([[2, 0, 1, 3]], dtype=np.int32)
    one, many = O.Cache.empty(4, H, D), O.Cache.empty(4, H, D)
    qa = O.append(one, q, k, v, table, [n], None)
    qb = np.concatenate([O.append(many, q[t:t + 1], k[t:t + 1], v[t:t + 1], table, [t + 1], None) for t in range(n)])
    return one, many, qa, qb


def test_append_one_at_a_time_equals_at_once_up_to_the_smallest_codes():
    one, many, qa, qb = _two_ways(75, np.random.default_rng(3))
    assert np.array_equal(qa, qb)
    assert np.array_equal(one.exps[:3], many.exps[:3])
    a, b = O.VALUES[one.codes], O.VALUES[many.codes]
    # rescaled codes are rounded again only below 2^-6
    assert np.abs(a - b).max() <= 2.0 ** -9
    assert np.array_equal(a[np.abs(a) > 2.0 ** -5], b[np.abs(a) > 2.0 ** -5])


def test_attention_against_a_direct_softmax():
    rng = np.random.default_rng(4)
    c = O.Cache.empty(4, 2, 64)
    O.fill_random(c, rng)
    table = np.array([[3, 1, 0, -1]], dtype=np.int32)
    q = rng.standard_normal((2, 4, 64))
    o, bound = O.attention(c, q, table, [70])
    toks = [(3, s) for s in range(32)] + [(1, s) for s in range(32)] + [(0, s) for s in range(6)]
    for row, n in ((0, 69), (1, 70)):
        for h in range(4):
            k = np.array([[O.VALUES[c.codes[i, h // 2, 0, O.k_address(s, d, 64)]] for d in range(64)] for i, s in toks[:n]])
            v = np.array([[O.VALUES[c.codes[i, h // 2, 1, O.v_address(s, d, 64)]] for d in range(64)] for i, s in toks[:n]])
            k *= np.array([2.0 ** int(c.exps[i, h // 2, 0]) for i, _ in toks[:n]])[:, None]
            v *= np.array([2.0 ** int(c.exps[i, h // 2, 1]) for i, _ in toks[:n]])[:, None]
            w = np.exp(k @ q[row, h] / 8.0)
            want = (w[:, None] * v).sum(0) / w.sum()
            assert np.abs(o[row, h] - want).max() < 1e-12 * np.abs(v).max()
            assert np.all(bound[row, h] > 0) and np.all(bound[row, h] < 0.01 * np.abs(v).max())


def test_attention_of_equal_keys_is_the_mean_and_of_nothing_is_zero():
    c = O.Cache.empty(2, 1, 64)
    rng = np.random.default_rng(5)
    c.codes[:, :, 1] = O.encode(rng.standard_normal((2, 1, 32 * 64)) * 20)
    q = rng.standard_normal((1, 2, 64))
    o, _ = O.attention(c, q, np.array([[0, 1]], dtype=np.int32), [40])
    mean = np.concatenate([O.VALUES[c.block_codes(0, 0, 1)], O.VALUES[c.block_codes(1, 0, 1)]])[:40].mean(0)
    assert np.allclose(o[0], mean)
    o, _ = O.attention(c, q, np.array([[0, 1]], dtype=np.int32), [0])
    assert not o.any()


def test_norm_and_logits_on_small_numbers():
    r, x = O.add_rmsnorm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), y=np.array([[1.0, 1.0]]), gate=np.array([2.0, 0.0]),
                         scale=0.5, mod=np.array([[0.0, 1.0]]), eps=0.0)
    assert np.array_equal(r, [[4.0, 4.0]]) and np.allclose(x, [[1.0, 4.0]])
    z = np.array([[2.0, -2.0, 1.0, 0.5]])
    out, _ = O.logits_adjust(z, history=[0, 1, 1, 2], cu=[0, 4], prompt=[1], rho=[2.0], frequency=[0.25], presence=[0.5],
                             bias_ids=[3, 3], bias=[1.0, 2.0], cu_bias=[0, 2], mask=np.array([[0b1011]]))
    assert np.array_equal(out, [[1.0, -4.0 - 0.5 - 0.5, -math.inf, 3.5]])
