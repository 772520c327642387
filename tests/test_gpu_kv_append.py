"""q4_kv_append against the oracle, bit for bit: codes, exponents and the
rotated q.  (Codes are decided by fp32 products and sums that both sides round
one by one; -0 and +0 are one value.)"""

import numpy as np
import pytest
import torch

from oracle import decoder_oracle as O
import q4_weight_only_amd as q4

from decoder_helpers import DEV, bf16, dev, device_cache, random_table
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _rope(positions, rot, theta=1.0e4):
    return q4.rope_table(positions, rot, theta, device="cpu").numpy() if rot else None


def _same_cache(cache: q4.KVCache, want: O.Cache, what):
    codes, exps = (t.cpu().numpy() for t in cache.planes())
    assert np.array_equal(exps, want.exps), f"{what}: exponents"
    a, b = O.VALUES[codes], O.VALUES[want.codes]
    assert np.array_equal(np.isnan(a), np.isnan(b)), f"{what}: NaN codes"
    assert np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)]), f"{what}: codes"


def _check(lengths, rows, *, heads=2, group=2, D=64, rot=None, inter=False, dtype=torch.float32, cu=True, seed=0,
           tweak=None, max_rows=None, table=None, blocks=None, positions=None, garbage=False):
    rng = np.random.default_rng(seed)
    total = sum(rows)
    rot = D if rot is None else rot
    hq = heads * group
    q, k, v = (rng.standard_normal((total, h, D)).astype(np.float32) for h in (hq, heads, heads))
    big = np.where(rng.random((total, 1, 1)) < 0.3, 8.0, 1.0).astype(np.float32)
    k, v = k * big, v * big
    if tweak:
        tweak(q, k, v)
    if dtype == torch.bfloat16:
        q, k, v = bf16(q), bf16(k), bf16(v)
    need = sum(-(-max(n, 0) // 32) for n in lengths)
    blocks = blocks or need + 2
    c = O.Cache.empty(blocks, heads, D)
    if garbage:
        c.data[:] = rng.integers(0, 256, c.data.size).astype(np.uint8)
        c.exps[:] = rng.integers(-6, 3, c.exps.shape)
    else:
        O.fill_random(c, rng)
    if table is None:
        table = random_table(rng, lengths, blocks)
    rope = _rope(positions or max(max(lengths), 1), rot)
    bounds = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32) if cu is True else cu
    cache = device_cache(c)
    args = (dev(table), dev(np.array(lengths, dtype=np.int32)), dev(rope), dev(bounds))
    say("append", lengths, rows, heads, group, D, rot, inter, dtype)
    for again in range(2):      # writing the same rows again changes nothing
        out = torch.full((total, hq * D), 7.0, dtype=torch.bfloat16, device=DEV)
        got = q4.kv_append(*(dev(x.reshape(total, -1), dtype) for x in (q, k, v)), cache, *args, interleaved=inter,
                           max_rows=max_rows, out=out)
        if again == 0:
            want_q = O.append(c, q, k, v, table, lengths, rope, bounds, inter)
            owned = np.zeros(total, dtype=bool)
            for b in range(len(lengths)):
                row0, n, _ = O._sequence(bounds, lengths, b, total)
                owned[row0:row0 + n] = True
            want_q[~owned] = 7.0      # rows of no sequence are left as they were
        _same_cache(cache, c, f"call {again}")
        assert np.array_equal(got.float().cpu().numpy().reshape(want_q.shape), bf16(want_q), equal_nan=True)
    return cache, c


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
def test_prompts_and_single_tokens(D, dtype, inter):
    _check([33, 1, 70, 40], [33, 1, 1, 9], D=D, dtype=dtype, inter=inter, seed=1)


@pytest.mark.parametrize("lengths,rows", [([1], [1]), ([32], [1]), ([33], [1]), ([33], [2]), ([64], [64]), ([65], [33]),
                                          ([95], [31]), ([300, 1], [1, 1]), ([20, 45, 61], [3, 14, 29])])
def test_edges_of_blocks(lengths, rows):
    _check(lengths, rows, seed=2)
    _check(lengths, rows, seed=3, D=128, heads=1, group=7, rot=64)


@pytest.mark.parametrize("heads,group,rot", [(1, 1, 64), (8, 4, 32), (3, 5, 0), (2, 64, 64), (20, 1, 32)])
def test_heads_and_partial_rotation(heads, group, rot):
    _check([5, 66], [5, 2], heads=heads, group=group, rot=rot, seed=4)
    _check([66, 5], [2, 5], heads=heads, group=group, rot=rot, inter=True, seed=5)


def test_uniform_rows_without_bounds():
    _check([7, 64, 35], [3, 3, 3], cu=None, seed=6)
    _check([7, 64, 35], [1, 1, 1], cu=None, seed=6)


def test_idle_slots_and_more_rows_than_tokens():
    _check([0, 40, 3, 0], [1, 1, 5, 0], seed=7)


def test_a_small_hint_for_the_rows_changes_nothing():
    _check([200, 9], [150, 9], max_rows=1, seed=8)


def test_row_bounds_out_of_range_are_held():
    _check([20, 20], [10, 10], cu=np.array([-5, 10, 99], dtype=np.int32), seed=9)
    _check([20, 20], [10, 10], cu=np.array([15, 3, 20], dtype=np.int32), seed=9)


def test_blocks_outside_the_cache_are_not_written():
    table = np.array([[0, 99, 2], [-7, 1, 2**31 - 1]], dtype=np.int32)
    _check([96, 70], [80, 70], table=table, blocks=3, seed=10)
    _check([200], [120], table=np.array([[2, 1]], dtype=np.int32), blocks=3, seed=11)     # past the table's width


def test_positions_past_the_rope_table_are_nan():
    _check([40], [12], positions=33, seed=12)
    _check([40], [12], positions=33, rot=32, inter=True, D=128, seed=12)


def test_bytes_of_an_earlier_use_are_overwritten_or_kept():
    _check([45, 64, 31], [45, 32, 1], garbage=True, seed=13)


def test_exponent_grows_with_the_block_and_starts_anew():
    """Tokens ten binades larger each time, then a block over an old one."""
    rng = np.random.default_rng(14)
    c = O.Cache.empty(2, 1, 64)
    cache = device_cache(c)
    table = np.array([[1]], dtype=np.int32)
    for n, size in ((1, 2.0 ** -20), (2, 2.0 ** -10), (3, 1.0), (4, 2.0 ** 10), (5, 1.0), (1, 1.0), (2, 0.5)):
        q, k, v = (rng.standard_normal((1, 1, 64)).astype(np.float32) * np.float32(size) for _ in range(3))
        say("append growth", n, size)
        q4.kv_append(*(dev(x.reshape(1, -1)) for x in (q, k, v)), cache, dev(table), dev(np.array([n], dtype=np.int32)), None)
        O.append(c, q, k, v, table, [n], None)
        _same_cache(cache, c, f"{n} {size}")


def test_values_that_are_not_finite_or_out_of_range():
    def tweak(q, k, v):
        k[0, 0, 3], k[1, 0, 5], k[2, 1, 0] = np.nan, np.inf, -np.inf
        v[0, 1, 9], v[3, 0, 0], v[4, 1, 1] = np.inf, np.nan, 3.0e38
        k[5] = 0.0
        v[6:9] = 1.0e-30
        q[0, 0, 0], q[1, 0, 0] = np.inf, np.nan

    _check([12, 50], [12, 6], rot=0, tweak=tweak, seed=15)
    _check([12, 50], [12, 6], rot=32, tweak=tweak, seed=15)
    _check([1], [1], rot=0, tweak=lambda q, k, v: (k.fill(0), v.fill(np.nan)), seed=16)


def test_values_on_the_edge_of_an_exponent():
    def tweak(q, k, v):
        k[:] = 0.1
        v[:] = 0.1
        k[0, 0, 0], v[0, 0, 0] = 448.0, np.nextafter(np.float32(448), np.float32(1e9))
        k[0, 1, 0], v[0, 1, 0] = -3.5, np.nextafter(np.float32(3.5), np.float32(0))

    _check([8], [8], rot=0, tweak=tweak, seed=17)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_a_wider_tensor(dtype):
    rng = np.random.default_rng(18)
    H, G, D, rows = 2, 3, 64, 37
    wide = torch.from_numpy(rng.standard_normal((rows, (H * G + 2 * H) * D + 16)).astype(np.float32)).to(DEV, dtype)
    q, k, v = wide[:, :H * G * D], wide[:, H * G * D:(H * G + H) * D], wide[:, (H * G + H) * D:(H * G + 2 * H) * D]
    c = O.Cache.empty(3, H, D)
    cache = device_cache(c)
    table, lengths, rope = np.array([[2, 0]], dtype=np.int32), np.array([rows], dtype=np.int32), _rope(rows, D)
    say("append strided", dtype)
    got = q4.kv_append(q, k, v, cache, dev(table), dev(lengths), dev(rope))
    a, b, e = (t.float().cpu().numpy().reshape(rows, -1, D) for t in (q, k, v))
    want = O.append(c, a, b, e, table, lengths, rope)
    _same_cache(cache, c, "strided")
    assert np.array_equal(got.float().cpu().numpy().reshape(want.shape), bf16(want))


def test_empty_batch():
    cache = q4.KVCache.empty(2, 1, 64, DEV)
    z = torch.empty((0, 64), device=DEV)
    out = q4.kv_append(z, z, z, cache, torch.zeros((1, 1), dtype=torch.int32, device=DEV),
                       torch.zeros(1, dtype=torch.int32, device=DEV), None)
    assert tuple(out.shape) == (0, 64)


def test_refusals():
    cache = q4.KVCache.empty(2, 2, 64, DEV)
    t = torch.zeros((1, 2), dtype=torch.int32, device=DEV)
    n = torch.ones(1, dtype=torch.int32, device=DEV)
    q, k = torch.zeros((1, 256), device=DEV), torch.zeros((1, 128), device=DEV)
    rope = q4.rope_table(4, 64, device=DEV)
    with pytest.raises(ValueError):
        q4.kv_append(q, k, k.half(), cache, t, n, rope)
    with pytest.raises(ValueError):
        q4.kv_append(q, k, k.bfloat16(), cache, t, n, rope)
    with pytest.raises(ValueError):
        q4.kv_append(q, k[:, :64], k, cache, t, n, rope)
    with pytest.raises(ValueError):
        q4.kv_append(q, k, k, cache, t.long(), n, rope)
    with pytest.raises(ValueError):
        q4.kv_append(q, k, k, cache, t, n, rope[:, :, 0].contiguous())
    with pytest.raises(ValueError):
        q4.kv_append(q, k, k, cache, t, n.cpu(), rope)
    with pytest.raises(q4.Q4Error):
        q4.kv_append(q[:, :192].contiguous(), k, k, cache, t, n, rope)      # 3 heads over 2
    with pytest.raises(q4.Q4Error):
        q4.kv_append(q, k, k, cache, t, n, q4.rope_table(4, 48, device=DEV))
    with pytest.raises(ValueError):
        q4.KVCache(torch.zeros(5, dtype=torch.uint8, device=DEV), 2, 2, 64)
    with pytest.raises(ValueError):
        q4.KVCache.empty(2, 2, 80, DEV)
