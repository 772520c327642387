"""Plain CPU oracle for the decoder operators of include/q4_decoder.h.

TEST INFRASTRUCTURE ONLY, like q4_0_oracle: no code shared with the HIP
library or its binding.  Everything is NumPy and written from the definitions,
one row, head or block at a time; values are fp64 except where a definition
rounds (the rotation's products and sums, which decide codes, are fp32).

The cache is a flat uint8 array: codes [blocks][heads][K | V][32 * D], then
int8 exponents [blocks][heads][K | V].
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = 32
E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -32, 32


# ------------------------------------------------------------------- e4m3
def _code_value(c: int) -> float:
    sign, exp, frac = c >> 7, (c >> 3) & 15, c & 7
    if exp == 15 and frac == 7:
        return math.nan
    mag = (1 + frac / 8) * 2.0 ** (exp - 7) if exp else frac / 8 * 2.0 ** -6
    return -mag if sign else mag


VALUES = np.array([_code_value(c) for c in range(256)])
_POSITIVE = VALUES[:127]   # ascending, 0 .. 448


def encode(x) -> np.ndarray:
    """Nearest e4m3 code (ties to the even code), held to +-448; what is not
    finite becomes 0x7F.  The sign of a zero is kept."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), E4M3_MAX)
    hi = np.clip(np.searchsorted(_POSITIVE, mag), 1, 126)
    lo = hi - 1
    up, down = _POSITIVE[hi] - mag, mag - _POSITIVE[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(lo % 2 == 0, lo, hi)))
    code = code + 128 * np.signbit(x)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def exponent(amax: float) -> int:
    """The smallest e in -32 .. 32 with amax <= 448 * 2^e (32 if there is none)."""
    for e in range(EXP_MIN, EXP_MAX):
        if amax <= E4M3_MAX * 2.0 ** e:
            return e
    return EXP_MAX


# ------------------------------------------------------------------ layout
def k_address(slot: int, d: int, D: int) -> int:
    return ((((slot // 16) * (D // 64) + d // 64) * 4 + d // 16 % 4) * 16 + slot % 16) * 16 + d % 16


def v_address(slot: int, d: int, D: int) -> int:
    return (((d // 32 * 4 + slot // 4 % 4) * 16 + d % 16) * 2 + d // 16 % 2) * 8 + slot // 16 * 4 + slot % 4


def addresses(D: int) -> np.ndarray:
    """[2, 32, D]: where K's and V's codes of a slot and dimension are."""
    return np.array([[[f(s, d, D) for d in range(D)] for s in range(BLOCK)] for f in (k_address, v_address)])


class Cache:
    """A NumPy view of a cache's bytes with its sizes."""

    def __init__(self, data: np.ndarray, blocks: int, heads: int, D: int):
        self.data, self.blocks, self.heads, self.D = data, blocks, heads, D
        n = blocks * heads * 2 * BLOCK * D
        assert data.dtype == np.uint8 and data.size == n + blocks * heads * 2
        self.codes = data[:n].reshape(blocks, heads, 2, BLOCK * D)
        self.exps = data[n:].view(np.int8).reshape(blocks, heads, 2)
        self.at = addresses(D)

    @classmethod
    def empty(cls, blocks, heads, D, fill=0):
        return cls(np.full(blocks * heads * 2 * (BLOCK * D + 1), fill, dtype=np.uint8), blocks, heads, D)

    def block_codes(self, i: int, head: int, which: int) -> np.ndarray:
        """[32, D] codes in token order."""
        return self.codes[i, head, which][self.at[which]]

    def put(self, i, head, which, codes, e):
        self.codes[i, head, which][self.at[which]] = codes
        self.exps[i, head, which] = e


def fill_random(cache: Cache, rng, spread: int = 2, tilt: float = 0.5):
    """Gaussian values (some channels larger, exponents that differ from block
    to block), quantized by the rule."""
    for which in range(2):
        chan = np.exp(tilt * rng.standard_normal((cache.heads, 1, cache.D)))
        for i in range(cache.blocks):
            x = rng.standard_normal((cache.heads, BLOCK, cache.D)) * chan * 2.0 ** rng.integers(-spread, spread + 1)
            for h in range(cache.heads):
                e = exponent(np.abs(x[h]).max())
                cache.put(i, h, which, encode(x[h] * 2.0 ** -e), e)


# ------------------------------------------------------------------ append
def rotate(x: np.ndarray, cs: np.ndarray, rot: int, interleaved: bool) -> np.ndarray:
    """One head's vector [D] (fp32) by a row [rot / 2, 2] of the rope table, in
    fp32 with every product and sum rounded."""
    y = x.astype(np.float32).copy()
    with np.errstate(all="ignore"):
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = np.float32(cs[i, 0]), np.float32(cs[i, 1])
            y[a] = np.float32(x[a] * c) - np.float32(x[b] * s)
            y[b] = np.float32(x[b] * c) + np.float32(x[a] * s)
    return y


def _sequence(cu, lengths, b, rows):
    n = len(lengths)
    if cu is None:
        each = rows // n
        return b * each, each, max(int(lengths[b]), 0)
    lo = min(max(int(cu[b]), 0), rows)
    hi = min(max(int(cu[b + 1]), lo), rows)
    return lo, hi - lo, max(int(lengths[b]), 0)


def block_id(cache, table, b, i):
    if i >= table.shape[1]:
        return -1
    t = int(table[b, i])
    return t if 0 <= t < cache.blocks else -1


def append(cache: Cache, q, k, v, table, lengths, rope, cu=None, interleaved=False):
    """Appends in place; returns the rotated q in fp32 (before its rounding to
    bf16).  q, k, v fp32 [rows, heads, D]; rope fp32 [positions, rot / 2, 2]."""
    rows = q.shape[0]
    rot = 2 * rope.shape[1] if rope is not None else 0
    out = np.zeros(q.shape, dtype=np.float32)
    for b in range(len(lengths)):
        row0, n, length = _sequence(cu, lengths, b, rows)
        written: dict = {}
        for t in range(n):
            pos = length - n + t
            if pos < 0:
                continue
            kk = k[row0 + t].astype(np.float32).copy()
            out[row0 + t] = q[row0 + t]
            if rot and pos >= rope.shape[0]:
                out[row0 + t, :, :rot] = np.nan
                kk[:, :rot] = np.nan
            elif rot:
                for h in range(q.shape[1]):
                    out[row0 + t, h] = rotate(q[row0 + t, h], rope[pos], rot, interleaved)
                for h in range(cache.heads):
                    kk[h] = rotate(k[row0 + t, h], rope[pos], rot, interleaved)
            written.setdefault(pos // BLOCK, []).append((pos % BLOCK, kk, v[row0 + t].astype(np.float32)))
        for j, tokens in written.items():
            i = block_id(cache, table, b, j)
            if i < 0:
                continue
            for h in range(cache.heads):
                for which in range(2):
                    new = np.array([tok[1 + which][h] for tok in tokens], dtype=np.float64)
                    finite = np.abs(new[np.isfinite(new)])
                    e = exponent(finite.max() if finite.size else 0.0)
                    codes = cache.block_codes(i, h, which).copy()
                    if tokens[0][0] > 0:
                        before = int(cache.exps[i, h, which])
                        e = max(e, before)
                        if e > before:
                            old = VALUES[codes]
                            codes = np.where(np.isnan(old), codes, encode(old * 2.0 ** (before - e)))
                    for tok, x in zip(tokens, new):
                        codes[tok[0]] = encode(x * 2.0 ** -e)
                    cache.put(i, h, which, codes, e)
    return out


# --------------------------------------------------------------- attention
def attention(cache: Cache, q, table, lengths, cu=None, window=0, scale=None):
    """(o, bound): fp64 [rows, q_heads, D] of q (fp64 values of bf16,
    [rows, q_heads, D]) and how far a result in the kernels' arithmetic may be
    from it, before the output's rounding.

    The bound, for one row and head, with p the softmax weights, u_j = p_j
    2^eV_j the weight of token j's codes, n the tokens seen, and E = 2^-24:
      scores: products are exact, so a score's error is that of summing D of
        them in fp32, D E sum|q k| scale, and of a few roundings of numbers the
        size of the score and of its distance to the maximum; 2^x itself is
        within 2 E.  It changes a weight by that factor, the weights' sum too.
      weights: fp16, 2^-11 of each, or, where they are below fp16's normal
        range, 2^-25; the largest is held at 2^7 or more, so 2^-32 of the
        largest u;
      sums over n tokens in fp32: n E each, and a rounding per rescaling
        (at most one a block) and per join."""
    rows, hq, D = q.shape
    G = hq // cache.heads
    scale = D ** -0.5 if scale is None else scale
    out = np.zeros(q.shape)
    bound = np.zeros(q.shape)
    E = 2.0 ** -24
    for b in range(len(lengths)):
        row0, n, length = _sequence(cu, lengths, b, rows)
        if n == 0 or length == 0:
            continue
        nblk = -(-length // BLOCK)
        k, v = (np.full((cache.heads, nblk * BLOCK, D), np.nan) for _ in range(2))
        ev = np.zeros((cache.heads, nblk * BLOCK))
        for j in range(nblk):
            i = block_id(cache, table, b, j)
            if i < 0:
                continue
            span = slice(j * BLOCK, (j + 1) * BLOCK)
            for h in range(cache.heads):
                k[h, span] = VALUES[cache.block_codes(i, h, 0)] * 2.0 ** int(cache.exps[i, h, 0])
                v[h, span] = VALUES[cache.block_codes(i, h, 1)] * 2.0 ** int(cache.exps[i, h, 1])
                ev[h, span] = int(cache.exps[i, h, 1])
        for t in range(n):
            pos = length - n + t
            if pos < 0:
                continue
            lo = max(0, pos - window + 1) if window else 0
            for h in range(hq):
                kk, vv, ee = (x[h // G, lo:pos + 1] for x in (k, v, ev))
                with np.errstate(all="ignore"):
                    z = scale * (kk @ q[row0 + t, h])
                    w = np.exp(z - z.max())
                    p = w / w.sum()
                    o = p @ vv
                    size = scale * (np.abs(kk) @ np.abs(q[row0 + t, h]))
                    dz = D * E * size.max() + 8 * E * (np.abs(z).max() + np.abs(z - z.max()).max() + np.abs(ee).max() + 1)
                    u = p * 2.0 ** ee
                    seen = pos + 1 - lo
                    rel = 2 * dz + 2.0 ** -11 + (2 * seen + 64) * E
                    low = 2.0 ** -32 * u.max() * (np.abs(vv) * 2.0 ** -ee[:, None]).sum(0)
                    out[row0 + t, h] = o
                    bound[row0 + t, h] = rel * (p @ np.abs(vv)) * 1.01 + low + 1e-30
    return out, bound


# ------------------------------------------------------------------- norms
def add_rmsnorm(residual, weight, y=None, post=None, gate=None, scale=1.0, mod=None, eps=1e-5):
    """(r', x) in fp64; gate and mod [rows, C] with rows dividing M."""
    M = residual.shape[0]

    def spread(t):
        t = np.atleast_2d(t).astype(np.float64)
        return np.repeat(t, M // t.shape[0], axis=0)

    r = residual.astype(np.float64)
    if y is not None:
        u = y.astype(np.float64)
        if post is not None:
            u = u / np.sqrt((u * u).mean(1, keepdims=True) + eps) * post.astype(np.float64)
        if gate is not None:
            u = u * spread(gate)
        r = r + scale * u
    x = r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * weight.astype(np.float64)
    if mod is not None:
        x = x * (1.0 + spread(mod))
    return r, x


# ------------------------------------------------------------------ logits
def logits_adjust(z, history=None, cu=None, prompt=None, rho=None, frequency=None, presence=None, bias_ids=None,
                  bias=None, cu_bias=None, mask=None):
    """(out, size): fp64 [M, V] and the sum of the magnitudes that were added
    (what an fp32 evaluation's error is measured by)."""
    M, V = z.shape
    out = z.astype(np.float64).copy()
    size = np.abs(np.where(np.isfinite(out), out, 0.0))
    for m in range(M):
        seen, count = set(), {}
        if history is not None:
            lo = min(max(int(cu[m]), 0), len(history))
            hi = min(max(int(cu[m + 1]), lo), len(history))
            for i in range(lo, hi):
                t = int(history[i])
                if not 0 <= t < V:
                    continue
                seen.add(t)
                if i - lo >= (0 if prompt is None else int(prompt[m])):
                    count[t] = count.get(t, 0) + 1
        r = 1.0 if rho is None else float(rho[m])
        for t in seen:
            out[m, t] = out[m, t] / r if out[m, t] > 0 else out[m, t] * r
            size[m, t] = max(size[m, t], abs(out[m, t]) if np.isfinite(out[m, t]) else 0.0)
        for t, n in count.items():
            for x in ((float(frequency[m]) * n if frequency is not None else 0.0),
                      (float(presence[m]) if presence is not None else 0.0)):
                out[m, t] -= x
                size[m, t] += abs(x)
        if bias_ids is not None:
            lo = min(max(int(cu_bias[m]), 0), len(bias_ids))
            hi = min(max(int(cu_bias[m + 1]), lo), len(bias_ids))
            for i in range(lo, hi):
                t = int(bias_ids[i])
                if 0 <= t < V:
                    out[m, t] += float(bias[i])
                    size[m, t] += abs(float(bias[i]))
        if mask is not None:
            for t in range(V):
                if not (int(mask[m, t // 32]) >> (t % 32)) & 1:
                    out[m, t] = -np.inf
    return out, size
