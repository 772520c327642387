"""Plain CPU oracle for the operators of include/q4_search.h.

TEST INFRASTRUCTURE ONLY, like decoder_oracle, whose cache it uses: no code
shared with the HIP library or its binding.  NumPy and Python's whole numbers,
written from the definitions, one sequence, block or candidate at a time.
"""

from __future__ import annotations

import math

import numpy as np

from .decoder_oracle import BLOCK, VALUES, Cache, _sequence, block_id


# ------------------------------------------------------------- beam search
def beam_select(logits, scores, keep, finished=None, pad=0):
    """(parents, tokens, scores in 64 bits), each [groups, keep]."""
    groups, beams = scores.shape
    V = logits.shape[1]
    parents, tokens = (np.full((groups, keep), -1, dtype=np.int64) for _ in range(2))
    best = np.full((groups, keep), -np.inf)
    for g in range(groups):
        found = []
        for b in range(beams):
            base = float(scores[g, b])
            if finished is not None and finished[g, b]:
                if math.isfinite(base):
                    found.append((-base, b, pad))
                continue
            z = logits[g * beams + b].astype(np.float64)
            with np.errstate(all="ignore"):
                top = z.max()
                s = base + (z - (top + np.log(np.exp(z - top).sum())))
            at = np.flatnonzero(np.isfinite(s))
            if at.size > 4 * keep:     # those that can be among the first
                at = at[s[at] >= np.sort(s[at])[-keep]]
            found += [(-float(s[t]), b, int(t)) for t in at]
        for i, (s, b, t) in enumerate(sorted(found)[:keep]):
            parents[g, i], tokens[g, i], best[g, i] = g * beams + b, t, -s
    assert V >= 1
    return parents, tokens, best


def beam_advance(sequences, lengths, parents, tokens, finished=None, eos=-1, pad=0):
    rows, width = sequences.shape
    n = len(parents)
    out = np.full((n, width), pad, dtype=np.int64)
    out_lengths, out_finished = np.zeros(n, dtype=np.int64), np.ones(n, dtype=np.int64)
    for i, (p, t) in enumerate(zip(parents, tokens)):
        if not 0 <= p < rows:
            continue
        was = min(max(int(lengths[p]), 0), width)
        out[i, :was] = sequences[p, :was]
        out_lengths[i] = was
        if (finished is None or not finished[p]) and was < width:
            out[i, was] = t
            out_lengths[i] = was + 1
            out_finished[i] = eos >= 0 and t == eos
    return out, out_lengths, out_finished


# ------------------------------------------------------------------- pages
def _blocks_of(table, length, num_blocks):
    """The used entries of a table row."""
    n = min(max(int(length), 0), BLOCK * len(table))
    return n, [int(x) for x in table[:-(-n // BLOCK)]]


def kv_fork(table, lengths, parents, num_blocks, grow, held=None):
    """dict of block_table, lengths, refs, src, dst, short."""
    rows, width = table.shape
    n = len(parents)
    grow = [grow] * n if np.isscalar(grow) else list(grow)
    news = []
    for p, g in zip(parents, grow):
        was, ids = _blocks_of(table[p], lengths[p], num_blocks) if 0 <= p < rows else (0, [])
        news.append([was, max(0, int(g)) if 0 <= p < rows else 0, ids])
    refs = np.zeros(num_blocks, dtype=np.int64) if held is None else np.maximum(np.asarray(held, dtype=np.int64), 0)
    for _, _, ids in news:
        for x in ids:
            if 0 <= x < num_blocks:
                refs[x] += 1
    free = iter(np.flatnonzero(refs == 0).tolist())
    out = np.full((n, width), -1, dtype=np.int64)
    src, dst, short = np.full(n, -1), np.full(n, -1), np.zeros(n, dtype=np.int64)
    for i, (was, g, ids) in enumerate(news):
        if g > 0 and was % BLOCK and 0 <= ids[-1] < num_blocks and refs[ids[-1]] > 1:
            refs[ids[-1]] -= 1
            to = next(free, -1)
            if to >= 0:
                src[i], dst[i] = ids[-1], to
                refs[to] += 1
            else:
                short[i] += 1
            ids[-1] = to
        while len(ids) < -(-(was + g) // BLOCK):
            to = next(free, -1) if len(ids) < width else -1
            if to >= 0:
                refs[to] += 1
            else:
                short[i] += 1
            ids.append(to)
        out[i, :min(len(ids), width)] = ids[:width]
    return dict(block_table=out, lengths=np.array([w + g for w, g, _ in news], dtype=np.int64), refs=refs, src=src, dst=dst, short=short)


def kv_compact(table, lengths, num_blocks, held=None):
    """dict of block_table, src, dst, live."""
    used = [_blocks_of(t, n, num_blocks)[1] for t, n in zip(table, lengths)]
    pinned = set() if held is None else {i for i in range(num_blocks) if held[i] > 0}
    live = {x for ids in used for x in ids if 0 <= x < num_blocks} | pinned
    count = len(live)
    moves = sorted(x for x in live - pinned if x >= count)
    slots = [x for x in range(count) if x not in live]
    to = dict(zip(moves, slots))
    half = max(1, num_blocks // 2)
    src, dst = np.full(half, -1), np.full(half, -1)
    src[:len(moves)], dst[:len(moves)] = moves, slots[:len(moves)]
    out = np.full(table.shape, -1, dtype=np.int64)
    for row, ids in zip(out, used):
        row[:len(ids)] = [to.get(x, x) if 0 <= x < num_blocks else -1 for x in ids]
    return dict(block_table=out, src=src, dst=dst, live=np.array([count]))


# --------------------------------------------------------- selected blocks
def bounds(codes):
    """(hi, lo) [D] of the codes [tokens, D] of a block's tokens."""
    v = VALUES[codes]
    bad = np.isnan(v).any(0)
    with np.errstate(all="ignore"):
        hi, lo = np.ceil(np.where(bad, 0, v.max(0)) / 4), np.floor(np.where(bad, 0, v.min(0)) / 4)
    return np.where(bad, 127, hi).astype(np.int64), np.where(bad, -127, lo).astype(np.int64)


def summarize(cache: Cache, summary, table, lengths, rows, cu=None):
    """Into summary [blocks, heads, 2, D], for the blocks of the batch's rows."""
    for b in range(len(lengths)):
        _, n, length = _sequence(cu, lengths, b, rows)
        if n == 0 or length == 0:
            continue
        for j in range(max(0, length - n) // BLOCK, -(-length // BLOCK)):
            i = block_id(cache, table, b, j)
            if i < 0:
                continue
            for h in range(cache.heads):
                summary[i, h] = bounds(cache.block_codes(i, h, 0)[:length - j * BLOCK])


def select(cache: Cache, summary, q, table, lengths, keep, first, recent, cu=None, max_blocks=1 << 30):
    """chosen [rows, heads, keep]; q fp64 values of bf16 [rows, q_heads, D]."""
    rows, hq, D = q.shape
    group = hq // cache.heads
    out = np.full((rows, cache.heads, keep), -1, dtype=np.int64)
    for b in range(len(lengths)):
        row0, n, length = _sequence(cu, lengths, b, rows)
        for t in range(n):
            pos = length - n + t
            if pos < 0 or pos // BLOCK >= max_blocks:
                continue
            count = pos // BLOCK + 1
            for h in range(cache.heads):
                qq = q[row0 + t, h * group:(h + 1) * group]
                up, down = np.where(qq < 0, 0, qq).sum(0), np.where(qq > 0, 0, qq).sum(0)
                whole = np.zeros(2 * D, dtype=np.int64)
                if np.isfinite(qq).all() and max(up.max(), -down.min()) > 0:
                    e = math.frexp(max(up.max(), -down.min()))[1]
                    whole = np.rint(np.concatenate((up, down)) * 2.0 ** (13 - e)).astype(np.int64)
                order = []
                for j in range(count):
                    i = block_id(cache, table, b, j)
                    if j < first or j >= count - recent:
                        s = math.inf
                    elif i < 0:
                        s = -math.inf
                    else:
                        total = int(whole @ summary[i, h].astype(np.int64).reshape(-1))
                        s = float(np.float32(total)) * 2.0 ** int(cache.exps[i, h, 0])
                    order.append((-s, j))
                mine = sorted(j for _, j in sorted(order)[:keep])
                out[row0 + t, h, :len(mine)] = mine
    return out


def attention_blocks(cache: Cache, q, chosen, table, lengths, cu=None, scale=None):
    """(o, bound) in 64 bits, [rows, q_heads, D]: decoder_oracle.attention's
    formula and bound over the tokens of the chosen blocks, with one rounding more
    for every join of splits (at most 64) and the block's order."""
    rows, hq, D = q.shape
    group = hq // cache.heads
    scale = D ** -0.5 if scale is None else scale
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    E = 2.0 ** -24
    for b in range(len(lengths)):
        row0, n, length = _sequence(cu, lengths, b, rows)
        for t in range(n):
            pos = length - n + t
            if pos < 0:
                continue
            for h in range(cache.heads):
                ks, vs, es = [], [], []
                for j in chosen[row0 + t, h]:
                    if j < 0 or j > pos // BLOCK:
                        continue
                    i = block_id(cache, table, b, int(j))
                    m = min(BLOCK, pos + 1 - j * BLOCK)
                    if i < 0:
                        ks.append(np.full((m, D), np.nan))
                        vs.append(np.full((m, D), np.nan))
                        es.append(np.zeros(m))
                        continue
                    ek, ev = (int(cache.exps[i, h, x]) for x in (0, 1))
                    ks.append(VALUES[cache.block_codes(i, h, 0)[:m]] * 2.0 ** ek)
                    vs.append(VALUES[cache.block_codes(i, h, 1)[:m]] * 2.0 ** ev)
                    es.append(np.full(m, float(ev)))
                if not ks:
                    continue
                kk, vv, ee = (np.concatenate(x) for x in (ks, vs, es))
                for g in range(group):
                    at = row0 + t, h * group + g
                    with np.errstate(all="ignore"):
                        z = scale * (kk @ q[at])
                        w = np.exp(z - z.max())
                        p = w / w.sum()
                        size = abs(scale) * (np.abs(kk) @ np.abs(q[at]))
                        dz = D * E * size.max() + 8 * E * (np.abs(z).max() + np.abs(z - z.max()).max() + np.abs(ee).max() + 1)
                        u = p * 2.0 ** ee
                        rel = 2 * dz + 2.0 ** -11 + (2 * len(z) + 128) * E
                        low = 2.0 ** -32 * u.max() * (np.abs(vv) * 2.0 ** -ee[:, None]).sum(0)
                        out[at] = p @ vv
                        bound[at] = rel * (p @ np.abs(vv)) * 1.01 + low + 1e-30
    return out, bound
