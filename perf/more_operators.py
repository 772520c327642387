"""Beam search and very long contexts over the paged 8-bit cache, as cases to be timed and compared: the selection of
beams with the reordering of their tokens, the cache's pages (forked with their copies, compacted), and attention over
blocks that a cheap score selects for each query.

`run` computes a case in elementary torch operations in 32 bits (64 where values stand next to a border), or, where
`own` is set, through this package.

The cache: blocks of 32 tokens.  For a block, a kv head and K or V there are 32 * D codes (e4m3) and one int8 exponent
e; a value is code * 2^e.  Data plane [blocks][heads][K | V][32 * D], then the exponents [blocks][heads][2].  Within K:
[2][D / 64][4][16][16] = token / 16, d / 64, d / 16 % 4, token % 16, d % 16.  Within V: [D / 32][4][16][2][2][4] = d / 32,
token / 4 % 4, d % 16, d / 16 % 2, token / 16, token % 4.  A block's summary, int8 [blocks][heads][2][D], bounds its keys
from above and below, in units of 4 * 2^e.
"""

import math

import torch

own = False

BLOCK = 32          # tokens of a cache block
E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -32, 32
Q_BITS = 13         # a query's sums are held as integers of up to 2^13
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request with 4 beams, a short answer so far: latency
        {"name": "beam_1x4", "op": "beam", "groups": 1, "beams": 4, "keep": 4, "v": 131072, "length": 40, "room": 256,
         "first": False, "ended": 0.0, "masked": 0.0},
        # the first step of 7 requests, whose beams are alike but for the first, under a grammar; an odd vocabulary
        {"name": "beam_7x5_first", "op": "beam", "groups": 7, "beams": 5, "keep": 5, "v": 32003, "length": 1, "room": 100,
         "first": True, "ended": 0.0, "masked": 0.9},
        # 16 requests with 8 beams, twice as many candidates kept as beams, some beams finished, long answers
        {"name": "beam_16x8", "op": "beam", "groups": 16, "beams": 8, "keep": 16, "v": 131072, "length": 1500, "room": 4096,
         "first": False, "ended": 0.15, "masked": 0.0},
        # the pages of one request's 4 beams: after a prompt of some seconds of audio and a few tokens
        {"name": "fork_1x4", "op": "fork", "groups": 1, "beams": 4, "length": 205, "shared": 0.9, "layers": 8, "hkv": 8, "d": 128,
         "first": False, "ragged": False, "spare": 40},
        # 16 requests with 8 beams each, unequal lengths
        {"name": "fork_16x8", "op": "fork", "groups": 16, "beams": 8, "length": 1505, "shared": 0.85, "layers": 4, "hkv": 8, "d": 128,
         "first": False, "ragged": True, "spare": 300},
        # very long contexts: 262144 table entries, few of the layers' heads on this GPU
        {"name": "fork_16x4_131072", "op": "fork", "groups": 16, "beams": 4, "length": 131050, "shared": 0.98, "layers": 1, "hkv": 1,
         "d": 64, "first": False, "ragged": False, "spare": 2000},
        # a pool with holes after requests have ended, to be given back in part
        {"name": "compact_4096", "op": "compact", "blocks": 4096, "fill": 0.55, "sequences": 40, "layers": 1, "hkv": 8, "d": 128,
         "pinned": 0.0},
        # a large pool of small blocks, some of them held by a prefix store
        {"name": "compact_60000", "op": "compact", "blocks": 60000, "fill": 0.8, "sequences": 64, "layers": 1, "hkv": 1, "d": 64,
         "pinned": 0.02},
        # one stream with a long context: latency
        {"name": "sparse_1x32768", "op": "sparse", "batch": 1, "rows": 1, "length": 32768, "hq": 32, "hkv": 8, "d": 128, "keep": 64,
         "first": 1, "recent": 2, "ragged": False, "idle": 0},
        # the pair of a guided decode, each with a very long context
        {"name": "sparse_2x131072", "op": "sparse", "batch": 2, "rows": 1, "length": 131072, "hq": 32, "hkv": 8, "d": 128, "keep": 128,
         "first": 1, "recent": 4, "ragged": False, "idle": 0},
        # 32 concurrent sequences of unequal length, one slot idle
        {"name": "sparse_32x65536", "op": "sparse", "batch": 32, "rows": 1, "length": 65501, "hq": 32, "hkv": 8, "d": 128, "keep": 96,
         "first": 1, "recent": 2, "ragged": True, "idle": 1},
        # a chunk of a turn's new tokens behind a long context
        {"name": "sparse_chunk_61", "op": "sparse", "batch": 1, "rows": 61, "length": 30011, "hq": 24, "hkv": 8, "d": 64, "keep": 40,
         "first": 1, "recent": 3, "ragged": False, "idle": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("beam", "beam", "fork", "fork", "compact", "sparse", "sparse", "sparse"))
    if op == "beam":
        groups, beams = _log(rng, 1, 16), rng.randint(1, 8)
        return {"op": op, "groups": groups, "beams": beams, "keep": beams * rng.choice((1, 1, 2)), "v": _log(rng, 1000, 131072),
                "length": (n := _log(rng, 1, 1500)), "room": n + _log(rng, 1, 2500), "first": rng.random() < 0.2,
                "ended": rng.choice((0.0, 0.2)), "masked": rng.choice((0.0, 0.0, 0.7))}
    if op == "fork":
        groups, beams = _log(rng, 1, 16), rng.randint(2, 8)
        hkv, d, layers = rng.choice(((8, 128, 4), (8, 64, 3), (2, 128, 8), (1, 64, 2)))
        return {"op": op, "groups": groups, "beams": beams, "length": _log(rng, 2, 1505), "shared": rng.choice((0.5, 0.85, 1.0)),
                "layers": layers, "hkv": hkv, "d": d, "first": rng.random() < 0.25, "ragged": rng.random() < 0.6,
                "spare": groups * beams + _log(rng, 1, 200)}
    if op == "compact":
        hkv, d, most = rng.choice(((8, 128, 4096), (2, 128, 8000), (1, 64, 50000)))
        return {"op": op, "blocks": _log(rng, 50, most), "fill": rng.uniform(0.2, 0.9), "sequences": _log(rng, 1, 64), "layers": 1,
                "hkv": hkv, "d": d, "pinned": rng.choice((0.0, 0.03))}
    hq, hkv, d = rng.choice(((32, 8, 128), (32, 8, 128), (24, 8, 64), (16, 2, 128), (7, 1, 128), (20, 20, 64)))
    first, recent = rng.randint(0, 2), rng.randint(1, 4)
    keep = first + recent + _log(rng, 4, 90)
    if rng.random() < 0.7:     # single or few tokens
        batch, rows = _log(rng, 1, 32), rng.choice((1, 1, 1, 3))
        length = rows + _log(rng, 1, min(131072, 1000000 // batch))
    else:                      # chunks
        batch, rows = rng.choice((1, 1, 2)), _log(rng, 5, 61)
        keep = min(keep, 40)
        length = rows + _log(rng, 1, 30000)
    return {"op": op, "batch": batch, "rows": rows, "length": length, "hq": hq, "hkv": hkv, "d": d, "keep": keep, "first": first,
            "recent": recent, "ragged": rng.random() < 0.6, "idle": 1 if batch > 4 and rng.random() < 0.5 else 0}


def _sequences(case):
    """(rows, length) of each sequence of a sparse case: unequal ones fall from the case's size to a quarter of it; the
    idle slots of a batch have a row and nothing in the cache."""
    n = case["batch"]
    seqs = []
    for b in range(n):
        f = 1.0 - 0.75 * b / max(1, n - 1) if case["ragged"] else 1.0
        rows = max(1, int(case["rows"] * f))
        seqs.append((rows, rows + int((case["length"] - case["rows"]) * f)))
    for b in range(n - case["idle"], n):
        seqs[b] = (1, 0)
    return seqs


def _group_lengths(case):
    """Tokens of each group of beams: unequal ones fall to a third."""
    n = case["groups"]
    return [max(1, int(case["length"] * (1.0 - 0.67 * i / max(1, n - 1) if case["ragged"] else 1.0))) for i in range(n)]


def _fork_blocks(case):
    """For each group: blocks that all its beams share, and blocks of each beam.  Before the first step there is one beam."""
    beams = 1 if case["first"] else case["beams"]
    out = []
    for n in _group_lengths(case):
        blocks = -(-n // BLOCK)
        shared = min(blocks, int(blocks * case["shared"])) if beams > 1 else 0
        out.append((shared, blocks - shared, beams))
    return out


def _fork_pool(case):
    return sum(s + o * beams for s, o, beams in _fork_blocks(case)) + case["spare"]


def _block_bytes(case):
    return case["hkv"] * 2 * (BLOCK * case["d"] + 1)


def work(case):
    op = case["op"]
    if op == "beam":
        m, out = case["groups"] * case["beams"], case["groups"] * case["keep"]
        return {"bytes": 4 * m * case["v"] + 4 * out * (case["length"] + case["room"]), "flops": 4 * m * case["v"]}
    if op == "fork":
        n, entries, copies = case["beams"], 0, 0.0
        for length, (shared, mine, beams) in zip(_group_lengths(case), _fork_blocks(case)):
            entries += beams * (shared + mine) + n * (shared + mine)
            if length % BLOCK:     # all but one of a parent's children copy the block that they go on in
                copies += n - beams * (1.0 - (1.0 - 1.0 / beams) ** n)
        return {"bytes": int(4 * entries + 4 * _fork_pool(case) + 2 * copies * case["layers"] * _block_bytes(case)), "flops": entries}
    if op == "compact":
        live = case["blocks"] * case["fill"]
        moves = live * (1.0 - case["fill"])
        return {"bytes": int(8 * live + 4 * case["blocks"] + 2 * moves * case["layers"] * _block_bytes(case)), "flops": case["blocks"]}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    seqs = _sequences(case)
    rows = sum(r for r, _ in seqs)
    bytes_, flops = rows * hq * d * 4, 0
    for r, n in seqs:
        if n < r:
            continue
        blocks = -(-n // BLOCK)
        read = min(blocks, r * case["keep"])
        written = blocks - (n - r) // BLOCK
        bytes_ += blocks * hkv * (2 * d + 1) + read * hkv * (2 * BLOCK * d) + written * hkv * (BLOCK * d + 2 * d) + 4 * r * hkv * case["keep"]
        flops += r * (4 * blocks * hkv * d + 4 * min(blocks, case["keep"]) * BLOCK * hq * d)
    return {"bytes": bytes_, "flops": flops}


# ----------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within the range that is stored."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= E4M3_MAX / 512, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(EXP_MIN, EXP_MAX)


def _k_blocks(codes):
    """[..., tokens 32, d] -> the order of K's bytes in a block."""
    *lead, _, d = codes.shape
    n = len(lead)
    return codes.reshape(*lead, 2, 16, d // 64, 4, 16).permute(*range(n), n, n + 2, n + 3, n + 1, n + 4).reshape(*lead, 32 * d)


def _v_blocks(codes):
    """[..., tokens 32, d] -> the order of V's bytes in a block."""
    *lead, _, d = codes.shape
    n = len(lead)
    return codes.reshape(*lead, 2, 4, 4, d // 32, 2, 16).permute(*range(n), n + 3, n + 1, n + 5, n + 4, n, n + 2).reshape(*lead, 32 * d)


def _k_tokens(data):
    """K's bytes [..., 32 * d] -> [..., tokens 32, d]."""
    *lead, size = data.shape
    n, d = len(lead), size // BLOCK
    return data.reshape(*lead, 2, d // 64, 4, 16, 16).permute(*range(n), n, n + 3, n + 1, n + 2, n + 4).reshape(*lead, BLOCK, d)


def _v_tokens(data):
    """V's bytes [..., 32 * d] -> [..., tokens 32, d]."""
    *lead, size = data.shape
    n, d = len(lead), size // BLOCK
    return data.reshape(*lead, d // 32, 4, 16, 2, 2, 4).permute(*range(n), n + 4, n + 1, n + 5, n, n + 3, n + 2).reshape(*lead, BLOCK, d)


def _random_caches(layers, blocks, hkv, d, g):
    """Caches of all layers in one tensor [layers, bytes], filled with codes that are numbers."""
    plane = blocks * hkv * 2 * BLOCK * d
    size = -(-(plane + blocks * hkv * 2) // 16) * 16
    data = torch.randint(0, 256, (layers, size), dtype=torch.uint8, generator=g, device=DEV)
    codes = data[:, :plane]
    codes.masked_fill_((codes & 127) == 127, 0x38)
    data[:, plane:] = torch.randint(-8, 9, (layers, size - plane), dtype=torch.int8, generator=g, device=DEV).view(torch.uint8)
    return data


def _prepare_beam(case, g):
    groups, beams, v = case["groups"], case["beams"], case["v"]
    m = groups * beams
    s = {"logits": torch.randn((m, v), generator=g, device=DEV) * 3.0}
    s["scores"] = -torch.rand((groups, beams), generator=g, device=DEV) * 3.0 - 0.5 * case["length"] ** 0.5
    lengths = torch.full((m,), case["length"], dtype=torch.int32, device=DEV)
    finished = (torch.rand((groups, beams), generator=g, device=DEV) < case["ended"]).int()
    if case["first"]:            # the beams are alike: the first one alone counts
        s["logits"] = s["logits"].view(groups, beams, v)[:, :1].expand(-1, beams, -1).reshape(m, v).contiguous()
        s["scores"][:, 0] = 0.0
        s["scores"][:, 1:] = -math.inf
    if case["masked"]:           # a grammar's tokens, among them at least 64 that are allowed
        allow = torch.rand((m, v), generator=g, device=DEV) >= case["masked"]
        allow[:, torch.randperm(v, generator=g, device=DEV)[:64]] = True
        s["logits"].masked_fill_(~allow, -math.inf)
    # finished beams ended earlier
    cut = (torch.rand(m, generator=g, device=DEV) * case["length"]).int()
    s["lengths"] = torch.where(finished.view(-1) != 0, torch.maximum(cut, torch.ones_like(cut)), lengths)
    s["finished"] = finished
    s["sequences"] = torch.randint(0, v, (m, case["room"]), dtype=torch.int32, generator=g, device=DEV)
    s["eos"], s["pad"] = 2, 0
    return s


def _prepare_fork(case, g):
    """Tables of groups of beams: a group's first blocks are shared, the rest each beam's own; ids in no order, the table
    wider than the longest sequence."""
    parts, lengths, pool = _fork_blocks(case), _group_lengths(case), _fork_pool(case)
    ids = torch.randperm(pool, generator=g, device=DEV).int()
    width = max(a + b for a, b, _ in parts) + 2
    rows, at = [], 0
    for shared, mine, beams in parts:
        t = torch.full((beams, width), -1, dtype=torch.int32, device=DEV)
        t[:, :shared] = ids[at:at + shared]
        at += shared
        t[:, shared:shared + mine] = ids[at:at + mine * beams].view(beams, mine)
        at += mine * beams
        rows.append(t)
    beams = parts[0][2]
    s = {"table": torch.cat(rows), "blocks": pool}
    s["lengths"] = torch.tensor([n for n in lengths for _ in range(beams)], dtype=torch.int32, device=DEV)
    group = torch.arange(case["groups"], device=DEV)[:, None] * beams
    s["parents"] = (group + torch.randint(0, beams, (case["groups"], case["beams"]), generator=g, device=DEV)).int()
    s["caches"] = _random_caches(case["layers"], pool, case["hkv"], case["d"], g)
    return s


def _prepare_compact(case, g):
    blocks, n = case["blocks"], case["sequences"]
    pinned = int(blocks * case["pinned"])
    live = max(1, int(blocks * case["fill"]) - pinned)
    ids = torch.randperm(blocks, generator=g, device=DEV).int()
    # the sequences' shares of the live blocks, from long to short
    cut = [int(live * (1.0 - (1.0 - i / n) ** 1.5)) for i in range(n + 1)]
    width = max(1, max(b - a for a, b in zip(cut, cut[1:]))) + 1
    table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    for i, (a, b) in enumerate(zip(cut, cut[1:])):
        table[i, :b - a] = ids[a:b]
    lengths = torch.tensor([(b - a) * BLOCK - (i % BLOCK if b > a else 0) for i, (a, b) in enumerate(zip(cut, cut[1:]))],
                           dtype=torch.int32, device=DEV)
    held = torch.zeros(blocks, dtype=torch.int32, device=DEV)
    held[ids[live:live + pinned].long()] = 1
    return {"table": table, "lengths": lengths, "blocks": blocks, "held": held if pinned else None,
            "caches": _random_caches(case["layers"], blocks, case["hkv"], case["d"], g)}


def _bounds(codes, valid):
    """Summary of blocks: K's values [..., tokens 32, d] -> [..., 2, d] int8, over the tokens that count."""
    hi = torch.where(valid, codes, -math.inf).amax(-2)
    lo = torch.where(valid, codes, math.inf).amin(-2)
    return torch.stack((torch.ceil(hi / 4), torch.floor(lo / 4)), -2).to(torch.int8)


def _prepare_sparse(case, g):
    """A filled cache with its summaries, all but those of the blocks that the call's rows are in, its block table, lengths
    and row bounds: blocks in no order, a table wider than the longest sequence."""
    hkv, d = case["hkv"], case["d"]
    seqs = _sequences(case)
    need = [-(-n // BLOCK) for _, n in seqs]
    nb = max(1, sum(need))
    order = torch.randperm(nb, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.full((len(seqs), max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = torch.empty(nb * hkv * 2 * (BLOCK * d + 1), dtype=torch.uint8, device=DEV)
    data = cache[:nb * hkv * 2 * BLOCK * d].view(nb, hkv, 2, BLOCK * d)
    exps = cache[nb * hkv * 2 * BLOCK * d:].view(torch.int8).view(nb, hkv, 2)
    summary = torch.empty((nb, hkv, 2, d), dtype=torch.int8, device=DEV)
    tilt = torch.exp(0.6 * torch.randn((2, hkv, 1, d), generator=g, device=DEV))      # some channels are larger
    step = max(1, (1 << 27) // (hkv * 2 * BLOCK * d))
    for i in range(0, nb, step):
        n = min(step, nb - i)
        for kv, blocks in ((0, _k_blocks), (1, _v_blocks)):
            # a block's tokens are near each other, so that some blocks matter more to a query
            x = torch.randn((n, hkv, BLOCK, d), generator=g, device=DEV) * 0.8 + torch.randn((n, hkv, 1, d), generator=g, device=DEV) * 0.6
            x *= tilt[kv]
            e = _exponent(x.abs().amax((2, 3)))
            codes = torch.ldexp(x, -e[:, :, None, None]).to(E4M3)
            data[i:i + n, :, kv] = blocks(codes.view(torch.uint8))
            exps[i:i + n, :, kv] = e.to(torch.int8)
            if kv == 0:
                summary[i:i + n] = _bounds(codes.float(), torch.ones((BLOCK, 1), dtype=torch.bool, device=DEV))
    cu = [0]
    for r, _ in seqs:
        cu.append(cu[-1] + r)
    # the scheduler's list of the blocks that the rows are in, with how many of their tokens there are
    touched = [(int(table[b, j]), min(BLOCK, n - j * BLOCK)) for b, (r, n) in enumerate(seqs) if n >= r
               for j in range((n - r) // BLOCK, -(-n // BLOCK))]
    blocks, counts = (torch.tensor(x, device=DEV) for x in zip(*touched))
    summary[blocks] = 0
    uneven = len({r for r, _ in seqs}) > 1
    return {"cache": cache, "blocks": nb, "table": table.to(DEV), "summary": summary, "touched": blocks, "counts": counts,
            "lengths": torch.tensor([n for _, n in seqs], dtype=torch.int32, device=DEV),
            "cu": torch.tensor(cu, dtype=torch.int32, device=DEV) if uneven else None,
            "rows": cu[-1], "max_rows": max(r for r, _ in seqs), "max_length": max(n for _, n in seqs),
            "q": torch.randn((cu[-1], case["hq"] * d), generator=g, device=DEV).bfloat16()}


def prepare(case, seed):
    make = {"beam": _prepare_beam, "fork": _prepare_fork, "compact": _prepare_compact, "sparse": _prepare_sparse}[case["op"]]
    return {"case": case, **make(case, _generator(seed))}


# ------------------------------------------------------------ plain forms
def _beam(s):
    c = s["case"]
    groups, beams, keep, v = c["groups"], c["beams"], c["keep"], c["v"]
    z = s["logits"].double()
    # scores stand next to each other: 64 bits
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    n = min(keep, v)
    # each beam's largest logits, of equal ones the first: a key of the value's order and the place
    bits = s["logits"].add(0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits)
    key = order * 2 ** 24 + (2 ** 24 - 1 - torch.arange(v, device=DEV))
    token = 2 ** 24 - 1 - (torch.topk(key, n, 1).values & (2 ** 24 - 1))
    score = s["scores"].double().view(-1, 1) + (torch.gather(z, 1, token) - lse)
    ended = s["finished"].view(-1, 1) != 0
    place = torch.arange(n, device=DEV)
    score = torch.where(ended, torch.where(place == 0, s["scores"].double().view(-1, 1), -math.inf), score)
    token = torch.where(ended, s["pad"], token)
    score = torch.where(torch.isfinite(score), score, -math.inf).view(groups, beams * n)
    if beams * n < keep:
        score = torch.cat((score, torch.full((groups, keep - beams * n), -math.inf, dtype=torch.float64, device=DEV)), 1)
    best, at = torch.sort(score, dim=1, descending=True, stable=True)
    best, at = best[:, :keep], at[:, :keep].clamp(max=beams * n - 1)
    some = best > -math.inf
    row = torch.arange(groups, device=DEV)[:, None] * beams + at // n
    parents = torch.where(some, row, -1)
    tokens = torch.where(some, torch.gather(token.view(groups, beams * n), 1, at), -1)
    # the tokens so far, and this one
    p, t = parents.view(-1), tokens.view(-1)
    live, p = p >= 0, p.clamp(min=0)
    room = c["room"]
    was, done = s["lengths"].long()[p], s["finished"].view(-1)[p] != 0
    adds = live & ~done & (was < room)
    length = torch.where(live, was + adds, 0)
    place = torch.arange(room, device=DEV)
    seq = torch.where(place < torch.where(live, was, 0)[:, None], s["sequences"][p], s["pad"])
    seq = torch.where(adds[:, None] & (place == was[:, None]), t[:, None].int(), seq)
    done = ~live | done | ~adds | (t == s["eos"])
    return {"parents": parents.int(), "tokens": tokens.int(), "scores": best.float(), "sequences": seq, "lengths": length.int(),
            "finished": done.int()}


def _planes(caches, blocks, hkv, d):
    """(codes [layers, blocks, heads, 2, 32 * d], exponents [layers, blocks, heads, 2]) of caches in one tensor."""
    n = blocks * hkv * 2 * BLOCK * d
    layers = caches.shape[0]
    return (caches[:, :n].unflatten(1, (blocks, hkv, 2, BLOCK * d)),
            caches[:, n:n + blocks * hkv * 2].view(torch.int8).unflatten(1, (blocks, hkv, 2)))


def _copy_blocks(s, src, dst):
    """Copies blocks in every layer.  Places without a copy do one of the others again."""
    c = s["case"]
    some = src >= 0
    one = some.int().argmax()
    src = torch.where(some, src, src[one].clamp(min=0)).long()
    dst = torch.where(some, dst, dst[one].clamp(min=0)).long()
    codes, exps = _planes(s["caches"], s["blocks"], c["hkv"], c["d"])
    codes[:, dst] = codes[:, src]
    exps[:, dst] = exps[:, src]


def _caches_out(s):
    codes, exps = _planes(s["caches"], s["blocks"], s["case"]["hkv"], s["case"]["d"])
    return {"codes": codes.view(E4M3), "exponents": exps}


def _fork(s):
    blocks, (_, width) = s["blocks"], s["table"].shape
    parents = s["parents"].view(-1).long()
    was = s["lengths"].long()[parents]
    table = s["table"][parents]
    n = parents.shape[0]
    place = torch.arange(width, device=DEV)
    have = (was + BLOCK - 1) // BLOCK
    table = torch.where(place < have[:, None], table, -1)
    flat = torch.where(table >= 0, table, blocks).view(-1).long()
    refs = torch.zeros(blocks + 1, dtype=torch.int64, device=DEV).index_add_(0, flat, torch.ones_like(flat))
    refs[blocks] = 0
    # a row's last block where it is partly filled: rows before it that go on in the same block have left it
    part = was % BLOCK != 0
    last = torch.where(part, table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0].long(), -1)
    row = torch.arange(n, device=DEV)
    before = ((last[:, None] == last) & (row < row[:, None])).sum(1)
    copies = part & (refs[last.clamp(min=0)] - before > 1)
    fresh = (was % BLOCK == 0).long()                    # one new token
    want = copies.long() + fresh
    upto = want.cumsum(0)
    free = refs[:blocks] == 0
    rank = free.long().cumsum(0) - 1
    ids = torch.full((blocks + 1,), -1, dtype=torch.int64, device=DEV)
    ids[torch.where(free, rank, blocks)] = torch.arange(blocks, device=DEV)
    ids[blocks] = -1
    got = torch.where(want > 0, ids[(upto - want).clamp(max=blocks)], -1)
    src, dst = torch.where(copies & (got >= 0), last, -1), torch.where(copies, got, -1)
    at = torch.where(copies, have - 1, have)
    table = torch.where((want > 0)[:, None] & (place == at[:, None]), got[:, None].int(), table)
    refs = refs.index_add(0, last.clamp(min=0), -copies.long())
    refs = refs.index_add(0, torch.where(got >= 0, got, blocks), torch.ones_like(got))[:blocks]
    short = torch.where((want > 0) & (got < 0), 1, 0)
    _copy_blocks(s, src, dst)
    return {"table": table, "lengths": (was + 1).int(), "refs": refs.int(), "src": src.int(), "dst": dst.int(),
            "short": short.int(), **_caches_out(s)}


def _compact(s):
    blocks, (_, width) = s["blocks"], s["table"].shape
    have = (s["lengths"].long() + BLOCK - 1) // BLOCK
    used = torch.arange(width, device=DEV) < have[:, None]
    flat = torch.where(used & (s["table"] >= 0), s["table"], blocks).view(-1).long()
    live = torch.zeros(blocks + 1, dtype=torch.int64, device=DEV)
    live[flat] = 1
    live = live[:blocks]
    pinned = s["held"] > 0 if s["held"] is not None else torch.zeros(blocks, dtype=torch.bool, device=DEV)
    live = torch.where(pinned, 1, live)
    count = live.sum()
    ids = torch.arange(blocks, device=DEV)
    moves = (live > 0) & ~pinned & (ids >= count)
    slots = (live == 0) & (ids < count)
    half = max(1, blocks // 2)
    src, dst = torch.full((blocks + 1,), -1, dtype=torch.int64, device=DEV), torch.full((blocks + 1,), -1, dtype=torch.int64, device=DEV)
    src[torch.where(moves, moves.long().cumsum(0) - 1, blocks)] = ids
    dst[torch.where(slots, slots.long().cumsum(0) - 1, blocks)] = ids
    src, dst = src[:half], dst[:half]
    dst = torch.where(src >= 0, dst, -1)
    to = torch.cat((ids, ids[:1]))
    to[torch.where(src >= 0, src, blocks)] = dst
    table = torch.where(used & (s["table"] >= 0), to[s["table"].clamp(min=0).long()].int(), -1)
    _copy_blocks(s, src, dst)
    return {"table": table, "src": src.int(), "dst": dst.int(), "live": count.int().view(1), **_caches_out(s)}


def _rows_of(s):
    """For every row: its sequence, its place among that sequence's rows, and its position (negative: none)."""
    n = s["lengths"].shape[0]
    row = torch.arange(s["rows"], device=DEV)
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(n + 1, device=DEV) * (s["rows"] // n)
    b = torch.searchsorted(cu, row, right=True) - 1
    t = row - cu[b]
    return b, t, s["lengths"].long()[b] - (cu[b + 1] - cu[b]) + t


def _sparse(s):
    c = s["case"]
    hq, hkv, d, keep = c["hq"], c["hkv"], c["d"], c["keep"]
    group = hq // hkv
    n = s["blocks"] * hkv * 2 * BLOCK * d
    data, exps = s["cache"][:n].view(s["blocks"], hkv, 2, BLOCK * d), s["cache"][n:].view(torch.int8).view(s["blocks"], hkv, 2)
    # the summaries of the rows' blocks
    codes = _k_tokens(data[s["touched"], :, 0]).view(E4M3).float()
    valid = torch.arange(BLOCK, device=DEV)[:, None] < s["counts"][:, None, None, None]
    s["summary"][s["touched"]] = _bounds(codes, valid)
    # the group's queries in integers of one power of two
    b, t, pos = _rows_of(s)
    rows = s["rows"]
    q = s["q"].double().view(rows, hkv, group, d)
    both = torch.stack((q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)), 2)
    e = torch.frexp(both.abs().amax((2, 3)))[1]
    whole = torch.round(torch.ldexp(both, (Q_BITS - e)[:, :, None, None])).view(rows, hkv, 2 * d)
    # every block's score for every row: whole numbers below 2^28, exact in 64 bits
    nblk = -(-s["max_length"] // BLOCK)
    ids = s["table"][:, :nblk].long()
    known = ids >= 0
    ids = ids.clamp(min=0)
    most, batch = s["max_rows"], s["lengths"].shape[0]
    wide = torch.zeros((batch, most, hkv, 2 * d), dtype=torch.float64, device=DEV)
    wide[b, t] = whole
    kk = s["summary"][ids].view(batch, nblk, hkv, 2 * d).permute(0, 2, 3, 1).double().contiguous()
    score = torch.matmul(wide.permute(0, 2, 1, 3).contiguous(), kk).permute(0, 2, 1, 3)[b, t].float()
    score = torch.ldexp(score, exps[ids][..., 0].permute(0, 2, 1)[b].int())
    score = torch.where(known[b][:, None], score, -math.inf)
    block = torch.arange(nblk, device=DEV)
    count = torch.where(pos >= 0, pos // BLOCK + 1, 0)[:, None, None]
    score = torch.where((block < c["first"]) | (block >= count - c["recent"]), math.inf, score)
    # those past the row come last, in their order
    score = torch.where(block < count, score.double(), -math.inf)
    late = (block >= count).expand(score.shape)
    bits = score.float().add(0.0).view(torch.int32).long()
    order = torch.where(late, -2 ** 32, torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits))
    key = order * 2 ** 24 + (2 ** 24 - 1 - block)
    m = min(keep, nblk)
    chosen = 2 ** 24 - 1 - (torch.topk(key, m, -1).values & (2 ** 24 - 1))
    chosen = torch.where(chosen < count, chosen, 2 ** 24).sort(-1).values
    if m < keep:
        chosen = torch.cat((chosen, torch.full((rows, hkv, keep - m), 2 ** 24, device=DEV)), -1)
    chosen = torch.where(chosen < 2 ** 24, chosen, -1)
    # attention over them
    blk = chosen.clamp(min=0)
    got = s["table"].long()[b][:, None].expand(-1, hkv, -1).gather(2, blk).clamp(min=0)
    head = torch.arange(hkv, device=DEV)[:, None]
    k = _k_tokens(data[got, head, 0]).view(E4M3).float() * torch.exp2(exps[got, head, 0].float())[..., None, None]
    v = _v_tokens(data[got, head, 1]).view(E4M3).float() * torch.exp2(exps[got, head, 1].float())[..., None, None]
    token = blk[..., None] * BLOCK + torch.arange(BLOCK, device=DEV)
    sees = ((token <= pos[:, None, None, None]) & (chosen >= 0)[..., None]).view(rows, hkv, keep * BLOCK, 1)
    k, v = k.view(rows, hkv, keep * BLOCK, d), v.view(rows, hkv, keep * BLOCK, d)
    k, v = torch.where(sees, k, 0.0), torch.where(sees, v, 0.0)
    sees = sees.transpose(2, 3)
    z = torch.matmul(s["q"].float().view(rows, hkv, group, d), k.transpose(2, 3).contiguous()) * d ** -0.5
    z = torch.where(sees, z, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.where(sees, torch.exp(z - torch.where(top == -math.inf, 0.0, top)), 0.0)
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, torch.matmul(p, v) / total, 0.0)
    return {"summary": s["summary"], "chosen": chosen.int(), "out": o.reshape(rows, hq * d).bfloat16()}


def run(s):
    c = s["case"]
    if not own:
        return {"beam": _beam, "fork": _fork, "compact": _compact, "sparse": _sparse}[c["op"]](s)
    import q4_weight_only_amd as q4

    if c["op"] == "beam":
        parents, tokens, scores = q4.beam_select(s["logits"], s["scores"], c["keep"], finished=s["finished"], pad=s["pad"])
        seq, lengths, finished = q4.beam_advance(s["sequences"], s["lengths"], parents, tokens, finished=s["finished"],
                                                 eos=s["eos"], pad=s["pad"])
        return {"parents": parents, "tokens": tokens, "scores": scores, "sequences": seq, "lengths": lengths, "finished": finished}
    if c["op"] == "sparse":
        cache = q4.KVCache(s["cache"], s["blocks"], c["hkv"], c["d"])
        q4.kv_summarize(cache, s["summary"], s["table"], s["lengths"], s["cu"], rows=s["rows"], max_rows=s["max_rows"])
        chosen = q4.kv_select(s["q"], cache, s["summary"], s["table"], s["lengths"], s["cu"], keep=c["keep"], first=c["first"],
                              recent=c["recent"], max_rows=s["max_rows"], max_length=s["max_length"])
        out = q4.kv_attention_blocks(s["q"], cache, chosen, s["table"], s["lengths"], s["cu"], max_rows=s["max_rows"])
        return {"summary": s["summary"], "chosen": chosen, "out": out}
    stack = q4.KVStack(s["caches"], s["blocks"], c["hkv"], c["d"])
    if c["op"] == "fork":
        f = q4.kv_fork(s["table"], s["lengths"], s["parents"], s["blocks"], grow=1)
        q4.kv_copy_blocks(stack, f.src, f.dst)
        return {"table": f.block_table, "lengths": f.lengths, "refs": f.refs, "src": f.src, "dst": f.dst, "short": f.short,
                **_caches_out(s)}
    f = q4.kv_compact(s["table"], s["lengths"], s["blocks"], held=s["held"])
    q4.kv_copy_blocks(stack, f.src, f.dst)
    return {"table": f.block_table, "src": f.src, "dst": f.dst, "live": f.live, **_caches_out(s)}


# ------------------------------------------------------- 64-bit definition
def _numbers(codes):
    """e4m3 bytes as float64, from the format: sign, 4 exponent bits of bias 7, 3 fraction bits; all ones is no number."""
    c = codes.long()
    exp, frac = (c >> 3) & 15, (c & 7).double()
    v = torch.where(exp > 0, (1 + frac / 8) * torch.exp2((exp - 7).double()), frac / 8 * 2.0 ** -6)
    v = torch.where((c & 127) == 127, math.nan, v)
    return torch.where(c >= 128, -v, v)


def _index(d, slot):
    """Where the d values of a token at `slot` of a block are among K's and V's bytes."""
    i = torch.arange(d, device=DEV)
    k = ((((slot // 16) * (d // 64) + i // 64) * 4 + i // 16 % 4) * 16 + slot % 16) * 16 + i % 16
    v = ((((i // 32 * 4 + slot // 4 % 4) * 16 + i % 16) * 2 + i // 16 % 2) * 2 + slot // 16) * 4 + slot % 4
    return k, v


def _exact_beam(s, case):
    groups, beams, keep = case["groups"], case["beams"], case["keep"]
    scores = torch.full((groups, keep), -math.inf, dtype=torch.float64, device=DEV)
    for i in range(groups):
        found = []
        for b in range(beams):
            base = float(s["scores"][i, b])
            z = s["logits"][i * beams + b].double()
            if int(s["finished"][i, b]):
                found += [base]
            else:
                p = torch.log_softmax(z, 0).sort(descending=True).values[:keep] + base
                found += p.tolist()
        found = sorted((x for x in found if math.isfinite(x)), reverse=True)[:keep]
        scores[i, :len(found)] = torch.tensor(found, dtype=torch.float64, device=DEV)
    return {"parents": None, "tokens": None, "scores": scores, "sequences": None, "lengths": None, "finished": None}


def _exact_fork(s, case):
    codes = _numbers(_planes(s["caches"], s["blocks"], case["hkv"], case["d"])[0]).clone()
    parents, lengths, table = s["parents"].view(-1).tolist(), s["lengths"].tolist(), s["table"].cpu()
    holders = {}
    rows = [table[p, :-(-lengths[p] // BLOCK)].tolist() for p in parents]
    for r in rows:
        for x in r:
            holders[x] = holders.get(x, 0) + 1
    free = iter(x for x in range(s["blocks"]) if x not in holders)
    for p, r in zip(parents, rows):
        if lengths[p] % BLOCK == 0:
            next(free, None)
        elif holders[r[-1]] > 1:
            to = next(free, None)
            if to is not None:
                holders[r[-1]] -= 1
                codes[:, to] = codes[:, r[-1]]
    return {"table": None, "lengths": None, "refs": None, "src": None, "dst": None, "short": None, "codes": codes, "exponents": None}


def _exact_compact(s, case):
    codes = _numbers(_planes(s["caches"], s["blocks"], case["hkv"], case["d"])[0]).clone()
    live, held = set(), set()
    if s["held"] is not None:
        held = set(torch.nonzero(s["held"])[:, 0].tolist())
    for r, n in zip(s["table"].cpu(), s["lengths"].tolist()):
        live |= set(r[:-(-n // BLOCK)].tolist())
    live |= held
    count = len(live)
    src = sorted(x for x in live - held if x >= count)
    dst = [x for x in range(count) if x not in live][:len(src)]
    if src:
        codes[:, torch.tensor(dst, device=DEV)] = codes[:, torch.tensor(src, device=DEV)]
    return {"table": None, "src": None, "dst": None, "live": None, "codes": codes, "exponents": None}


def _exact_sparse(s, case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    group = hq // hkv
    n = s["blocks"] * hkv * 2 * BLOCK * d
    data, exps = s["cache"][:n].view(-1, hkv, 2, BLOCK * d), s["cache"][n:].view(torch.int8).view(-1, hkv, 2)
    table = s["table"].long()
    out = torch.zeros((s["rows"], hkv, group, d), dtype=torch.float64, device=DEV)
    where = _index(d, torch.arange(BLOCK, device=DEV)[:, None])
    row = 0
    for b, (r, length) in enumerate(_sequences(case)):
        if length < r:
            row += r
            continue
        count = -(-length // BLOCK)
        ids = table[b, :count]
        for h in range(hkv):
            # bounds of the keys, from the codes themselves
            kn = _numbers(data[ids, h, 0][:, where[0]])
            there = torch.arange(count * BLOCK, device=DEV).view(count, BLOCK, 1) < length
            hi = torch.ceil(torch.where(there, kn, -math.inf).amax(1) / 4)
            lo = torch.floor(torch.where(there, kn, math.inf).amin(1) / 4)
            scale = torch.exp2(exps[ids, h, 0].double())
            for t in range(r):
                pos = length - r + t
                mine = pos // BLOCK + 1
                q = s["q"][row + t].double().view(hkv, group, d)[h]
                up, down = q.clamp(min=0).sum(0), q.clamp(max=0).sum(0)
                e = math.frexp(float(torch.maximum(up, -down).max()))[1]
                up, down = (torch.round(x * 2.0 ** (Q_BITS - e)) for x in (up, down))
                score = ((hi[:mine] * up).sum(1) + (lo[:mine] * down).sum(1)).float().double() * scale[:mine]
                score[:case["first"]] = math.inf
                score[max(0, mine - case["recent"]):] = math.inf
                keep = score.sort(descending=True, stable=True).indices[:case["keep"]].sort().values
                at = ids[keep]
                k = kn[keep] * scale[keep][:, None, None]
                v = _numbers(data[at, h, 1][:, where[1]]) * torch.exp2(exps[at, h, 1].double())[:, None, None]
                sees = (keep[:, None] * BLOCK + torch.arange(BLOCK, device=DEV) <= pos).view(-1)
                k, v = k.view(-1, d)[sees], v.view(-1, d)[sees]
                out[row + t, h] = torch.softmax(q @ k.T / math.sqrt(d), -1) @ v
        row += r
    return {"summary": None, "chosen": None, "out": out.view(s["rows"], hq * d)}


def exact(case, seed):
    make = {"beam": _exact_beam, "fork": _exact_fork, "compact": _exact_compact, "sparse": _exact_sparse}[case["op"]]
    return make(prepare(case, seed), case)
