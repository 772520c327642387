"""The decoder operators between the 4-bit linears, as cases to be timed and compared: appending rotated keys and values
to the paged 8-bit cache, attention over that cache, the fused norms around a block, and the adjustment of the logits.

`run` computes a case in elementary torch operations in 32 bits, or, where `own` is set, through this package.

The cache: blocks of 32 tokens.  For a block, a kv head and K or V there are 32 * D codes (e4m3) and one int8 exponent
e; a value is code * 2^e.  Data plane [blocks][heads][K | V][32 * D], then the exponents [blocks][heads][2].  Within K:
[2][D / 64][4][16][16] = token / 16, d / 64, d / 16 % 4, token % 16, d % 16.  Within V: [D / 32][4][16][2][2][4] = d / 32,
token / 4 % 4, d % 16, d / 16 % 2, token / 16, token % 4.
"""

import math

import torch

own = False

BLOCK = 32          # tokens of a cache block
E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -32, 32
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one stream, 120 s of audio at 12.5 frames a second in the cache, one new token: latency
        {"name": "attention_1x1505", "op": "attention", "batch": 1, "rows": 1, "length": 1505, "hq": 32, "hkv": 8, "d": 128,
         "window": 0, "ragged": False, "idle": 0},
        # 32 concurrent sequences of unequal length, one of the batch's slots idle
        {"name": "attention_32x8192", "op": "attention", "batch": 32, "rows": 1, "length": 8191, "hq": 32, "hkv": 8, "d": 128,
         "window": 0, "ragged": True, "idle": 1},
        # the pair of a guided decode, each with a very long context
        {"name": "attention_2x131072", "op": "attention", "batch": 2, "rows": 1, "length": 131072, "hq": 32, "hkv": 8,
         "d": 128, "window": 0, "ragged": False, "idle": 0},
        # a prompt of 2048 tokens
        {"name": "attention_prompt_2048", "op": "attention", "batch": 1, "rows": 2048, "length": 2048, "hq": 32, "hkv": 8,
         "d": 128, "window": 0, "ragged": False, "idle": 0},
        # one chunk of an audio encoder's rows: a window of 750, as many kv heads as heads, the rest of 6020 rows before it
        {"name": "attention_window_1505", "op": "attention", "batch": 1, "rows": 1505, "length": 6020, "hq": 20, "hkv": 20,
         "d": 64, "window": 750, "ragged": False, "idle": 0},
        # one new token for each of 32 sequences, one slot idle
        {"name": "append_32", "op": "append", "batch": 32, "rows": 1, "length": 411, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "ragged": True, "idle": 1},
        # prompts of unequal length, started inside a block (the sequences' first tokens are in the cache already)
        {"name": "append_prompts_3x1505", "op": "append", "batch": 3, "rows": 1505, "length": 1517, "hq": 32, "hkv": 8,
         "d": 128, "rot": 128, "interleaved": True, "ragged": True, "idle": 0},
        # around the attention of a decode step of a guided pair: residual add and norm
        {"name": "norm_2x3072", "op": "norm", "m": 2, "c": 3072, "post": False, "gate": 0, "mod": 0, "res_bf16": False,
         "y_bf16": False, "out_bf16": True},
        # a prompt through the same place with everything on: norm after the block, gate, modulation
        {"name": "norm_2048x3072", "op": "norm", "m": 2048, "c": 3072, "post": True, "gate": 1, "mod": 1, "res_bf16": False,
         "y_bf16": False, "out_bf16": True},
        # an audio encoder's rows with a bf16 residual stream
        {"name": "norm_6020x1280", "op": "norm", "m": 6020, "c": 1280, "post": False, "gate": 0, "mod": 0, "res_bf16": True,
         "y_bf16": False, "out_bf16": True},
        # one sequence's logits
        {"name": "logits_1", "op": "logits", "m": 1, "v": 131072, "history": 200, "bias": 16, "mask": True},
        # 32 concurrent sequences with longer histories
        {"name": "logits_32", "op": "logits", "m": 32, "v": 131072, "history": 4099, "bias": 300, "mask": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attention", "attention", "attention", "append", "append", "norm", "logits"))
    if op in ("attention", "append"):
        hq, hkv, d = rng.choice(((32, 8, 128), (32, 8, 128), (20, 20, 64), (16, 2, 128), (24, 8, 64), (7, 1, 128)))
        if op == "append":
            prompt = rng.random() < 0.5
            batch = _log(rng, 1, 6) if prompt else _log(rng, 1, 64)
            rows = _log(rng, 5, 1505) if prompt else rng.choice((1, 1, 2, 4))
            return {"op": op, "batch": batch, "rows": rows, "length": rows + _log(rng, 1, 500), "hq": hq, "hkv": hkv, "d": d,
                    "rot": rng.choice((d, d, d // 2)), "interleaved": rng.random() < 0.5, "ragged": rng.random() < 0.7,
                    "idle": 1 if batch > 4 and rng.random() < 0.5 else 0}
        if rng.random() < 0.6:     # single or few tokens
            batch, rows = _log(rng, 1, 64), rng.choice((1, 1, 1, 2, 5))
            length = rows - 1 + _log(rng, 1, min(131072, 200000 // batch))
        else:                      # prompts and chunks
            batch = _log(rng, 1, 4)
            rows = _log(rng, 9, int(1400 / batch ** 0.5))
            length = rows + rng.choice((0, _log(rng, 1, max(1, 2000000 // (batch * rows) - rows))))
        return {"op": op, "batch": batch, "rows": rows, "length": length, "hq": hq, "hkv": hkv, "d": d,
                "window": rng.choice((0, 0, 750, _log(rng, 1, 2000))), "ragged": rng.random() < 0.6,
                "idle": 1 if batch > 4 and rng.random() < 0.5 else 0}
    if op == "norm":
        return {"op": op, "m": _log(rng, 1, 6020), "c": 32 * _log(rng, 1, 96), "post": rng.random() < 0.5,
                "gate": rng.choice((0, 1, 2)), "mod": rng.choice((0, 1, 2)), "res_bf16": rng.random() < 0.4,
                "y_bf16": rng.random() < 0.3, "out_bf16": rng.random() < 0.8}
    return {"op": op, "m": _log(rng, 1, 32), "v": _log(rng, 1000, 131072), "history": _log(rng, 1, 8000), "bias": _log(rng, 1, 300),
            "mask": rng.random() < 0.7}


def _sequences(case):
    """(rows, length) of each sequence: unequal ones fall from the case's size to a quarter of it; the idle slots of a batch
    have a row and nothing in the cache."""
    n = case["batch"]
    seqs = []
    for b in range(n):
        f = 1.0 - 0.75 * b / max(1, n - 1) if case["ragged"] else 1.0
        rows = max(1, int(case["rows"] * f))
        seqs.append((rows, rows + int((case["length"] - case["rows"]) * f)))
    for b in range(n - case["idle"], n):
        seqs[b] = (1, 0)
    return seqs


def work(case):
    if case["op"] in ("attention", "append"):
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        seqs = _sequences(case)
        rows = sum(r for r, _ in seqs)
        if case["op"] == "append":
            new = sum(min(r, n) for r, n in seqs)
            return {"bytes": rows * hq * d * 6 + new * hkv * d * 10 + new * case["rot"] * 4, "flops": rows * (hq + hkv) * case["rot"] * 3}
        w, pairs, seen = case["window"], 0, 0
        for r, n in seqs:
            for p in range(max(0, n - r), n):
                pairs += min(p + 1, w) if w else p + 1
            seen += min(n, w + r - 1) if w else n
        return {"bytes": rows * hq * d * 4 + seen * hkv * d * 2, "flops": 4 * pairs * hq * d}
    if case["op"] == "norm":
        m, c = case["m"], case["c"]
        per = 4 - 2 * case["y_bf16"] + 2 * (4 - 2 * case["res_bf16"]) + 4 - 2 * case["out_bf16"]
        wide = {0: 0, 1: 1, 2: m}
        return {"bytes": m * c * per + 4 * c * (1 + case["post"] + wide[case["gate"]] + wide[case["mod"]]), "flops": m * c * 10}
    m, v = case["m"], case["v"]
    return {"bytes": m * (8 * v + (v // 8 if case["mask"] else 0) + 4 * case["history"] + 8 * case["bias"]), "flops": m * v * 4}


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


def _paged(case, g):
    """A filled cache, its block table, lengths and row bounds: blocks in no order, a table wider than the longest
    sequence, and bytes of an earlier use in the unused slots of the last blocks."""
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
    tilt = torch.exp(0.6 * torch.randn((2, hkv, 1, d), generator=g, device=DEV))      # some channels are larger
    step = max(1, (1 << 27) // (hkv * 2 * BLOCK * d))
    for i in range(0, nb, step):
        n = min(step, nb - i)
        for kv, blocks in ((0, _k_blocks), (1, _v_blocks)):
            x = torch.randn((n, hkv, BLOCK, d), generator=g, device=DEV) * tilt[kv]
            e = _exponent(x.abs().amax((2, 3)))
            data[i:i + n, :, kv] = blocks(torch.ldexp(x, -e[:, :, None, None]).to(E4M3).view(torch.uint8))
            exps[i:i + n, :, kv] = e.to(torch.int8)
    cu = [0]
    for r, _ in seqs:
        cu.append(cu[-1] + r)
    uneven = len({r for r, _ in seqs}) > 1
    return {"cache": cache, "blocks": nb, "table": table.to(DEV),
            "lengths": torch.tensor([n for _, n in seqs], dtype=torch.int32, device=DEV),
            "cu": torch.tensor(cu, dtype=torch.int32, device=DEV) if uneven else None,
            "rows": cu[-1], "max_rows": max(r for r, _ in seqs), "max_length": max(n for _, n in seqs)}


def _rope(positions, rot):
    freq = 1.0e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    angle = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * freq
    return torch.stack((angle.cos(), angle.sin()), -1).float()


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "attention":
        s.update(_paged(case, g))
        s["q"] = torch.randn((s["rows"], case["hq"] * case["d"]), generator=g, device=DEV).bfloat16()
        return s
    if case["op"] == "append":
        s.update(_paged(case, g))
        s["q"] = torch.randn((s["rows"], case["hq"] * case["d"]), generator=g, device=DEV)
        # one call's linear outputs; now and then a row is larger than what the block holds so far
        big = 1.0 + 3.0 * (torch.rand((s["rows"], 1), generator=g, device=DEV) < 0.2)
        s["k"] = torch.randn((s["rows"], case["hkv"] * case["d"]), generator=g, device=DEV) * big
        s["v"] = torch.randn((s["rows"], case["hkv"] * case["d"]), generator=g, device=DEV) * big
        s["rope"] = _rope(case["length"], case["rot"])
        # the scheduler's list of the blocks that the call writes
        touched = [s["table"][b, j] for b, (r, n) in enumerate(_sequences(case)) if n >= r
                   for j in range((n - r) // BLOCK, -(-n // BLOCK))]
        s["touched"] = torch.stack(touched).long()
        return s
    if case["op"] == "norm":
        m, c = case["m"], case["c"]

        def rand(*shape):
            return torch.randn(shape, generator=g, device=DEV)

        s["y"] = (rand(m, c) * 0.7).to(torch.bfloat16 if case["y_bf16"] else torch.float32)
        s["residual"] = (rand(m, c) * 2.0).to(torch.bfloat16 if case["res_bf16"] else torch.float32)
        s["weight"] = 1.0 + 0.2 * rand(c)
        s["post"] = 1.0 + 0.2 * rand(c) if case["post"] else None
        s["gate"] = (0.5 + 0.3 * rand(1 if case["gate"] == 1 else m, c)) if case["gate"] else None
        s["mod"] = 0.3 * rand(1 if case["mod"] == 1 else m, c) if case["mod"] else None
        s["scale"], s["eps"] = (0.7 if case["post"] else 1.0), 1e-5
        return s
    m, v = case["m"], case["v"]
    s["logits"] = torch.randn((m, v), generator=g, device=DEV) * 3.0
    # a history repeats some tokens often
    n = m * case["history"]
    s["history"] = (v * torch.rand(n, generator=g, device=DEV) ** 3).int().clamp_(max=v - 1)
    s["cu_history"] = torch.arange(m + 1, dtype=torch.int32, device=DEV) * case["history"]
    s["prompt"] = (torch.rand(m, generator=g, device=DEV) * (case["history"] + 1)).int()
    s["repetition"] = 1.0 + 0.5 * torch.rand(m, generator=g, device=DEV)
    s["frequency"] = 0.4 * torch.rand(m, generator=g, device=DEV)
    s["presence"] = torch.rand(m, generator=g, device=DEV)
    nb = min(case["bias"], v)
    s["bias_ids"] = torch.stack([torch.randperm(v, generator=g, device=DEV)[:nb] for _ in range(m)]).int().view(-1)
    s["bias"] = torch.randn(m * nb, generator=g, device=DEV) * 5.0
    s["cu_bias"] = torch.arange(m + 1, dtype=torch.int32, device=DEV) * nb
    s["mask"] = None
    if case["mask"]:               # some words allow nothing, some all, some a part
        w = (v + 31) // 32
        bits = torch.randint(-2 ** 31, 2 ** 31, (m, w), generator=g, device=DEV, dtype=torch.int64)
        kind = torch.randint(0, 3, (m, w), generator=g, device=DEV)
        s["mask"] = torch.where(kind == 0, bits, torch.where(kind == 1, -torch.ones_like(bits), torch.zeros_like(bits))).int()
    return s


# ------------------------------------------------------------ plain forms
def _planes(s):
    c = s["case"]
    n = s["blocks"] * c["hkv"] * 2 * BLOCK * c["d"]
    return (s["cache"][:n].view(s["blocks"], c["hkv"], 2, BLOCK * c["d"]),
            s["cache"][n:].view(torch.int8).view(s["blocks"], c["hkv"], 2))


def _rows_of(s):
    """For every row: its sequence, its place among that sequence's rows, and its position (negative: none)."""
    n = s["lengths"].shape[0]
    row = torch.arange(s["rows"], device=DEV)
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(n + 1, device=DEV) * (s["rows"] // n)
    b = torch.searchsorted(cu, row, right=True) - 1
    t = row - cu[b]
    return b, t, s["lengths"].long()[b] - (cu[b + 1] - cu[b]) + t


def _attention(s):
    c = s["case"]
    hq, hkv, d, w = c["hq"], c["hkv"], c["d"], c["window"]
    data, exps = _planes(s)
    nblk = -(-s["max_length"] // BLOCK)
    ids = s["table"][:, :nblk].long().clamp(min=0)
    n, length = ids.shape[0], nblk * BLOCK
    got, e = data[ids], exps[ids].float()
    ek, ev = (torch.exp2(e[..., i]).permute(0, 2, 1).repeat_interleave(BLOCK, 2)[..., None] for i in (0, 1))
    k = got[:, :, :, 0].reshape(n, nblk, hkv, 2, d // 64, 4, 16, 16).permute(0, 2, 1, 3, 6, 4, 5, 7).reshape(n, hkv, length, d)
    v = got[:, :, :, 1].reshape(n, nblk, hkv, d // 32, 4, 16, 2, 2, 4).permute(0, 2, 1, 7, 4, 8, 3, 6, 5).reshape(n, hkv, length, d)
    k, v = k.view(E4M3).float() * ek, v.view(E4M3).float() * ev
    token = torch.arange(length, device=DEV)
    here = (token < s["lengths"][:, None])[:, None, :, None]
    k, v = torch.where(here, k, 0.0), torch.where(here, v, 0.0)
    b, t, pos = _rows_of(s)
    most, group = s["max_rows"], hq // hkv
    q = torch.zeros((n, most, hkv, group, d), device=DEV)
    q[b, t] = s["q"].float().view(-1, hkv, group, d)
    at = torch.full((n, most), -1, device=DEV)
    at[b, t] = pos
    scores = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(n, hkv, most * group, d), k.transpose(2, 3).contiguous()) * d ** -0.5
    sees = token <= at[:, :, None]
    if w:
        sees &= token > at[:, :, None] - w
    scores = scores.view(n, hkv, most, group, length)
    sees = sees[:, None, :, None]
    scores = torch.where(sees, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.where(sees, torch.exp(scores - torch.where(top == -math.inf, 0.0, top)), 0.0)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(n, hkv, most * group, length), v).view(n, hkv, most, group, d)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 2, 1, 3, 4)[b, t].reshape(s["rows"], hq * d).bfloat16()


def _rotate(x, cs, rot, interleaved):
    """x [rows, heads, d], cs [rows, rot / 2, 2]"""
    c, sn = cs[:, None, :, 0], cs[:, None, :, 1]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * c - b * sn, b * c + a * sn), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * c - b * sn, b * c + a * sn), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _append(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    data, exps = _planes(s)
    b, t, pos = _rows_of(s)
    live = pos >= 0
    at = pos.clamp(min=0)
    cs = s["rope"][at]
    q = _rotate(s["q"].view(-1, hq, d), cs, c["rot"], c["interleaved"])
    q = torch.where(live[:, None, None], q, 0.0).bfloat16().view(-1, hq * d)
    kv = torch.stack((_rotate(s["k"].view(-1, hkv, d), cs, c["rot"], c["interleaved"]), s["v"].view(-1, hkv, d)), 2)
    # rows without a position go nowhere: to a block after the last
    block = torch.where(live, s["table"][b, at // BLOCK].long(), s["blocks"])
    slot = at % BLOCK
    amax = torch.zeros((s["blocks"] + 1, hkv, 2), device=DEV).index_reduce_(0, block, kv.abs().amax(-1), "amax")
    fresh = torch.zeros(s["blocks"] + 1, device=DEV).index_reduce_(0, block, (slot == 0).float(), "amax") > 0
    touched = s["touched"]
    before, found = exps[touched].int(), _exponent(amax[touched])
    after = torch.where(fresh[touched][:, None, None], found, torch.maximum(before, found))
    factor = torch.where(fresh[touched][:, None, None], torch.zeros_like(after), before - after)
    old = data[touched].view(E4M3).float()
    data[touched] = torch.ldexp(old, factor[..., None]).to(E4M3).view(torch.uint8)
    exps[touched] = after.to(torch.int8)
    e = torch.cat((exps, exps[:1]))[block].int()
    codes = torch.ldexp(kv, -e[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)
    # one extra block takes what goes nowhere
    wide = torch.cat((data, data[:1]))
    kk = wide[:, :, 0].view(-1, hkv, 2, d // 64, 4, 16, 16)
    kk[block, :, slot // 16, :, :, slot % 16] = codes[:, :, 0].reshape(-1, hkv, d // 64, 4, 16)
    vv = wide[:, :, 1].view(-1, hkv, d // 32, 4, 16, 2, 2, 4)
    vv[block, :, :, slot // 4 % 4, :, :, slot // 16, slot % 4] = codes[:, :, 1].reshape(-1, hkv, d // 32, 2, 16).transpose(3, 4)
    data.copy_(wide[:-1])
    return _append_outputs(s, q)


def _append_outputs(s, q):
    data, exps = _planes(s)
    codes = data.view(E4M3)
    return {"q": q, "k": codes[:, :, 0], "v": codes[:, :, 1], "exponents": exps}


def _rms(x, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)


def _norm(s):
    c = s["case"]
    u, r = s["y"].float(), s["residual"].float()
    if s["post"] is not None:
        u = _rms(u, s["eps"]) * s["post"]
    if s["gate"] is not None:
        u = u * s["gate"]
    r = r + s["scale"] * u
    x = _rms(r, s["eps"]) * s["weight"]
    if s["mod"] is not None:
        x = x * (1.0 + s["mod"])
    return {"residual": r.to(s["residual"].dtype), "x": x.to(torch.bfloat16 if c["out_bf16"] else torch.float32)}


def _logits(s):
    z = s["logits"]
    m, v = z.shape
    row = torch.repeat_interleave(torch.arange(m, device=DEV), (s["cu_history"][1:] - s["cu_history"][:-1]).long(),
                                  output_size=s["history"].shape[0])
    answer = torch.arange(s["history"].shape[0], device=DEV) - s["cu_history"].long()[row] >= s["prompt"][row]
    at = row * v + s["history"].long()
    seen = torch.zeros(m * v, device=DEV).index_add_(0, at, torch.ones_like(at, dtype=torch.float32)).view(m, v) > 0
    count = torch.zeros(m * v, device=DEV).index_add_(0, at, answer.float()).view(m, v)
    rho = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rho, z * rho), z)
    z = z - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0).float()
    brow = torch.repeat_interleave(torch.arange(m, device=DEV), (s["cu_bias"][1:] - s["cu_bias"][:-1]).long(),
                                   output_size=s["bias"].shape[0])
    z = z.reshape(-1).index_add(0, brow * v + s["bias_ids"].long(), s["bias"]).view(m, v)
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
        z = torch.where(bits.view(m, -1)[:, :v] != 0, z, -math.inf)
    return z


def run(s):
    c = s["case"]
    if not own:
        return {"attention": _attention, "append": _append, "norm": _norm, "logits": _logits}[c["op"]](s)
    import q4_weight_only_amd as q4

    if c["op"] == "attention":
        cache = q4.KVCache(s["cache"], s["blocks"], c["hkv"], c["d"])
        return q4.kv_attention(s["q"], cache, s["table"], s["lengths"], s["cu"], max_rows=s["max_rows"],
                               max_length=s["max_length"], window=c["window"])
    if c["op"] == "append":
        cache = q4.KVCache(s["cache"], s["blocks"], c["hkv"], c["d"])
        q = q4.kv_append(s["q"], s["k"], s["v"], cache, s["table"], s["lengths"], s["rope"], s["cu"],
                         max_rows=s["max_rows"], interleaved=c["interleaved"])
        return _append_outputs(s, q)
    if c["op"] == "norm":
        residual, x = q4.add_rmsnorm(s["residual"], s["weight"], s["y"], post_weight=s["post"], gate=s["gate"],
                                     scale=s["scale"], modulation=s["mod"], eps=s["eps"],
                                     dtype=torch.bfloat16 if c["out_bf16"] else torch.float32)
        return {"residual": residual, "x": x}
    return q4.logits_adjust(s["logits"], history=s["history"], cu_history=s["cu_history"], prompt_lengths=s["prompt"],
                            repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                            bias_ids=s["bias_ids"], bias=s["bias"], cu_bias=s["cu_bias"], mask=s["mask"])


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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        u, r = s["y"].double(), s["residual"].double()
        if s["post"] is not None:
            u = u / torch.sqrt(u.square().mean(1, keepdim=True) + s["eps"]) * s["post"].double()
        r = r + s["scale"] * u * (1.0 if s["gate"] is None else s["gate"].double())
        x = r / torch.sqrt(r.square().mean(1, keepdim=True) + s["eps"]) * s["weight"].double()
        return {"residual": r, "x": x if s["mod"] is None else x * (1 + s["mod"].double())}
    if case["op"] == "logits":
        out = s["logits"].double()
        m, v = out.shape
        for i in range(m):
            ids = s["history"][s["cu_history"][i]:s["cu_history"][i + 1]].long()
            seen = torch.bincount(ids, minlength=v) > 0
            n = torch.bincount(ids[int(s["prompt"][i]):], minlength=v).double()
            rho, z = s["repetition"][i].double(), out[i]
            z = torch.where(seen & (z > 0), z / rho, torch.where(seen, z * rho, z))
            z = z - s["frequency"][i].double() * n - s["presence"][i].double() * (n > 0)
            one = slice(s["cu_bias"][i], s["cu_bias"][i + 1])
            z[s["bias_ids"][one].long()] += s["bias"][one].double()
            if s["mask"] is not None:
                word = torch.arange(v, device=DEV)
                z[(s["mask"][i].long()[word // 32] >> (word % 32)) & 1 == 0] = -math.inf
            out[i] = z
        return out
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    n = s["blocks"] * hkv * 2 * BLOCK * d
    data, exps = s["cache"][:n].view(-1, hkv, 2, BLOCK * d), s["cache"][n:].view(torch.int8).view(-1, hkv, 2)
    table, group = s["table"].long().cpu(), hq // hkv
    if case["op"] == "append":
        values, scale = _numbers(data), exps.clone()
        q = s["q"].double().view(-1, hq, d)
        k, v = s["k"].double().view(-1, hkv, d), s["v"].double().view(-1, hkv, d)
        i = torch.arange(d, device=DEV)
        rot = case["rot"]
        if case["interleaved"]:
            pair, mate, sign = i // 2, i ^ 1, torch.where(i % 2 == 0, -1.0, 1.0).double()
        else:
            pair, mate, sign = i % (rot // 2), (i + rot // 2) % rot, torch.where(i < rot // 2, -1.0, 1.0).double()
        turns = i < rot
        pair, mate = torch.where(turns, pair, 0), torch.where(turns, mate, i)
        row, turned_q = 0, torch.zeros_like(q)
        for b, (r, length) in enumerate(_sequences(case)):
            rows = slice(row, row + r)
            row += r
            if length < r:
                continue
            cs = s["rope"][length - r:length].double()
            co, si = (torch.where(turns, cs[:, pair, x], 1.0 - x)[:, None] for x in (0, 1))
            turned_q[rows] = q[rows] * co + q[rows][..., mate] * si * sign
            kk = k[rows] * co + k[rows][..., mate] * si * sign
            for j in range((length - r) // BLOCK, -(-length // BLOCK)):
                first = max(length - r, j * BLOCK)
                last = min(length, (j + 1) * BLOCK)
                blk = int(table[b, j])
                part = slice(first - (length - r), last - (length - r))
                new = (kk[part], v[rows][part])
                for which in (0, 1):
                    e = torch.ceil(torch.log2(new[which].abs().amax((0, 2)) / E4M3_MAX)).clamp(EXP_MIN, EXP_MAX)
                    if first % BLOCK:
                        old = scale[blk, :, which].double()
                        e = torch.maximum(e, old)
                        values[blk, :, which] *= torch.exp2(old - e)[:, None]
                    scale[blk, :, which] = e.to(torch.int8)
                    slots = torch.arange(first % BLOCK, first % BLOCK + last - first, device=DEV)
                    where = _index(d, slots[:, None])[which]
                    values[blk][:, which][:, where] = (new[which] / torch.exp2(e)[:, None]).transpose(0, 1)
        return {"q": turned_q.view(-1, hq * d), "k": values[:, :, 0], "v": values[:, :, 1], "exponents": None}
    out = torch.zeros((s["rows"], hkv, group, d), dtype=torch.float64, device=DEV)
    where = _index(d, torch.arange(BLOCK, device=DEV)[:, None])
    row = 0
    for b, (r, length) in enumerate(_sequences(case)):
        blocks = table[b, :-(-length // BLOCK)].to(DEV)
        for h in range(hkv if length else 0):
            k, v = ((_numbers(data[blocks, h, x][:, where[x]]) * torch.exp2(exps[blocks, h, x].double())[:, None, None]).view(-1, d)[:length]
                    for x in (0, 1))
            for t in range(0, r, 512):
                m = min(512, r - t)
                p = torch.arange(length - r + t, length - r + t + m, device=DEV)[:, None]
                j = torch.arange(length, device=DEV)
                sees = (j <= p) & (j > p - case["window"]) if case["window"] else j <= p
                q = s["q"][row + t:row + t + m].double().view(m, hkv, group, d)[:, h]
                z = torch.einsum("mgd,nd->mgn", q, k) / math.sqrt(d)
                w = torch.softmax(z.masked_fill(~sees[:, None], -math.inf), -1)
                out[row + t:row + t + m, h] = torch.einsum("mgn,nd->mgd", w, v)
        row += r
    return out.view(s["rows"], hq * d)
