"""kv_fork, kv_compact and kv_copy_blocks: whole numbers and bytes, equal to the oracle's."""

import numpy as np
import pytest
import torch

from oracle import search_oracle as S
import q4_weight_only_amd as q4

from decoder_helpers import DEV, dev
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _i32(x):
    return dev(np.asarray(x), torch.int32)


def _fork(table, lengths, parents, blocks, grow=1, held=None, **kw):
    say("kv_fork", np.shape(table), len(parents), blocks)
    g = grow if np.isscalar(grow) else _i32(grow)
    got = q4.kv_fork(_i32(table), _i32(lengths), _i32(parents), blocks, grow=g, held=None if held is None else _i32(held), **kw)
    want = S.kv_fork(np.asarray(table), lengths, parents, blocks, grow, held)
    for name, a in zip(got._fields, got):
        assert np.array_equal(a.cpu().numpy(), want[name]), name
    return want


def _tables(rng, rows, width, blocks, *, spoil=False):
    """Rows that share prefixes of random depth, of random lengths."""
    table = np.full((rows, width), -1)
    lengths = rng.integers(0, 32 * width + 1, rows)
    for r in range(rows):
        n = -(-lengths[r] // 32)
        table[r, :n] = rng.integers(0, blocks, n)
        if r and rng.random() < 0.7:
            other = rng.integers(r)
            depth = min(n, -(-lengths[other] // 32))
            table[r, :depth] = table[other, :depth]
            if rng.random() < 0.5 and depth == n and lengths[other] >= lengths[r]:
                lengths[r] = max(0, min(32 * n, lengths[other] - 32 * rng.integers(0, 2)))
                lengths[r] = max(lengths[r], 32 * n - 31) if n else 0
    if spoil:      # ids outside the cache, lengths outside the table
        table[rng.random(table.shape) < 0.1] = blocks + 3
        table[rng.random(table.shape) < 0.05] = -9
        lengths[rng.random(rows) < 0.2] = 32 * width + 50
        lengths[rng.random(rows) < 0.2] = -4
    return table, lengths


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("rows,width,n,blocks", [(1, 1, 1, 1), (1, 3, 4, 20), (4, 5, 4, 60), (8, 17, 8, 300), (30, 9, 50, 400), (5, 1100, 12, 9000)])
def test_fork(rows, width, n, blocks, seed):
    rng = np.random.default_rng(seed)
    table, lengths = _tables(rng, rows, width, blocks, spoil=seed % 2)
    parents = rng.integers(-2, rows + 1, n)
    held = rng.integers(-1, 2, blocks) * (rng.random(blocks) < 0.3) if seed % 3 else None
    _fork(table, lengths, parents, blocks, 1, held)
    _fork(table, lengths, parents, blocks, 0, held)
    _fork(table, lengths, parents, blocks, rng.integers(-3, 200, n), held)


def test_fork_of_more_sequences_than_threads():
    rng = np.random.default_rng(1)
    table, lengths = _tables(rng, 700, 6, 9000)
    parents = rng.integers(-1, 700, 2500)
    _fork(table, lengths, parents, 9000, rng.integers(0, 70, 2500))


def test_fork_over_a_large_pool():
    """More blocks than one turn of the search, the free ones at its end, and more wanted than a turn has."""
    rng = np.random.default_rng(2)
    blocks, width = 50000, 700
    table = rng.permutation(49000)[:60 * width].reshape(60, width)
    lengths = np.full(60, 32 * (width - 100))
    held = (np.arange(blocks) < 40000).astype(int)
    _fork(table, lengths, np.arange(60), blocks, 90 * 32, held)


def test_all_that_go_on_in_a_block():
    """The same partly filled block under many sequences, some of which do not grow."""
    table, lengths = np.array([[4, 2], [4, 2], [2, -1]]), [50, 64, 32]
    for parents, grow in (([0] * 7, 1), ([0, 0, 0], [1, 0, 1]), ([0, 1, 0], 1), ([0, 2], 1), ([0], 1), ([0, 0], 0), ([0, 0, -1], 15)):
        _fork(table, lengths, parents, 10, grow)
        _fork(table, lengths, parents, 10, grow, held=[0, 0, 1, 0, 0, 0, 0, 0, 0, 0])
        _fork(table, lengths, parents, 10, grow, held=[1, 1, 0, 1, 0, 0, 1, 1, 1, 0])     # one free block


def test_new_sequences_and_ended_ones():
    """A slot without a sequence starts one; parents outside the rows end theirs, and their blocks are free at once."""
    table, lengths = np.array([[0, 1, 2], [3, 4, 5], [-1, -1, -1]]), [96, 96, 0]
    want = _fork(table, lengths, [-1, 1, 2], 6, [5, 0, 90])
    assert want["block_table"].tolist() == [[-1] * 3, [3, 4, 5], [0, 1, 2]]


def test_no_sequences():
    f = q4.kv_fork(torch.empty((0, 4), dtype=torch.int32, device=DEV), _i32([]), _i32([]), 9, held=_i32([0, 1, 2, -3, 0, 0, 0, 0, 5]))
    assert f.refs.tolist() == [0, 1, 2, 0, 0, 0, 0, 0, 5] and f.block_table.shape == (0, 4)
    _fork(np.empty((0, 4), dtype=int), [], [0, -1], 9)


def test_outputs_of_the_caller():
    rng = np.random.default_rng(3)
    table, lengths = _tables(rng, 6, 8, 100)
    parents = rng.integers(0, 6, 9)
    want = q4.kv_fork(_i32(table), _i32(lengths), _i32(parents), 100)
    out = tuple(torch.full_like(x, 99) for x in want)
    ws = torch.full((q4.kv_fork_workspace(9, 100),), 255, dtype=torch.uint8, device=DEV)
    got = q4.kv_fork(_i32(table), _i32(lengths), _i32(parents), 100, out=out, workspace=ws)
    assert all(torch.equal(a, b) and a.data_ptr() == c.data_ptr() for a, b, c in zip(got, want, out))
    want = q4.kv_compact(_i32(table), _i32(lengths), 100)
    out = tuple(torch.full_like(x, 99) for x in want)
    ws = torch.full((q4.kv_compact_workspace(100),), 255, dtype=torch.uint8, device=DEV)
    got = q4.kv_compact(_i32(table), _i32(lengths), 100, out=out, workspace=ws)
    assert all(torch.equal(a, b) and a.data_ptr() == c.data_ptr() for a, b, c in zip(got, want, out))


# ---------------------------------------------------------------- compact
def _compact(table, lengths, blocks, held=None):
    say("kv_compact", np.shape(table), blocks)
    got = q4.kv_compact(_i32(table), _i32(lengths), blocks, held=None if held is None else _i32(held))
    want = S.kv_compact(np.asarray(table), lengths, blocks, held)
    for name, a in zip(got._fields, got):
        assert np.array_equal(a.cpu().numpy(), want[name]), name
    return want


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("rows,width,blocks", [(1, 1, 1), (1, 1, 2), (3, 4, 40), (20, 30, 700), (16, 200, 4096), (16, 200, 4097), (40, 300, 30000)])
def test_compact(rows, width, blocks, seed):
    rng = np.random.default_rng(seed)
    table, lengths = _tables(rng, rows, width, blocks, spoil=seed % 2)
    held = None if seed % 3 == 0 else (rng.random(blocks) < (0.05, 0.6)[seed % 2]).astype(int) * 2
    _compact(table, lengths, blocks, held)


@pytest.mark.parametrize("blocks", [8192, 8191, 12289])
def test_compact_at_the_borders_of_tiles(blocks):
    """As many blocks in use as tiles hold, one fewer, all and none; the ones that stay at the end."""
    rng = np.random.default_rng(1)
    for live in (0, 1, 4095, 4096, 4097, blocks - 1, blocks):
        ids = rng.permutation(blocks)[:live] if live < blocks else rng.permutation(blocks)
        if 0 < live < blocks:
            ids[np.argmax(ids)] = blocks - 1
            ids = np.unique(ids)
            rng.shuffle(ids)
        table = np.full((1, max(1, blocks)), -1)
        table[0, :len(ids)] = ids
        _compact(table, [32 * len(ids)], blocks)
    held = np.zeros(blocks, dtype=int)
    held[-3000:] = 1
    _compact(np.array([[5, 4090, 1]]), [96], blocks, held)
    _compact(np.array([[5, blocks - 3500, blocks - 3100]]), [96], blocks, held)


@pytest.mark.parametrize("blocks", [65535, 65536, 65537, 70001, 131072])
@pytest.mark.parametrize("rows,width", [(3, 900), (1024, 64), (1025, 3), (40, 1700), (1, 65536), (64, 4096), (64, 4097)])
def test_compact_of_large_pools_and_tables(blocks, rows, width):
    """Around the sizes up to which one launch does it all."""
    rng = np.random.default_rng(blocks + rows)
    table, lengths = _tables(rng, rows, width, blocks, spoil=True)
    _compact(table, lengths, blocks, (rng.random(blocks) < 0.3).astype(int) * 3 - 1)
    _compact(table, lengths, blocks)


@pytest.mark.parametrize("blocks", [66560, 67583, 69632])
def test_compact_at_the_borders_of_large_tiles(blocks):
    """As many blocks in use as tiles of 1024 hold, one fewer, one more, all and none."""
    rng = np.random.default_rng(1)
    for live in (0, 1, 1023, 1024, 1025, 65536, blocks - 1, blocks):
        ids = rng.permutation(blocks)[:live]
        if 0 < live < blocks:
            ids[0] = blocks - 1
            ids = np.unique(ids)
            rng.shuffle(ids)
        table = np.full((1, blocks), -1)
        table[0, :len(ids)] = ids
        _compact(table, [32 * len(ids)], blocks)


def test_compact_then_everything_reads_the_same():
    rng = np.random.default_rng(4)
    blocks, heads, D = 90, 2, 64
    table = np.full((3, 12), -1)
    ids = rng.permutation(blocks)
    table[0, :10], table[1, :12], table[2, :9] = ids[:10], ids[10:22], ids[15:24]
    lengths = [32 * 9 + 5, 32 * 12, 32 * 8 + 1]
    stack = q4.KVStack(torch.randint(0, 256, (3, -(-blocks * heads * 2 * (32 * D + 1) // 16) * 16), dtype=torch.uint8, device=DEV),
                       blocks, heads, D)
    before = [tuple(x[table[table >= 0]].clone() for x in c.planes()) for c in stack]
    f = q4.kv_compact(_i32(table), _i32(lengths), blocks)
    q4.kv_copy_blocks(stack, f.src, f.dst)
    now = f.block_table.cpu().numpy()
    assert (now[table >= 0] < int(f.live)).all() and int(f.live) == 24
    for c, b in zip(stack, before):
        assert all(torch.equal(x[now[table >= 0]], y) for x, y in zip(c.planes(), b))


# ------------------------------------------------------------------- copy
@pytest.mark.parametrize("heads,D,layers,n", [(1, 64, 1, 1), (1, 64, 3, 200), (3, 128, 2, 7), (8, 128, 33, 2), (8, 64, 70, 3), (256, 64, 1, 2), (2, 64, 2, 5000)])
@pytest.mark.parametrize("form", ["stack", "list"])
def test_copy(heads, D, layers, n, form):
    rng = np.random.default_rng(1)
    blocks = 2 * n + 3
    size = blocks * heads * 2 * (32 * D + 1)
    src, dst = np.split(rng.permutation(blocks)[:2 * n], 2)
    src[rng.random(n) < 0.2] = -1
    if n > 4:
        src[1], dst[2], src[3], dst[4] = blocks, -1, -7, blocks + 2
    say("kv_copy_blocks", heads, D, layers, n, form)
    data = torch.randint(0, 256, (layers, -(-size // 16) * 16), dtype=torch.uint8, device=DEV)
    summary = torch.randint(-128, 128, (layers, blocks, heads, 2, D), dtype=torch.int8, device=DEV)
    want, want_summary = data.clone(), summary.clone()
    good = (src >= 0) & (src < blocks) & (dst >= 0) & (dst < blocks)
    s, d = torch.from_numpy(src[good]).to(DEV), torch.from_numpy(dst[good]).to(DEV)
    codes, exps = (want[:, a:b].view(layers, blocks, -1) for a, b in ((0, blocks * heads * 64 * D), (blocks * heads * 64 * D, size)))
    codes[:, d], exps[:, d], want_summary[:, d] = codes[:, s], exps[:, s], want_summary[:, s]
    if form == "stack":
        q4.kv_copy_blocks(q4.KVStack(data, blocks, heads, D), _i32(src), _i32(dst), summaries=summary)
    else:
        caches = [q4.KVCache(data[i, :size].clone(), blocks, heads, D) for i in range(layers)]
        q4.kv_copy_blocks(caches, _i32(src), _i32(dst))
        data = torch.stack([torch.cat((c.data, data[i, size:])) for i, c in enumerate(caches)])
        want_summary = summary
    assert torch.equal(data, want) and torch.equal(summary, want_summary)


def test_copy_of_one_cache_and_of_nothing():
    c = q4.KVCache.empty(5, 2, 64)
    c.data.random_(0, 256)
    was = c.data.clone()
    q4.kv_copy_blocks(c, _i32([]), _i32([]))
    q4.kv_copy_blocks([], _i32([1]), _i32([2]))
    assert torch.equal(c.data, was)
    q4.kv_copy_blocks(c, _i32([4]), _i32([0]))
    codes, exps = c.planes()
    assert torch.equal(codes[0], codes[4]) and torch.equal(exps[0], exps[4])


# --------------------------------------------------------------- refusals
def test_refusals():
    t, n, p = _i32(np.zeros((3, 4))), _i32([0, 0, 0]), _i32([0, 1])
    c, d = q4.KVCache.empty(5, 2, 64), q4.KVCache.empty(6, 2, 64)
    stack = q4.KVStack.empty(2, 5, 2, 64)
    for bad in (lambda: q4.kv_fork(t.cpu(), n, p, 5), lambda: q4.kv_fork(t, n.long(), p, 5), lambda: q4.kv_fork(t, p, p, 5),
                lambda: q4.kv_fork(t, n, p.float(), 5), lambda: q4.kv_fork(t, n, p, 0), lambda: q4.kv_fork(t, n, p, 2**24 + 1),
                lambda: q4.kv_fork(t, n, p, 5, grow=-1), lambda: q4.kv_fork(t, n, p, 5, grow=n), lambda: q4.kv_fork(t, n, p, 5, held=n),
                lambda: q4.kv_fork(t, n, p, 5, out=(t,)), lambda: q4.kv_fork(t, n, p, 5, workspace=torch.empty(8, dtype=torch.uint8, device=DEV)),
                lambda: q4.kv_compact(t, n, 0), lambda: q4.kv_compact(t, n, 5, held=n), lambda: q4.kv_compact(t[:, ::2], n, 5),
                lambda: q4.kv_copy_blocks([c, d], p, p), lambda: q4.kv_copy_blocks(c, p, n), lambda: q4.kv_copy_blocks(c, p.cpu(), p.cpu()),
                lambda: q4.kv_copy_blocks(c, p, p, summaries=q4.kv_summary(d)[:1]),
                lambda: q4.kv_copy_blocks(stack, p, p, summaries=[q4.kv_summary(c)]),
                lambda: q4.KVStack(stack.data[:, 1:], 5, 2, 64), lambda: q4.KVStack(stack.data[:, ::2], 2, 2, 64),
                lambda: q4.KVStack(stack.data[0], 5, 2, 64), lambda: q4.KVStack(stack.data.cpu(), 5, 2, 64),
                lambda: q4.KVStack(stack.data, 5, 2, 96)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(IndexError):
        stack[2]
    assert len(stack) == 2 and len(list(stack)) == 2 and torch.equal(stack[1].data, stack.data[1, :stack[1].data.numel()])


def test_outputs_that_overlap_are_refused():
    t, n, p = _i32(np.zeros((3, 4))), _i32([0, 0, 0]), _i32([0, 1, 2])
    f = q4.kv_fork(t, n, p, 5)
    c = q4.kv_compact(t, n, 5)
    flat = _i32(np.zeros(20))
    for bad in (lambda: q4.kv_fork(t, n, p, 5, out=f._replace(block_table=t)), lambda: q4.kv_fork(t, n, p, 5, out=f._replace(lengths=n)),
                lambda: q4.kv_fork(t, n, p, 5, out=f._replace(src=p)), lambda: q4.kv_fork(t, n, p, 5, out=f._replace(src=f.dst)),
                lambda: q4.kv_fork(t, n, flat[:3], 5, out=f._replace(dst=flat[2:5])),
                lambda: q4.kv_fork(t, n, p, 5, grow=f.dst, out=f), lambda: q4.kv_fork(t, n, p, 5, held=f.refs, out=f),
                lambda: q4.kv_compact(t, n, 5, out=c._replace(block_table=t)), lambda: q4.kv_compact(t, n, 5, out=c._replace(src=c.dst)),
                lambda: q4.kv_compact(t, n, 5, held=flat[:5], out=c._replace(live=flat[4:5]))):
        with pytest.raises(ValueError, match="overlap"):
            bad()
    # next to each other, and parts of what an earlier call returned
    g = q4.kv_fork(t, n, flat[:3], 5, out=(None, None, None, flat[3:6], flat[6:9], None))
    h = q4.kv_fork(f.block_table, f.lengths, p, 5, out=q4.kv_fork(t, n, p, 5))
    assert g.src.data_ptr() == flat[3:6].data_ptr() and h.block_table.shape == (3, 4)


def test_a_summary_that_is_not_in_one_piece_is_refused():
    """(A copy of it would be written instead.)"""
    stack = q4.KVStack.empty(2, 6, 2, 64)
    wide = torch.zeros((2, 6, 2, 2, 128), dtype=torch.int8, device=DEV)
    p = _i32([0])
    for bad in (wide[..., :64], wide[..., ::2], torch.zeros(2, dtype=torch.int8, device=DEV)):
        with pytest.raises(ValueError):
            q4.kv_copy_blocks(stack, p, p + 1, summaries=bad)
    padded = torch.arange(2 * 3200, device=DEV).to(torch.int8).view(2, 3200)[:, :6 * 256]
    before = padded.clone().view(2, 6, 256)
    q4.kv_copy_blocks(stack, p, p + 1, summaries=padded)
    after = padded.reshape(2, 6, 256)
    assert torch.equal(after[:, 1], before[:, 0]) and torch.equal(after[:, 2:], before[:, 2:]) and torch.equal(after[:, 0], before[:, 0])


@pytest.mark.parametrize("rows,width,blocks", [(4, 6, 64), (40, 20, 9000), (300, 8, 900), (60, 900, 70000)])
def test_graph_replays_follow_their_inputs(rows, width, blocks):
    """The forms for small and for large tables, replayed over other tables, with eager calls in between."""
    rng = np.random.default_rng(rows)
    say("graph", rows, width, blocks)
    sets = []
    for _ in range(3):
        table, lengths = _tables(rng, rows, width, blocks)
        sets.append((_i32(table), _i32(lengths), _i32(rng.integers(-1, rows, rows))))
    held = _i32((rng.random(blocks) < 0.2).astype(int))
    t, n, p = (x.clone() for x in sets[0])
    q4.kv_fork(t, n, p, blocks, held=held), q4.kv_compact(t, n, blocks, held=held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = q4.kv_fork(t, n, p, blocks, held=held)
        c = q4.kv_compact(f.block_table, f.lengths, blocks, held=held)
    for i in (1, 2, 0, 1):
        for x, y in zip((t, n, p), sets[i]):
            x.copy_(y)
        graph.replay()
        wf = q4.kv_fork(*sets[i], blocks, held=held)
        wc = q4.kv_compact(wf.block_table, wf.lengths, blocks, held=held)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(f, wf)) and all(torch.equal(x, y) for x, y in zip(c, wc))


def test_fork_into_tensors_that_start_anywhere():
    """Counts of a large and nearly full pool, read four at a time, in a tensor that starts on 4 bytes alone."""
    rng = np.random.default_rng(8)
    blocks, rows, width = 30011, 20, 30
    free = np.sort(rng.permutation(blocks)[:rows + 3])
    held = np.ones(blocks, dtype=int)
    held[free] = 0
    table = rng.permutation(np.flatnonzero(held))[:rows * width].reshape(rows, width)
    table[:, -1] = -1
    lengths = np.full(rows, 32 * (width - 1))
    want = S.kv_fork(table, lengths, np.arange(rows), blocks, 1, held)
    for start in (0, 1, 2, 3):
        flat = torch.full((blocks + 8,), 77, dtype=torch.int32, device=DEV)
        got = q4.kv_fork(_i32(table), _i32(lengths), _i32(np.arange(rows)), blocks, held=_i32(held),
                         out=(None, None, flat[start:start + blocks], None, None, None))
        for name, a in zip(got._fields, got):
            assert np.array_equal(a.cpu().numpy(), want[name]), name
        assert (flat[:start] == 77).all() and (flat[start + blocks:] == 77).all()
