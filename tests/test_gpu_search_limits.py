"""The operators around the paged cache at sizes where a launch cannot hold one workgroup for each
piece of work, where one kernel takes over from another, and where offsets pass 32 bits."""

import numpy as np
import pytest
import torch

from oracle import search_oracle as S
import q4_weight_only_amd as q4

from decoder_helpers import DEV, dev
from gpu_helpers import say

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)


def _filled(blocks, heads, D, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = q4.KVCache.empty(blocks, heads, D)
    codes, exps = c.planes()
    codes.random_(0, 0x7E, generator=g)                # any finite code of either sign
    codes |= torch.randint(0, 2, codes.shape, dtype=torch.uint8, device=DEV, generator=g) << 7
    exps.copy_(torch.randint(-4, 5, exps.shape, device=DEV, generator=g))
    s = torch.randint(0, 112, (blocks, heads, 2, D), dtype=torch.int8, device=DEV, generator=g)
    s[:, :, 1].neg_()
    return g, c, s


def test_more_sequences_and_ranges_than_a_launch_has():
    """20000 sequences of up to 2048 blocks: each workgroup takes more than one range of blocks."""
    batch, width, heads, D, keep = 20000, 2048, 1, 64, 5
    g, c, s = _filled(300, heads, D, 1)
    table = torch.randint(-1, 302, (batch, width), generator=g, **I32)
    lengths = torch.randint(0, 32 * width + 1, (batch,), generator=g, **I32)
    q = torch.randn((batch, 2 * D), device=DEV, generator=g).bfloat16()
    say("kv_select", batch, width)
    got = q4.kv_select(q, c, s, table, lengths, keep=keep)
    out = q4.kv_attention_blocks(q, c, got, table, lengths)
    for i in (0, 1, 777, 9999, 19999, int(lengths.argmax()), int(lengths.argmin())):
        one = slice(i, i + 1)
        few = q4.kv_select(q[one], c, s, table[one], lengths[one], keep=keep)
        assert torch.equal(got[one], few)
        assert torch.equal(out[one].isnan(), q4.kv_attention_blocks(q[one], c, few, table[one], lengths[one]).isnan())


def test_more_rows_than_a_launch_has():
    """A chunk of 70000 rows: the rows at its end are those of a chunk of 64 at the same positions."""
    rows, heads, D, keep = 70000, 1, 64, 3
    blocks = rows // 32 + 9
    g, c, s = _filled(blocks, heads, D, 2)
    table = torch.randperm(blocks, device=DEV, generator=g).int()[None]
    lengths = torch.tensor([rows + 100], **I32)
    q = torch.randn((rows, D), device=DEV, generator=g).bfloat16()
    say("kv_select", rows)
    got = q4.kv_select(q, c, s, table, lengths, keep=keep)
    out = q4.kv_attention_blocks(q, c, got, table, lengths)
    few = q4.kv_select(q[-64:].contiguous(), c, s, table, lengths, keep=keep)
    assert torch.equal(got[-64:], few)
    # (3 blocks are not split, so the sums are in the same order)
    assert torch.equal(out[-64:], q4.kv_attention_blocks(q[-64:].contiguous(), c, few, table, lengths))
    # hints that are too small cost time alone
    assert torch.equal(got, q4.kv_select(q, c, s, table, lengths, keep=keep, max_rows=1000))
    assert torch.equal(out, q4.kv_attention_blocks(q, c, got, table, lengths, max_rows=1000))


@pytest.mark.parametrize("n,width,blocks", [(256, 64, 8192), (257, 64, 8192), (256, 64, 8193), (255, 64, 8192), (256, 65, 8192), (4, 4096, 8192),
                                            (4, 4097, 8192), (1, 16384, 8192), (1, 1, 1)])
def test_fork_at_the_border_of_one_workgroup(n, width, blocks):
    rng = np.random.default_rng(n + width)
    table = rng.integers(-1, blocks + 1, (n, width))
    table[:, : width // 2] = table[0, : width // 2]                  # what they have in common
    lengths = rng.integers(0, 32 * width + 1, n)
    held = (rng.random(blocks) < 0.1).astype(int)
    say("kv_fork", n, width, blocks)
    for parents, grow in ((rng.integers(-1, n, n), 1), (np.full(n, n - 1), 40), (rng.integers(0, n, n), 300)):
        got = q4.kv_fork(dev(table, torch.int32), dev(lengths, torch.int32), dev(parents, torch.int32), blocks, grow=grow, held=dev(held, torch.int32))
        want = S.kv_fork(table, lengths, parents, blocks, np.full(n, grow), held)
        for name in got._fields:
            assert np.array_equal(getattr(got, name).cpu().numpy(), np.asarray(want[name] if isinstance(want, dict) else getattr(want, name))), name


def test_copies_past_4_gigabytes():
    """A cache of 6 GB: blocks at both of its ends."""
    blocks, heads, D = 90000, 8, 128
    c = q4.KVCache.empty(blocks, heads, D)
    codes, exps = c.planes()
    ids = torch.tensor([0, 65535, 65536, blocks - 2], device=DEV)
    for i in ids.tolist():
        codes[i].random_(0, 256)
        exps[i].random_(-30, 30)
    src, dst = ids.int(), torch.tensor([blocks - 1, 70000, 3, 32768], **I32)
    say("kv_copy_blocks", blocks)
    q4.kv_copy_blocks(c, src, dst)
    assert torch.equal(codes[dst.long()], codes[ids]) and torch.equal(exps[dst.long()], exps[ids])
    assert int((codes.view(blocks, -1).view(torch.int64) != 0).any(1).sum()) == 8
    # and what reads them: the last block alone
    table, lengths = torch.full((1, 4), blocks - 1, **I32), torch.tensor([128], **I32)
    summary = q4.kv_summary(c)
    q4.kv_summarize(c, summary, table, lengths, rows=1)
    assert summary[blocks - 1].any() and not summary[:blocks - 1].any()


def test_as_many_beams_as_a_call_takes():
    groups, beams, V, keep = 1023, 64, 77, 3
    g = torch.Generator(device=DEV).manual_seed(3)
    z = torch.randn((groups * beams, V), device=DEV, generator=g)
    s = -torch.rand((groups, beams), device=DEV, generator=g)
    say("beam_select", groups, beams)
    p, t, best = q4.beam_select(z, s, keep)
    for i in (0, 511, 1022):
        rows = slice(i * beams, (i + 1) * beams)
        wp, wt, ws = S.beam_select(z[rows].cpu().numpy(), s[i:i + 1].cpu().numpy(), keep)
        assert np.array_equal(p[i].cpu().numpy(), wp[0] + i * beams) and np.array_equal(t[i].cpu().numpy(), wt[0])
        # rounded once to fp32, from sums that are 1e-9 off
        assert (np.abs(best[i].cpu().numpy() - ws[0]) <= 2.0 ** -24 * np.abs(ws[0]) + 1e-9).all()
