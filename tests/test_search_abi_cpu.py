"""C-ABI checks of the operators of include/q4_search.h that need no GPU: what the
header declares is exported, sizes come out as documented, and bad arguments are refused before the HIP
runtime is touched.  Fake device addresses are never dereferenced: only calls that
fail validation, or have nothing to do, are made."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

import q4_weight_only_amd as q4
from q4_weight_only_amd import _decoder as D
from q4_weight_only_amd import _search as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "q4_search.h")
FAKE, MISALIGNED = 0x10000, 0x10004
OK, NULL, ALIGN, RANGE = 0, 1, 3, 6
BIG = 2**40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(q4.library_path()):
        import sys
        subprocess.run([sys.executable, "-m", "q4_weight_only_amd.build"], check=True)
    return S.search_lib()


def test_every_declared_function_is_exported(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(q4_\w+)\s*\(", text)))
    assert names == sorted(S.SEARCH_EXPORTS)
    for name in names:
        assert hasattr(L, name), name


def cache(**kw):
    c = dict(data=FAKE, num_blocks=16, kv_heads=2, head_dim=64)
    c.update(kw)
    return ctypes.byref(D._Cache(**c))


def batch(**kw):
    b = dict(block_table=FAKE, lengths=FAKE, cu_rows=None, table_width=4, batch=2, rows=2, max_rows=1, max_length=64)
    b.update(kw)
    return ctypes.byref(D._Batch(**b))


BAD_CACHES = [dict(num_blocks=0), dict(num_blocks=2**24 + 1), dict(kv_heads=0), dict(kv_heads=257), dict(head_dim=80)]
BAD_BATCHES = [dict(batch=-1), dict(batch=65536), dict(rows=-1), dict(rows=2**20 + 2), dict(table_width=0),
               dict(table_width=2**20 + 1), dict(max_rows=0), dict(max_rows=2**20 + 1), dict(max_length=0),
               dict(max_length=2**25 + 1), dict(rows=3)]


def test_beam_select_validates_first(L):
    def call(z=FAKE, groups=2, beams=3, v=100, scores=FAKE, finished=None, pad=0, keep=3, parents=FAKE, tokens=FAKE,
             best=FAKE, ws=FAKE, nbytes=BIG):
        return L.q4_beam_select(z, groups, beams, v, scores, finished, pad, keep, parents, tokens, best, ws, nbytes, None)

    for kw in (dict(groups=-1), dict(beams=0), dict(beams=65), dict(groups=1025, beams=64), dict(v=0), dict(v=2**24 + 1),
               dict(keep=0), dict(keep=129), dict(pad=-1)):
        assert call(**kw) == RANGE, kw
    for kw in (dict(z=None), dict(scores=None), dict(parents=None), dict(tokens=None), dict(best=None), dict(ws=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(z=FAKE + 2), dict(scores=FAKE + 1), dict(finished=FAKE + 2), dict(parents=FAKE + 3), dict(tokens=FAKE + 2),
               dict(best=FAKE + 2), dict(ws=MISALIGNED)):
        assert call(**kw) == ALIGN, kw
    need = q4.beam_select_workspace(2, 3, 100)
    assert need > 0 and need % 16 == 0
    assert call(nbytes=need - 1) == RANGE
    assert call(groups=0, z=None, ws=None, nbytes=0) == OK
    assert q4.beam_select_workspace(0, 3, 100) == 0 and q4.beam_select_workspace(2, 65, 100) == 0
    # the largest: 65535 rows of 2^24 tokens, past 32 bits
    assert q4.beam_select_workspace(65535, 1, 2**24) > 2**32


def test_beam_advance_validates_first(L):
    def call(seq=FAKE, rows=4, width=8, lengths=FAKE, finished=None, parents=FAKE, tokens=FAKE, n=4, out=FAKE, out_l=FAKE,
             out_f=FAKE):
        return L.q4_beam_advance(seq, rows, width, lengths, finished, parents, tokens, n, 2, 0, out, out_l, out_f, None)

    for kw in (dict(rows=-1), dict(rows=2**20 + 1), dict(n=-1), dict(n=2**20 + 1), dict(width=0), dict(width=2**24 + 1)):
        assert call(**kw) == RANGE, kw
    for kw in (dict(seq=None), dict(lengths=None), dict(parents=None), dict(tokens=None), dict(out=None), dict(out_l=None), dict(out_f=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(seq=FAKE + 2), dict(finished=FAKE + 1), dict(out=FAKE + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(n=0, seq=None, parents=None, out=None) == OK


def test_fork_validates_first(L):
    def call(table=FAKE, rows=3, width=4, lengths=FAKE, parents=FAKE, n=3, grow=None, each=1, held=None, blocks=16, out=FAKE,
             out_l=FAKE, refs=FAKE, src=FAKE, dst=FAKE, short=FAKE, ws=FAKE, nbytes=BIG):
        return L.q4_kv_fork(table, rows, width, lengths, parents, n, grow, each, held, blocks, out, out_l, refs, src, dst, short, ws,
                            nbytes, None)

    for kw in (dict(rows=-1), dict(rows=65536), dict(n=-1), dict(n=65536), dict(width=0), dict(width=2**20 + 1), dict(blocks=0),
               dict(blocks=2**24 + 1), dict(rows=2**12, width=2**19), dict(n=2**12, width=2**19), dict(each=-1), dict(each=2**25 + 1)):
        assert call(**kw) == RANGE, kw
    for kw in (dict(table=None), dict(lengths=None), dict(parents=None), dict(out=None), dict(out_l=None), dict(refs=None),
               dict(src=None), dict(dst=None), dict(short=None), dict(ws=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(table=FAKE + 2), dict(grow=FAKE + 1), dict(held=FAKE + 2), dict(refs=FAKE + 1), dict(ws=MISALIGNED)):
        assert call(**kw) == ALIGN, kw
    need = q4.kv_fork_workspace(3, 16)
    assert need > 0 and need % 16 == 0 and call(nbytes=need - 1) == RANGE
    assert q4.kv_fork_workspace(65536, 16) == 0 and q4.kv_fork_workspace(3, 0) == 0


def test_compact_validates_first(L):
    def call(table=FAKE, rows=3, width=4, lengths=FAKE, held=None, blocks=16, out=FAKE, src=FAKE, dst=FAKE, live=FAKE, ws=FAKE,
             nbytes=BIG):
        return L.q4_kv_compact(table, rows, width, lengths, held, blocks, out, src, dst, live, ws, nbytes, None)

    for kw in (dict(rows=-1), dict(rows=65536), dict(width=0), dict(width=2**20 + 1), dict(blocks=0), dict(blocks=2**24 + 1),
               dict(rows=2**12, width=2**19)):
        assert call(**kw) == RANGE, kw
    for kw in (dict(table=None), dict(lengths=None), dict(out=None), dict(src=None), dict(dst=None), dict(live=None), dict(ws=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(table=FAKE + 2), dict(held=FAKE + 1), dict(live=FAKE + 2), dict(ws=MISALIGNED)):
        assert call(**kw) == ALIGN, kw
    need = q4.kv_compact_workspace(16)
    assert need > 0 and call(nbytes=need - 1) == RANGE and q4.kv_compact_workspace(0) == 0


def test_copy_validates_first(L):
    def call(c=None, data=(FAKE, FAKE), summaries=None, layers=2, src=FAKE, dst=FAKE, n=3):
        arrays = [None if x is None else (ctypes.c_void_p * max(1, len(x)))(*x) for x in (data, summaries)]
        return L.q4_kv_copy_blocks(c or cache(data=None), arrays[0], arrays[1], layers, src, dst, n, None)

    assert L.q4_kv_copy_blocks(None, None, None, 0, None, None, 0, None) == NULL
    for kw in BAD_CACHES:
        assert call(c=cache(**kw)) == RANGE, kw
    for kw in (dict(layers=-1), dict(layers=1025), dict(n=-1), dict(n=2**24 + 1)):
        assert call(**kw) == RANGE, kw
    for kw in (dict(data=None), dict(src=None), dict(dst=None), dict(data=(FAKE, None)), dict(summaries=(FAKE, None))):
        assert call(**kw) == NULL, kw
    for kw in (dict(data=(FAKE, MISALIGNED)), dict(summaries=(MISALIGNED, FAKE)), dict(src=FAKE + 2), dict(dst=FAKE + 1)):
        assert call(**kw) == ALIGN, kw
    assert call(n=0, data=None, src=None) == OK and call(layers=0, data=None) == OK


def test_summarize_validates_first(L):
    def call(c=None, b=None, summary=FAKE):
        return L.q4_kv_summarize(c or cache(), b or batch(), summary, None)

    assert L.q4_kv_summarize(None, batch(), FAKE, None) == NULL and L.q4_kv_summarize(cache(), None, FAKE, None) == NULL
    for kw in BAD_CACHES:
        assert call(c=cache(**kw)) == RANGE, kw
    for kw in BAD_BATCHES:
        assert call(b=batch(**kw)) == RANGE, kw
    for kw in (dict(summary=None), dict(c=cache(data=None)), dict(b=batch(lengths=None))):
        assert call(**kw) == NULL, kw
    assert call(summary=MISALIGNED) == ALIGN
    assert call(b=batch(rows=0), summary=None) == OK
    assert L.q4_kv_summary_bytes(7, 3, 128) == 7 * 3 * 2 * 128 and L.q4_kv_summary_bytes(7, 3, 96) == 0


def test_select_validates_first(L):
    def call(c=None, b=None, summary=FAKE, q=FAKE, hq=4, keep=4, first=1, recent=2, chosen=FAKE, ws=FAKE, nbytes=BIG):
        return L.q4_kv_select(c or cache(), b or batch(), summary, q, hq, keep, first, recent, chosen, ws, nbytes, None)

    for kw in BAD_CACHES:
        assert call(c=cache(**kw)) == RANGE, kw
    for kw in BAD_BATCHES:
        assert call(b=batch(**kw)) == RANGE, kw
    for kw in (dict(hq=3), dict(hq=130), dict(keep=0), dict(keep=2**16 + 1), dict(first=-1), dict(recent=-1), dict(first=3),
               dict(recent=2**62, first=2**62)):
        assert call(**kw) == RANGE, kw
    for kw in (dict(summary=None), dict(q=None), dict(chosen=None), dict(ws=None), dict(c=cache(data=None)), dict(b=batch(block_table=None))):
        assert call(**kw) == NULL, kw
    for kw in (dict(summary=MISALIGNED), dict(q=MISALIGNED), dict(chosen=FAKE + 2), dict(ws=MISALIGNED)):
        assert call(**kw) == ALIGN, kw
    need = L.q4_kv_select_workspace(cache(), batch(max_length=65))
    assert need == 2 * 2 * 3 * 4 // 16 * 16 + (16 if 2 * 2 * 3 * 4 % 16 else 0)
    assert call(b=batch(max_length=65), nbytes=need - 1) == RANGE
    assert L.q4_kv_select_workspace(cache(), batch(rows=0)) == 0
    assert call(b=batch(batch=0, rows=0), q=None, ws=None) == OK


def test_attention_blocks_validates_first(L):
    def call(c=None, b=None, q=FAKE, hq=4, chosen=FAKE, keep=4, scale=0.1, out=FAKE, dtype=1, ws=FAKE, nbytes=BIG):
        return L.q4_kv_attention_blocks(c or cache(), b or batch(), q, hq, chosen, keep, scale, out, dtype, ws, nbytes, None)

    for kw in BAD_CACHES:
        assert call(c=cache(**kw)) == RANGE, kw
    for kw in BAD_BATCHES:
        assert call(b=batch(**kw)) == RANGE, kw
    for kw in (dict(hq=5), dict(hq=130), dict(scale=float("nan")), dict(keep=0), dict(keep=2**16 + 1), dict(dtype=2)):
        assert call(**kw) == RANGE, kw
    for kw in (dict(q=None), dict(out=None), dict(chosen=None), dict(c=cache(data=None)), dict(b=batch(lengths=None))):
        assert call(**kw) == NULL, kw
    for kw in (dict(q=MISALIGNED), dict(out=MISALIGNED), dict(ws=MISALIGNED), dict(chosen=FAKE + 2)):
        assert call(**kw) == ALIGN, kw
    need = L.q4_kv_attention_blocks_workspace(cache(), batch(), 4, 256)   # few rows, many blocks: split
    assert need > 0 and need % 16 == 0
    assert call(keep=256, ws=None, nbytes=0) == NULL and call(keep=256, nbytes=need - 1) == RANGE
    assert L.q4_kv_attention_blocks_workspace(cache(), batch(), 4, 4) == 0
    assert call(b=batch(rows=0), q=None, out=None, ws=None) == OK


PROGRAM = r"""
#include <stdio.h>
#include "q4_search.h"

int main(void) {
    q4_kv_cache c = {0, 16, 2, 64};
    q4_kv_batch b = {0, 0, 0, 4, 2, 2, 1, 64};
    int bad = 0;
    if (q4_kv_summary_bytes(16, 2, 64) != (size_t)16 * 2 * 2 * 64) bad |= 1;
    if (q4_kv_select(&c, &b, 0, 0, 4, 4, 1, 2, 0, 0, 0, 0) != Q4_ERR_NULL) bad |= 2;
    if (q4_kv_copy_blocks(&c, 0, 0, 0, 0, 0, 0, 0) != Q4_OK) bad |= 4;
    if (q4_beam_select(0, 1, 1, 1, 0, 0, 0, 200, 0, 0, 0, 0, 0, 0) != Q4_ERR_RANGE) bad |= 8;
    printf("%d\n", bad);
    return bad;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
def test_plain_c_program_uses_the_header(L, tmp_path):
    src, exe = tmp_path / "consumer.c", tmp_path / "consumer"
    src.write_text(PROGRAM)
    libdir = os.path.dirname(q4.library_path())
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", f"-I{os.path.join(ROOT, 'include')}",
                    str(src), "-o", str(exe), f"-L{libdir}", "-l:libq4amd.so", f"-Wl,-rpath,{libdir}"], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, (out.returncode, out.stdout, out.stderr)
