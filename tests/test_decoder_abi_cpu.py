"""C-ABI checks of the decoder operators that need no GPU: every function that
include/q4_decoder.h declares is exported, sizes come out as documented, and
bad arguments are refused before the HIP runtime is touched.  Fake device
addresses are never dereferenced: only calls that fail validation, or have
nothing to do, are made."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

import q4_weight_only_amd as q4
from q4_weight_only_amd import _decoder as D

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "q4_decoder.h")
FAKE, MISALIGNED = 0x10000, 0x10004
OK, NULL, ALIGN, RANGE = 0, 1, 3, 6


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(q4.library_path()):
        import sys
        subprocess.run([sys.executable, "-m", "q4_weight_only_amd.build"], check=True)
    return D.decoder_lib()


def test_every_declared_function_is_exported(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(q4_\w+)\s*\(", text)))
    assert names == sorted(D.DECODER_EXPORTS)
    for name in names:
        assert hasattr(L, name), name
    assert q4.status_str(RANGE) != "unknown status"


@pytest.mark.parametrize("nb,h,d", [(1, 1, 64), (7, 8, 128), (2**24, 256, 128)])
def test_cache_bytes(L, nb, h, d):
    assert q4.kv_cache_bytes(nb, h, d) == nb * h * 2 * (32 * d + 1)


@pytest.mark.parametrize("nb,h,d", [(0, 8, 128), (2**24 + 1, 8, 128), (4, 0, 128), (4, 257, 128), (4, 8, 96), (4, 8, 256)])
def test_cache_bytes_invalid_is_zero(L, nb, h, d):
    assert q4.kv_cache_bytes(nb, h, d) == 0


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


def test_append_validates_first(L):
    def call(c=None, b=None, q=FAKE, qs=256, hq=4, k=FAKE, ks=128, v=FAKE, vs=128, dtype=0, rope=FAKE, positions=64,
             rot=64, inter=0, out=FAKE):
        return L.q4_kv_append(c or cache(), b or batch(), q, qs, hq, k, ks, v, vs, dtype, rope, positions, rot, inter,
                              out, None)

    assert L.q4_kv_append(None, batch(), FAKE, 256, 4, FAKE, 128, FAKE, 128, 0, FAKE, 64, 64, 0, FAKE, None) == NULL
    assert L.q4_kv_append(cache(), None, FAKE, 256, 4, FAKE, 128, FAKE, 128, 0, FAKE, 64, 64, 0, FAKE, None) == NULL
    for kw in BAD_CACHES:
        assert call(c=cache(**kw)) == RANGE, kw
    for kw in BAD_BATCHES:
        assert call(b=batch(**kw)) == RANGE, kw
    for kw in (dict(hq=0), dict(hq=3), dict(hq=2 * 65, qs=2 * 65 * 64), dict(dtype=2), dict(dtype=-1), dict(inter=2), dict(rot=-32),
               dict(rot=96), dict(rot=48), dict(positions=0), dict(positions=2**25 + 1), dict(qs=252), dict(ks=124),
               dict(vs=64)):
        assert call(**kw) == RANGE, kw
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(rope=None), dict(out=None), dict(c=cache(data=None)),
               dict(b=batch(block_table=None)), dict(b=batch(lengths=None))):
        assert call(**kw) == NULL, kw
    for kw in (dict(q=MISALIGNED), dict(k=MISALIGNED), dict(v=MISALIGNED), dict(rope=MISALIGNED), dict(out=MISALIGNED),
               dict(c=cache(data=MISALIGNED)), dict(b=batch(lengths=FAKE + 2)), dict(b=batch(cu_rows=FAKE + 1)),
               dict(qs=258), dict(ks=130), dict(vs=131), dict(dtype=1, qs=260)):
        assert call(**kw) == ALIGN, kw
    assert call(b=batch(batch=0, rows=0), q=None) == OK
    assert call(b=batch(rows=0), q=None) == OK


def test_attention_validates_first(L):
    def call(c=None, b=None, q=FAKE, hq=4, scale=0.1, window=0, out=FAKE, dtype=1, ws=FAKE, nbytes=2**40):
        return L.q4_kv_attention(c or cache(), b or batch(), q, hq, scale, window, out, dtype, ws, nbytes, None)

    for kw in BAD_CACHES:
        assert call(c=cache(**kw)) == RANGE, kw
    for kw in BAD_BATCHES:
        assert call(b=batch(**kw)) == RANGE, kw
    for kw in (dict(hq=5), dict(hq=130), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
               dict(window=2**30 + 1), dict(dtype=2)):
        assert call(**kw) == RANGE, kw
    for kw in (dict(q=None), dict(out=None), dict(c=cache(data=None)), dict(b=batch(lengths=None))):
        assert call(**kw) == NULL, kw
    for kw in (dict(q=MISALIGNED), dict(out=MISALIGNED), dict(ws=MISALIGNED)):
        assert call(**kw) == ALIGN, kw
    # a long cache is split, which needs a workspace
    long = batch(table_width=4096, max_length=131072)
    need = L.q4_kv_attention_workspace(cache(), long, 4)
    assert need > 0 and need % 16 == 0
    assert call(b=long, ws=None, nbytes=0) == NULL
    assert call(b=long, nbytes=need - 1) == RANGE
    assert L.q4_kv_attention_workspace(cache(), batch(batch=0, rows=0), 4) == 0
    assert L.q4_kv_attention_workspace(cache(head_dim=80), long, 4) == 0
    assert call(b=batch(rows=0), q=None, out=None, ws=None) == OK


def test_norm_validates_first(L):
    def call(res=FAKE, rd=0, y=FAKE, yd=0, m=4, c=64, w=FAKE, post=None, gate=None, grows=0, scale=1.0, mod=None,
             mrows=0, eps=1e-5, rout=FAKE, x=FAKE, xd=1):
        return L.q4_add_rmsnorm(res, rd, y, yd, m, c, w, post, gate, grows, scale, mod, mrows, eps, rout, x, xd, None)

    for kw in (dict(rd=2), dict(yd=-1), dict(xd=2), dict(m=-1), dict(m=2**20 + 1), dict(c=0), dict(c=48), dict(c=2**20 + 32),
               dict(eps=-1.0), dict(eps=float("nan")), dict(scale=float("inf")), dict(y=None, post=FAKE),
               dict(y=None, gate=FAKE, grows=1), dict(gate=FAKE, grows=3), dict(gate=FAKE, grows=0), dict(gate=FAKE, grows=8),
               dict(mod=FAKE, mrows=3)):
        assert call(**kw) == RANGE, kw
    for kw in (dict(res=None), dict(w=None), dict(x=None), dict(rout=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(res=MISALIGNED), dict(y=MISALIGNED), dict(w=MISALIGNED), dict(post=MISALIGNED), dict(x=MISALIGNED),
               dict(gate=MISALIGNED, grows=1), dict(mod=MISALIGNED, mrows=4), dict(rout=MISALIGNED)):
        assert call(**kw) == ALIGN, kw
    assert call(m=0, res=None) == OK


def test_logits_validates_first(L):
    def call(z=FAKE, m=2, v=100, h=None, cu=None, nh=0, pl=None, rho=None, fr=None, pr=None, bi=None, bv=None, cb=None,
             nb=0, mask=None, out=FAKE):
        return L.q4_logits_adjust(z, m, v, h, cu, nh, pl, rho, fr, pr, bi, bv, cb, nb, mask, out, None)

    for kw in (dict(m=-1), dict(m=65536), dict(v=0), dict(v=2**24 + 1), dict(nh=-1), dict(nh=2**31), dict(nb=-1), dict(nb=2**31)):
        assert call(**kw) == RANGE, kw
    for kw in (dict(z=None), dict(out=None), dict(nh=3), dict(nh=3, h=FAKE), dict(nb=3), dict(nb=3, bi=FAKE, bv=FAKE)):
        assert call(**kw) == NULL, kw
    for kw in (dict(z=MISALIGNED), dict(out=MISALIGNED), dict(mask=FAKE + 2), dict(rho=FAKE + 1)):
        assert call(**kw) == ALIGN, kw
    assert call(m=0, z=None) == OK


PROGRAM = r"""
#include <stdio.h>
#include "q4_decoder.h"

int main(void) {
    q4_kv_cache c = {0, 16, 2, 64};
    q4_kv_batch b = {0, 0, 0, 4, 2, 2, 1, 64};
    int bad = 0;
    if (q4_kv_cache_bytes(16, 2, 64) != (size_t)16 * 2 * 2 * (Q4_KV_BLOCK * 64 + 1)) bad |= 1;
    if (q4_kv_attention(&c, &b, 0, 4, 0.125f, 0, 0, Q4_BF16, 0, 0, 0) != Q4_ERR_NULL) bad |= 2;
    if (q4_add_rmsnorm(0, Q4_F32, 0, Q4_F32, 0, 64, 0, 0, 0, 0, 1.0f, 0, 0, 1e-5f, 0, 0, Q4_BF16, 0) != Q4_OK) bad |= 4;
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
