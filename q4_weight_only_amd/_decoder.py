"""Python interface of libq4amd's decoder operators (include/q4_decoder.h).

The computation runs in the HIP library on the current stream of the tensors'
device; the calls go through the native binding csrc/decoder_binding.cpp, which
checks the tensors and makes the outputs.  A missing build raises.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import _binding as B

KV_BLOCK = 32
DECODER_EXPORTS = ("q4_kv_cache_bytes", "q4_kv_append", "q4_kv_attention_workspace", "q4_kv_attention",
                   "q4_kv_attention_plan", "q4_add_rmsnorm", "q4_logits_adjust")

_lib = None
_native = None
_lock = threading.Lock()


class _Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_blocks", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class _Batch(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("cu_rows", ctypes.c_void_p),
                ("table_width", ctypes.c_int64), ("batch", ctypes.c_int64), ("rows", ctypes.c_int64),
                ("max_rows", ctypes.c_int64), ("max_length", ctypes.c_int64)]


def decoder_lib() -> ctypes.CDLL:
    """libq4amd with the decoder operators' argument types set."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                L = B.lib()
                vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
                L.q4_kv_cache_bytes.argtypes = [i64, i64, i64]
                L.q4_kv_cache_bytes.restype = ctypes.c_size_t
                L.q4_kv_append.argtypes = [vp, vp, vp, i64, i64, vp, i64, vp, i64, i32, vp, i64, i64, i32, vp, vp]
                L.q4_kv_append.restype = i32
                L.q4_kv_attention_workspace.argtypes = [vp, vp, i64]
                L.q4_kv_attention_workspace.restype = ctypes.c_size_t
                L.q4_kv_attention.argtypes = [vp, vp, vp, i64, f32, i64, vp, i32, vp, ctypes.c_size_t, vp]
                L.q4_kv_attention.restype = i32
                L.q4_kv_attention_plan.argtypes = [vp, vp, i64, i64, vp, vp, vp]
                L.q4_kv_attention_plan.restype = i32
                L.q4_add_rmsnorm.argtypes = [vp, i32, vp, i32, i64, i64, vp, vp, vp, i64, f32, vp, i64, f32, vp, vp,
                                             i32, vp]
                L.q4_add_rmsnorm.restype = i32
                L.q4_logits_adjust.argtypes = [vp, i64, i64, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp]
                L.q4_logits_adjust.restype = i32
                _lib = L
    return _lib


def _load():
    """The native binding (built with the library); raises if it has not been."""
    global _native
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_q4decoder.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m q4_weight_only_amd.build` "
                           "(or __graft_entry__.build()) first")
    B.lib()
    from . import _q4decoder

    _q4decoder.set_error(B.Q4Error)
    _native = _q4decoder
    return _native


# ------------------------------------------------------------------ cache
def kv_cache_bytes(num_blocks: int, kv_heads: int, head_dim: int) -> int:
    return int(decoder_lib().q4_kv_cache_bytes(int(num_blocks), int(kv_heads), int(head_dim)))


class KVCache:
    """A paged 8-bit cache of keys and values of one layer: `num_blocks` blocks
    of 32 tokens of kv_heads * head_dim, in a uint8 device tensor `data` of
    kv_cache_bytes() bytes (KVCache.empty allocates one)."""

    __slots__ = ("data", "num_blocks", "kv_heads", "head_dim")

    def __init__(self, data: torch.Tensor, num_blocks: int, kv_heads: int, head_dim: int):
        if not (1 <= num_blocks <= 1 << 24 and 1 <= kv_heads <= 256 and head_dim in (64, 128)):
            raise ValueError("need 1..2^24 blocks, 1..256 kv heads and a head_dim of 64 or 128")
        if not isinstance(data, torch.Tensor) or not data.is_cuda or data.dtype != torch.uint8:
            raise ValueError("data must be a uint8 CUDA/HIP tensor")
        if data.numel() != num_blocks * kv_heads * 2 * (KV_BLOCK * head_dim + 1) or not data.is_contiguous():
            raise ValueError(f"data must hold {kv_cache_bytes(num_blocks, kv_heads, head_dim)} contiguous bytes")
        self.data, self.num_blocks, self.kv_heads, self.head_dim = data, num_blocks, kv_heads, head_dim

    @classmethod
    def empty(cls, num_blocks: int, kv_heads: int, head_dim: int, device="cuda") -> "KVCache":
        """A cache of zeros."""
        nbytes = kv_cache_bytes(num_blocks, kv_heads, head_dim)
        return cls(torch.zeros(nbytes, dtype=torch.uint8, device=device), num_blocks, kv_heads, head_dim)

    @property
    def device(self) -> torch.device:
        return self.data.device

    def planes(self):
        """(codes [blocks, kv_heads, 2, 32 * head_dim] uint8, exponents
        [blocks, kv_heads, 2] int8), views of the data."""
        n = self.num_blocks * self.kv_heads * 2 * KV_BLOCK * self.head_dim
        return (self.data[:n].view(self.num_blocks, self.kv_heads, 2, KV_BLOCK * self.head_dim),
                self.data[n:].view(torch.int8).view(self.num_blocks, self.kv_heads, 2))


def rope_table(positions: int, rot: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """fp32 [positions, rot / 2, 2]: cosine and sine of position * theta^(-2 i / rot),
    computed in 64 bits."""
    freq = float(theta) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.stack((angle.cos(), angle.sin()), -1).float().to(device)


def kv_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: KVCache, block_table: torch.Tensor,
              lengths: torch.Tensor, rope: torch.Tensor | None, cu_rows: torch.Tensor | None = None, *,
              max_rows: int | None = None, interleaved: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotate q and k by their positions, append k and v to the cache, return
    the rotated q [rows, q_heads * D] in bf16.

    q [rows, q_heads * D], k and v [rows, kv_heads * D] are all fp32 or all
    bf16; their rows may lie apart (slices of a wider tensor).  lengths int32
    [batch] counts the appended tokens; cu_rows int32 [batch + 1] bounds the
    sequences' rows (None: as many for each); max_rows is the most rows of a
    sequence, which the launch is shaped for.  rope is rope_table() or None
    for no rotation; `interleaved` pairs dimensions 2 i and 2 i + 1 instead of
    i and i + rot / 2."""
    return (_native or _load()).kv_append(q, k, v, cache.data, cache.num_blocks, cache.kv_heads, cache.head_dim,
                                          block_table, lengths, cu_rows, max_rows, None, rope, interleaved, out)


def kv_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, lengths: torch.Tensor,
                 cu_rows: torch.Tensor | None = None, *, max_rows: int | None = None, max_length: int | None = None,
                 scale: float | None = None, window: int = 0, out: torch.Tensor | None = None,
                 dtype: torch.dtype = torch.bfloat16, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention of the rows q [rows, q_heads * D] (bf16, kv_append's
    result) over the cache: [rows, q_heads * D] in `dtype` (bf16 or fp32).

    lengths and cu_rows as for kv_append; max_rows and max_length, the most
    rows and the largest length, shape the launch (None: what the tensors'
    shapes allow, which costs time where the table is much wider than the
    longest sequence).  scale: of q . k (None: head_dim ** -0.5); window > 0: the
    last `window` tokens only.  A row without tokens gives 0.  workspace: a
    uint8 device tensor kept by the caller, of kv_attention_workspace() bytes;
    None takes one from torch's allocator for the call."""
    return (_native or _load()).kv_attention(q, cache.data, cache.num_blocks, cache.kv_heads, cache.head_dim, block_table,
                                             lengths, cu_rows, max_rows, max_length, scale, window, out, dtype, workspace)


def kv_attention_workspace(cache: KVCache, block_table: torch.Tensor, rows: int, q_heads: int, *, max_rows: int,
                           max_length: int) -> int:
    """Bytes of workspace of kv_attention for these sizes."""
    c, bt = _shapes(cache, block_table, rows, max_rows, max_length)
    return int(decoder_lib().q4_kv_attention_workspace(ctypes.byref(c), ctypes.byref(bt), int(q_heads)))


def kv_attention_plan(cache: KVCache, block_table: torch.Tensor, rows: int, q_heads: int, *, max_rows: int,
                      max_length: int, window: int = 0) -> tuple[int, int, int]:
    """(rows, waves, parts): the launch that kv_attention takes for these sizes:
    rows (times heads of a kv head) and waves of a workgroup, and into how many
    parts the tokens of its rows are divided."""
    c, bt = _shapes(cache, block_table, rows, max_rows, max_length)
    out = (ctypes.c_int32 * 3)()
    at = [ctypes.addressof(out) + 4 * i for i in range(3)]
    B._check(decoder_lib().q4_kv_attention_plan(ctypes.byref(c), ctypes.byref(bt), int(q_heads), int(window), *at),
             "q4_kv_attention_plan")
    return tuple(out)


def _shapes(cache: KVCache, block_table: torch.Tensor, rows: int, max_rows: int, max_length: int):
    """The sizes of a call, without its memory."""
    n, width = block_table.shape
    return (_Cache(None, cache.num_blocks, cache.kv_heads, cache.head_dim),
            _Batch(None, None, 4, width, n, int(rows), max(1, int(max_rows)), max(1, int(max_length))))


def add_rmsnorm(residual: torch.Tensor, weight: torch.Tensor, y: torch.Tensor | None = None, *,
                post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None, scale: float = 1.0,
                modulation: torch.Tensor | None = None, eps: float = 1e-5, dtype: torch.dtype = torch.bfloat16,
                residual_out: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """(r', x): r' = residual + scale * gate * norm(y, post_weight), each part
    where it is given, and x = norm(r', weight) * (1 + modulation) in `dtype`.

    residual and y are [M, C] in fp32 or bf16, r' has the residual's type
    (residual_out may be the residual itself); weights are fp32 [C], gate and
    modulation fp32 [C] or [rows, C] with rows dividing M: a row for each run
    of M / rows rows.  Without y, r' is the residual and x its norm."""
    return (_native or _load()).add_rmsnorm(residual, weight, y, post_weight, gate, scale, modulation, eps, dtype,
                                            residual_out, out)


def logits_adjust(logits: torch.Tensor, *, history: torch.Tensor | None = None, cu_history: torch.Tensor | None = None,
                  prompt_lengths: torch.Tensor | None = None, repetition: torch.Tensor | None = None,
                  frequency: torch.Tensor | None = None, presence: torch.Tensor | None = None,
                  bias_ids: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                  cu_bias: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Logits [M, V] (fp32) with penalties, biases and a mask applied; `out`
    may be the logits themselves.

    history int32 holds the rows' token ids one after the other, cu_history
    int32 [M + 1] their bounds, prompt_lengths int32 [M] how many of a row's
    ids are its prompt (counted by repetition alone); repetition, frequency
    and presence are fp32 [M].  bias_ids int32, bias fp32 and cu_bias int32
    [M + 1] are the rows' biases in the same form.  mask int32 [M, ceil(V / 32)]:
    bit t % 32 of word t / 32 is set where token t is allowed."""
    return (_native or _load()).logits_adjust(logits, history, cu_history, prompt_lengths, repetition, frequency, presence,
                                              bias_ids, bias, cu_bias, mask, out)
