"""ctypes binding of libq4amd's decoder operators (include/q4_decoder.h).

Argument marshalling only, as in _binding: the computation runs in the HIP
library on the current stream of the tensors' device, and a missing build
raises.
"""

from __future__ import annotations

import ctypes
import threading

import torch

from . import _binding as B

KV_BLOCK = 32
F32, BF16 = 0, 1
DECODER_EXPORTS = ("q4_kv_cache_bytes", "q4_kv_append", "q4_kv_attention_workspace", "q4_kv_attention",
                   "q4_add_rmsnorm", "q4_logits_adjust")

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}
_lib = None
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
                L.q4_add_rmsnorm.argtypes = [vp, i32, vp, i32, i64, i64, vp, vp, vp, i64, f32, vp, i64, f32, vp, vp,
                                             i32, vp]
                L.q4_add_rmsnorm.restype = i32
                L.q4_logits_adjust.argtypes = [vp, i64, i64, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp]
                L.q4_logits_adjust.restype = i32
                _lib = L
    return _lib


class _on:
    """The tensors' device made current for a call, where it is not already."""

    __slots__ = ("index", "before")

    def __init__(self, index: int):
        self.index = index

    def __enter__(self):
        self.before = torch.cuda.current_device()
        if self.before != self.index:
            torch.cuda.set_device(self.index)
        return torch.cuda.current_stream(self.index).cuda_stream

    def __exit__(self, *_):
        if self.before != self.index:
            torch.cuda.set_device(self.before)


def _tensor(t, name: str, dtype: torch.dtype, device: torch.device) -> int:
    """The address of a contiguous tensor of `dtype` on `device`."""
    if not isinstance(t, torch.Tensor) or t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA/HIP tensor on the inputs' device")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _activation(t, name: str) -> int:
    """The type code of an fp32 or bf16 device tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA/HIP tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


# ------------------------------------------------------------------ cache
def kv_cache_bytes(num_blocks: int, kv_heads: int, head_dim: int) -> int:
    return int(decoder_lib().q4_kv_cache_bytes(int(num_blocks), int(kv_heads), int(head_dim)))


class KVCache:
    """A paged 8-bit cache of keys and values of one layer: `num_blocks` blocks
    of 32 tokens of kv_heads * head_dim, in a uint8 device tensor `data` of
    kv_cache_bytes() bytes (KVCache.empty allocates one)."""

    __slots__ = ("data", "num_blocks", "kv_heads", "head_dim", "_c")

    def __init__(self, data: torch.Tensor, num_blocks: int, kv_heads: int, head_dim: int):
        nbytes = kv_cache_bytes(num_blocks, kv_heads, head_dim)
        if nbytes == 0:
            raise ValueError("need 1..2^24 blocks, 1..256 kv heads and a head_dim of 64 or 128")
        if not isinstance(data, torch.Tensor) or not data.is_cuda:
            raise ValueError("data must be a CUDA/HIP tensor")
        _tensor(data, "data", torch.uint8, data.device)
        if data.numel() != nbytes:
            raise ValueError(f"data must hold {nbytes} bytes")
        self.data, self.num_blocks, self.kv_heads, self.head_dim = data, int(num_blocks), int(kv_heads), int(head_dim)
        self._c = _Cache(data.data_ptr(), self.num_blocks, self.kv_heads, self.head_dim)

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


def _batch(block_table, lengths, cu_rows, rows: int, max_rows, max_length, device) -> _Batch:
    table = _tensor(block_table, "block_table", torch.int32, device)
    lens = _tensor(lengths, "lengths", torch.int32, device)
    if block_table.dim() != 2 or lengths.dim() != 1 or block_table.shape[0] != lengths.shape[0]:
        raise ValueError("block_table must be [batch, width] and lengths [batch]")
    n, width = block_table.shape
    cu = None
    if cu_rows is not None:
        cu = _tensor(cu_rows, "cu_rows", torch.int32, device)
        if cu_rows.dim() != 1 or cu_rows.shape[0] != n + 1:
            raise ValueError("cu_rows must be [batch + 1]")
    if max_rows is None:
        max_rows = rows if cu_rows is not None else max(1, rows // n) if n else 1
    return _Batch(table, lens, cu, width, n, rows, max(1, int(max_rows)),
                  width * KV_BLOCK if max_length is None else max(1, int(max_length)))


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
    dtype = _activation(q, "q")
    dev = q.device
    for t, name in ((k, "k"), (v, "v"), (q, "q")):
        if _activation(t, name) != dtype or t.device != dev:
            raise ValueError("q, k and v must share a type and a device")
        if t.dim() != 2 or t.shape[0] != q.shape[0] or (t.shape[0] > 0 and t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError(f"{name} must be [rows, heads * head_dim] with contiguous rows")
    if cache.data.device != dev:
        raise ValueError(f"the cache is on {cache.data.device}, not {dev}")
    rows, width = q.shape
    d, kv_width = cache.head_dim, cache.kv_heads * cache.head_dim
    if width % d or k.shape[1] != kv_width or v.shape[1] != kv_width:
        raise ValueError(f"need whole heads of {d}, and k and v [rows, {kv_width}]")
    bt = _batch(block_table, lengths, cu_rows, rows, max_rows, None, dev)
    rot = positions = 0
    table = None
    if rope is not None:
        table = _tensor(rope, "rope", torch.float32, dev)
        if rope.dim() != 3 or rope.shape[2] != 2:
            raise ValueError("rope must be [positions, rot / 2, 2]")
        positions, rot = rope.shape[0], 2 * rope.shape[1]
    if out is None:
        out = torch.empty((rows, width), dtype=torch.bfloat16, device=dev)
    dst = _tensor(out, "out", torch.bfloat16, dev)
    if tuple(out.shape) != (rows, width):
        raise ValueError("out has the wrong shape")
    one = rows <= 1   # the stride of a single row says nothing
    with _on(dev.index) as stream:
        B._check(decoder_lib().q4_kv_append(
            ctypes.addressof(cache._c), ctypes.addressof(bt), q.data_ptr(), width if one else q.stride(0), width // d,
            k.data_ptr(), kv_width if one else k.stride(0), v.data_ptr(), kv_width if one else v.stride(0), dtype,
            table, positions, rot, int(interleaved), dst, stream), "q4_kv_append")
    return out


def kv_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, lengths: torch.Tensor,
                 cu_rows: torch.Tensor | None = None, *, max_rows: int | None = None, max_length: int | None = None,
                 scale: float | None = None, window: int = 0, out: torch.Tensor | None = None,
                 dtype: torch.dtype = torch.bfloat16, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention of the rows q [rows, q_heads * D] (bf16, kv_append's
    result) over the cache: [rows, q_heads * D] in `dtype` (bf16 or fp32).

    lengths and cu_rows as for kv_append; max_rows and max_length, the most
    rows and the largest length, shape the launch (None: what the tensors'
    shapes allow).  scale: of q . k (None: head_dim ** -0.5); window > 0: the
    last `window` tokens only.  A row without tokens gives 0.  workspace: a
    uint8 device tensor kept by the caller, where it is large enough; else one
    is taken from torch's allocator for the call."""
    dev = q.device
    src = _tensor(q, "q", torch.bfloat16, dev)
    if q.dim() != 2 or q.shape[1] % cache.head_dim:
        raise ValueError(f"q must be [rows, heads * {cache.head_dim}]")
    if cache.data.device != dev:
        raise ValueError(f"the cache is on {cache.data.device}, not {dev}")
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("dtype must be torch.float32 or torch.bfloat16")
    heads = q.shape[1] // cache.head_dim
    bt = _batch(block_table, lengths, cu_rows, q.shape[0], max_rows, max_length, dev)
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=dev)
    dst = _tensor(out, "out", dtype, dev)
    if out.shape != q.shape:
        raise ValueError("out has the wrong shape")
    L = decoder_lib()
    pc, pb = ctypes.addressof(cache._c), ctypes.addressof(bt)
    need = L.q4_kv_attention_workspace(pc, pb, heads)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    elif _tensor(workspace, "workspace", torch.uint8, dev) and workspace.numel() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    with _on(dev.index) as stream:
        B._check(L.q4_kv_attention(
            pc, pb, src, heads, cache.head_dim ** -0.5 if scale is None else scale, int(window), dst, code,
            workspace.data_ptr() if workspace is not None else None,
            workspace.numel() if workspace is not None else 0, stream), "q4_kv_attention")
    return out


def kv_attention_workspace(cache: KVCache, block_table: torch.Tensor, rows: int, q_heads: int, *, max_rows: int,
                           max_length: int) -> int:
    """Bytes of workspace of kv_attention for these sizes."""
    n, width = block_table.shape
    bt = _Batch(None, None, 1, width, n, int(rows), max(1, int(max_rows)), max(1, int(max_length)))
    return int(decoder_lib().q4_kv_attention_workspace(ctypes.addressof(cache._c), ctypes.addressof(bt), int(q_heads)))


# ------------------------------------------------------------------ norms
def _shared_rows(t, name: str, m: int, c: int, device):
    """(address, rows) of a gate or modulation: [C], or [rows, C] with rows dividing M."""
    if t is None:
        return None, 0
    at = _tensor(t, name, torch.float32, device)
    if t.dim() not in (1, 2) or t.shape[-1] != c:
        raise ValueError(f"{name} must be [{c}] or [rows, {c}]")
    rows = t.shape[0] if t.dim() == 2 else 1
    if rows < 1 or (m and m % rows):
        raise ValueError(f"the rows of {name} must divide the {m} rows of the residual")
    return at, rows


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
    res_code = _activation(residual, "residual")
    dev = residual.device
    src = _tensor(residual, "residual", residual.dtype, dev)
    if residual.dim() != 2:
        raise ValueError("residual must be [M, C]")
    m, c = residual.shape
    w = _tensor(weight, "weight", torch.float32, dev)
    if tuple(weight.shape) != (c,):
        raise ValueError(f"weight must be [{c}]")
    x_code = _DTYPES.get(dtype)
    if x_code is None:
        raise ValueError("dtype must be torch.float32 or torch.bfloat16")
    post = None
    if post_weight is not None:
        post = _tensor(post_weight, "post_weight", torch.float32, dev)
        if tuple(post_weight.shape) != (c,):
            raise ValueError(f"post_weight must be [{c}]")
    at_gate, gate_rows = _shared_rows(gate, "gate", m, c, dev)
    at_mod, mod_rows = _shared_rows(modulation, "modulation", m, c, dev)
    y_code, at_y, at_res = F32, None, None
    if y is None:
        if post is not None or gate is not None or residual_out is not None:
            raise ValueError("post_weight, gate and residual_out need y")
        residual_out = residual
    else:
        y_code = _activation(y, "y")
        at_y = _tensor(y, "y", y.dtype, dev)
        if y.shape != residual.shape:
            raise ValueError("y must have the residual's shape")
        if residual_out is None:
            residual_out = torch.empty_like(residual)
        at_res = _tensor(residual_out, "residual_out", residual.dtype, dev)
        if residual_out.shape != residual.shape:
            raise ValueError("residual_out has the wrong shape")
    if out is None:
        out = torch.empty((m, c), dtype=dtype, device=dev)
    dst = _tensor(out, "out", dtype, dev)
    if tuple(out.shape) != (m, c):
        raise ValueError("out has the wrong shape")
    with _on(dev.index) as stream:
        B._check(decoder_lib().q4_add_rmsnorm(src, res_code, at_y, y_code, m, c, w, post, at_gate, gate_rows, scale,
                                              at_mod, mod_rows, eps, at_res, dst, x_code, stream), "q4_add_rmsnorm")
    return residual_out, out


# ----------------------------------------------------------------- logits
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
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise ValueError("logits must be a CUDA/HIP tensor")
    dev = logits.device
    src = _tensor(logits, "logits", torch.float32, dev)
    if logits.dim() != 2:
        raise ValueError("logits must be [M, V]")
    m, v = logits.shape

    def rows(t, name, dtype, n):
        if t is None:
            return None
        at = _tensor(t, name, dtype, dev)
        if t.dim() != 1 or t.shape[0] != n:
            raise ValueError(f"{name} must be [{n}]")
        return at

    i32, f32 = torch.int32, torch.float32
    if (history is None) != (cu_history is None):
        raise ValueError("history and cu_history go together")
    nh = history.shape[0] if history is not None else 0
    nb = bias_ids.shape[0] if bias_ids is not None else 0
    if not (bias is None) == (bias_ids is None) == (cu_bias is None):
        raise ValueError("bias, bias_ids and cu_bias go together")
    args = (rows(history, "history", i32, nh), rows(cu_history, "cu_history", i32, m + 1), nh,
            rows(prompt_lengths, "prompt_lengths", i32, m), rows(repetition, "repetition", f32, m),
            rows(frequency, "frequency", f32, m), rows(presence, "presence", f32, m),
            rows(bias_ids, "bias_ids", i32, nb), rows(bias, "bias", f32, nb), rows(cu_bias, "cu_bias", i32, m + 1), nb)
    at_mask = None
    if mask is not None:
        at_mask = _tensor(mask, "mask", i32, dev)
        if tuple(mask.shape) != (m, (v + 31) // 32):
            raise ValueError(f"mask must be [{m}, {(v + 31) // 32}]")
    if out is None:
        out = torch.empty_like(logits)
    dst = _tensor(out, "out", f32, dev)
    if out.shape != logits.shape:
        raise ValueError("out has the wrong shape")
    with _on(dev.index) as stream:
        B._check(decoder_lib().q4_logits_adjust(src, m, v, *args, at_mask, dst, stream), "q4_logits_adjust")
    return out
