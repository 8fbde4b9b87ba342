"""Python binding of the attention operators (``include/lora_kv.h``): argument
marshalling only.

Everything between the q/k/v projections and the o projection of a mixed
multi-LoRA batch: block tables and slot maps (``lora_kv_build``), rotary
positions (``lora_rope``), the paged 4-bit cache (``lora_kv_append``,
``lora_kv_gather``), attention over it (``lora_kv_attend``) and over whole
prompts (``lora_prompt_attend``).  The steps run in liblora.so's HIP kernels;
this module checks tensors, fills the C structs and raises on a non-zero
status.  All tensors of a call must be on one GPU; the call runs on that GPU's
current stream, or on ``stream``.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import lora

ROPE_HALF, ROPE_INTERLEAVED = 0, 1
SCALING_NONE, SCALING_LINEAR, SCALING_NTK, SCALING_YARN, SCALING_BANDS = range(5)
COUNT_TOKENS, COUNT_NEW_BLOCKS, COUNT_ITEMS, COUNT_PARTS, COUNT_CHUNK, COUNT_FLAGS = 0, 1, 2, 3, 4, 8
FLAG_LENGTH, FLAG_TOKENS, FLAG_FREE_LIST, FLAG_BLOCK_RANGE, FLAG_NONFINITE, FLAG_BATCH = 1, 2, 4, 8, 16, 32
N_COUNTS = 16
MAX_SEQS = 1 << 16
EXPORTS = ("lora_kv_block_bytes", "lora_kv_batch_size", "lora_kv_batch_init", "lora_kv_build", "lora_rope_frequencies",
           "lora_rope", "lora_kv_append", "lora_kv_gather", "lora_kv_workspace_size", "lora_kv_attend",
           "lora_prompt_attend")

_vp, _i32, _i64, _f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double


class lora_heads_t(ctypes.Structure):
    _fields_ = [("data", _vp), ("token_stride", _i64), ("head_stride", _i64), ("heads", _i32)]


class lora_kv_cache_t(ctypes.Structure):
    _fields_ = [("base", _vp), ("block_stride", _i64), ("num_blocks", _i32), ("block_tokens", _i32),
                ("num_kv_heads", _i32), ("head_dim", _i32)]


class lora_kv_batch_t(ctypes.Structure):
    _fields_ = [("max_tokens", _i32), ("max_seqs", _i32), ("num_q_heads", _i32), ("num_kv_heads", _i32),
                ("head_dim", _i32), ("q_indptr", _vp), ("kv_len", _vp), ("token_seq", _vp), ("positions", _vp),
                ("slots", _vp), ("counts", _vp), ("plan", _vp)]


class lora_rope_t(ctypes.Structure):
    _fields_ = [("inv_freq", _vp), ("rot_dim", _i32), ("layout", _i32), ("scale", _f64)]


_bound = None


def lib():
    """liblora.so with this module's functions declared."""
    global _bound
    if _bound is None:
        L, P = lora.lib(), ctypes.POINTER
        heads, sz = P(lora_heads_t), ctypes.c_size_t
        sigs = {
            "lora_kv_block_bytes": (sz, [_i32] * 3),
            "lora_kv_batch_size": (sz, [_i32] * 5),
            "lora_kv_batch_init": (_i32, [_vp, sz] + [_i32] * 5 + [P(lora_kv_batch_t)]),
            "lora_kv_build": (_i32, [_vp, _vp, _i32, _i32, _vp, _i64, _i32, _vp, _i32, _i32, _i32, P(lora_kv_batch_t), _vp]),
            "lora_rope_frequencies": (_i32, [_i32, _f64, _i32, _f64, _f64, _f64, _f64, _vp, P(_f64)]),
            "lora_rope": (_i32, [heads, heads, heads, heads, _vp, _i32, _i32, _i32, P(lora_rope_t), _vp]),
            "lora_kv_append": (_i32, [heads, heads, heads, heads, _vp, _vp, _i32, _i32, P(lora_rope_t),
                                      P(lora_kv_cache_t), _vp, _vp]),
            "lora_kv_gather": (_i32, [P(lora_kv_cache_t), _vp, _i32, heads, heads, _i32, _vp]),
            "lora_kv_workspace_size": (sz, [P(lora_kv_batch_t)]),
            "lora_kv_attend": (_i32, [heads, heads, _i32, _i32, _i32, P(lora_kv_batch_t), _vp, _i64, _i32,
                                      P(lora_kv_cache_t), ctypes.c_float, _vp, sz, _vp]),
            "lora_prompt_attend": (_i32, [heads, heads, heads, heads, _vp, _i32, _i32, _i32, _i32, ctypes.c_float, _vp]),
        }
        for name, (res, args) in sigs.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _bound = L
    return _bound


# ------------------------------------------------------------------ checking
def _heads(t: torch.Tensor, name: str) -> lora_heads_t:
    if t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] > 1):
        raise ValueError(f"{name} must have shape (tokens, heads, head_dim) with contiguous dims")
    return lora_heads_t(t.data_ptr(), t.stride(0), t.stride(1), t.shape[1])


def _ints(t: torch.Tensor, name: str, dim: int = 1) -> None:
    if t.dtype != torch.int32 or t.dim() != dim or (t.numel() and t.stride(-1) != 1):
        raise ValueError(f"{name} must be int32 with {dim} dimension(s), its last one contiguous")


def _same_type(*named) -> int:
    first = named[0][1].dtype
    for name, t in named[1:]:
        if t.dtype != first:
            raise ValueError(f"{name} has type {t.dtype}, not {first}")
    return lora.dtype_code(first)


class _On:
    """The device of a call's tensors, made current, and its stream."""

    def __init__(self, stream, *tensors):
        self.dev = dev = tensors[0].device
        for t in tensors:
            if t.device != dev:
                raise ValueError(f"tensors of one call on {dev} and {t.device}")
        if dev.type != "cuda":
            raise ValueError(f"the attention operators need GPU tensors, got {dev}")
        if stream is not None and stream.device != dev:
            raise ValueError(f"a stream of {stream.device} for tensors on {dev}")
        self.stream = stream

    def call(self, name: str, *args) -> None:
        if torch.cuda.current_device() == self.dev.index:
            st = self._run(name, args)
        else:
            with torch.cuda.device(self.dev):
                st = self._run(name, args)
        if st != 0:
            raise lora.LoraError(name, st)

    def _run(self, name, args):
        s = self.stream if self.stream is not None else torch.cuda.current_stream(self.dev)
        return getattr(lib(), name)(*args, s.cuda_stream)


# ------------------------------------------------------------------ handles
def block_bytes(block_tokens: int, num_kv_heads: int, head_dim: int) -> int:
    """Bytes of one cache block (0: unsupported geometry)."""
    return int(lib().lora_kv_block_bytes(block_tokens, num_kv_heads, head_dim))


class Cache:
    """One layer's paged 4-bit cache over ``data``, a uint8 tensor (blocks,
    bytes per block), rows contiguous."""

    def __init__(self, data: torch.Tensor, block_tokens: int, num_kv_heads: int, head_dim: int):
        need = block_bytes(block_tokens, num_kv_heads, head_dim)
        if need == 0:
            raise ValueError("unsupported cache geometry")
        if data.dtype != torch.uint8 or data.dim() != 2 or data.shape[1] < need or data.stride(1) != 1:
            raise ValueError(f"cache data must be uint8 (blocks, at least {need} bytes), rows contiguous")
        self.data, self.block_tokens, self.num_blocks = data, block_tokens, data.shape[0]
        self.num_kv_heads, self.head_dim = num_kv_heads, head_dim
        stride = data.stride(0) if data.shape[0] > 1 else max(data.stride(0), need)
        self.c = lora_kv_cache_t(data.data_ptr(), stride, data.shape[0], block_tokens, num_kv_heads, head_dim)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def in_pool(cls, pool: "lora.Pool", block_tokens: int, num_kv_heads: int, head_dim: int) -> "Cache":
        """A cache whose blocks are the pages of an adapter pool: page ids are
        block ids, so adapters and cache share one pool and one allocator."""
        return cls(pool.base.view(torch.uint8), block_tokens, num_kv_heads, head_dim)


class Rope:
    """Rotary positions: inv_freq (float64, rot_dim/2 radians per position, on
    the GPU), layout and the scale of cos and sin."""

    def __init__(self, inv_freq: torch.Tensor, layout: int = ROPE_HALF, scale: float = 1.0):
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous float64 vector")
        self.inv_freq, self.rot_dim, self.layout, self.scale = inv_freq, 2 * inv_freq.numel(), layout, scale
        self.c = lora_rope_t(inv_freq.data_ptr(), self.rot_dim, layout, scale)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def scaled(cls, rot_dim: int, theta: float = 10000.0, scaling: int = SCALING_NONE, factor: float = 1.0,
               original: float = 0.0, low: float = 0.0, high: float = 0.0, layout: int = ROPE_HALF,
               device="cuda") -> "Rope":
        freq, scale = lora_rope_frequencies(rot_dim, theta, scaling, factor, original, low, high)
        return cls(torch.tensor(freq, dtype=torch.float64, device=device), layout, scale)


class Batch:
    """Device buffer of one step's batch: rows, positions, slots and the work
    plan, for up to max_tokens new tokens of max_seqs requests."""

    def __init__(self, max_tokens: int, max_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                 device="cuda"):
        L = lib()
        n = L.lora_kv_batch_size(max_tokens, max_seqs, num_q_heads, num_kv_heads, head_dim)
        if n == 0:
            raise ValueError("unsupported batch capacity or head geometry")
        # zeroed: a buffer that was never built must not look like one that was
        self.buf = torch.zeros(n, dtype=torch.uint8, device=device)
        self.c = lora_kv_batch_t()
        self.ref = ctypes.byref(self.c)
        st = L.lora_kv_batch_init(self.buf.data_ptr(), n, max_tokens, max_seqs, num_q_heads, num_kv_heads, head_dim, self.ref)
        if st != 0:
            raise lora.LoraError("lora_kv_batch_init", st)
        self.T = self.B = 0  # of the last build
        self._all = {name: self._view(name, size) for name, size in
                     (("q_indptr", max_seqs + 1), ("kv_len", max_seqs), ("token_seq", max_tokens),
                      ("positions", max_tokens), ("slots", max_tokens), ("counts", N_COUNTS))}

    def _view(self, field: str, n: int) -> torch.Tensor:
        off = getattr(self.c, field) - self.buf.data_ptr()
        return self.buf[off:off + 4 * n].view(torch.int32)

    q_indptr = property(lambda self: self._all["q_indptr"][:self.B + 1])
    kv_len = property(lambda self: self._all["kv_len"][:self.B])
    token_seq = property(lambda self: self._all["token_seq"][:self.T])
    positions = property(lambda self: self._all["positions"][:self.T])
    slots = property(lambda self: self._all["slots"][:self.T])
    counts = property(lambda self: self._all["counts"])
    flags = property(lambda self: self._all["counts"][COUNT_FLAGS:COUNT_FLAGS + 1])
    new_blocks = property(lambda self: self._all["counts"][COUNT_NEW_BLOCKS:COUNT_NEW_BLOCKS + 1])


def attend_workspace(batch: Batch) -> torch.Tensor:
    """Workspace of lora_kv_attend for a batch buffer (one serves every layer)."""
    n = lib().lora_kv_workspace_size(batch.ref)
    return torch.empty(n, dtype=torch.uint8, device=batch.buf.device)


# ------------------------------------------------------- the C entry points
def lora_rope_frequencies(rot_dim: int, theta: float = 10000.0, scaling: int = SCALING_NONE, factor: float = 1.0,
                          original: float = 0.0, low: float = 0.0, high: float = 0.0):
    """(frequencies as a list of floats, scale of cos and sin)."""
    out, scale = (_f64 * max(rot_dim // 2, 1))(), _f64()
    st = lib().lora_rope_frequencies(rot_dim, theta, scaling, factor, original, low, high, out, ctypes.byref(scale))
    if st != 0:
        raise lora.LoraError("lora_rope_frequencies", st)
    return list(out), scale.value


def lora_kv_build(ctx_len: torch.Tensor, new_len: torch.Tensor, T: int, block_table: torch.Tensor,
                  free_blocks: torch.Tensor, num_blocks: int, block_tokens: int, batch: Batch, stream=None) -> None:
    """Rows, positions, slots and plan of a step from request lengths; new
    blocks go from free_blocks into block_table (B, width)."""
    _ints(ctx_len, "ctx_len"), _ints(new_len, "new_len"), _ints(free_blocks, "free_blocks")
    _ints(block_table, "block_table", 2)
    B = ctx_len.numel()
    if new_len.numel() != B or block_table.shape[0] != B:
        raise ValueError("one length of each kind and one table row per request")
    on = _On(stream, ctx_len, new_len, block_table, free_blocks, batch.buf)
    on.call("lora_kv_build", ctx_len.data_ptr(), new_len.data_ptr(), B, T, block_table.data_ptr(),
            max(block_table.stride(0), block_table.shape[1]), block_table.shape[1], free_blocks.data_ptr(),
            free_blocks.numel(), num_blocks, block_tokens, batch.ref)
    batch.T, batch.B = T, B


def _rows(name: str, t: torch.Tensor, n: int) -> None:
    if t.shape[0] != n:
        raise ValueError(f"{name} has {t.shape[0]} rows, not {n}")


def lora_rope(q: Optional[torch.Tensor], q_out: Optional[torch.Tensor], k: Optional[torch.Tensor],
              k_out: Optional[torch.Tensor], positions: torch.Tensor, rope: Rope, stream=None) -> None:
    """Rotate q and k (T, heads, head_dim; either may be None) into q_out and
    k_out, which may be q and k."""
    _ints(positions, "positions")
    named = [(n, t) for n, t in (("q", q), ("q_out", q_out), ("k", k), ("k_out", k_out)) if t is not None]
    if not named or (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("q with q_out, k with k_out, or both")
    T, D = positions.numel(), named[0][1].shape[2]
    code = _same_type(*named)
    for n, t in named:
        _rows(n, t, T)
        if t.dim() != 3 or t.shape[2] != D:
            raise ValueError("q and k must have the same head_dim")
    ref = [None if t is None else ctypes.byref(_heads(t, n)) for n, t in (("q", q), ("q_out", q_out), ("k", k), ("k_out", k_out))]
    on = _On(stream, positions, rope.inv_freq, *(t for _, t in named))
    on.call("lora_rope", *ref, positions.data_ptr(), T, D, code, rope.ref)


def lora_kv_append(q: Optional[torch.Tensor], q_out: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                   positions: Optional[torch.Tensor], slots: torch.Tensor, rope: Optional[Rope], cache: Cache,
                   batch: Optional[Batch] = None, stream=None) -> None:
    """Rotate q into q_out and put rotated k, and v, into the cache at slots.
    rope None: no rotation.  batch: whose flags take FLAG_NONFINITE."""
    _ints(slots, "slots")
    T = slots.numel()
    if rope is None and q is not None:
        raise ValueError("q is only rotated: pass rope, or no q")
    if rope is not None and positions is None:
        raise ValueError("rope needs positions")
    if (q is None) != (q_out is None):
        raise ValueError("q with q_out")
    tensors = [slots, cache.data, k, v]
    named = [("k", k), ("v", v)]
    if q is not None:
        named += [("q", q), ("q_out", q_out)]
        tensors += [q, q_out]
    if positions is not None:
        _ints(positions, "positions")
        _rows("positions", positions, T)
        tensors.append(positions)
    if rope is not None:
        tensors.append(rope.inv_freq)
    code = _same_type(*named)
    for n, t in named:
        _rows(n, t, T)
        if t.dim() != 3 or t.shape[2] != cache.head_dim:
            raise ValueError(f"{n} must have the cache's head_dim {cache.head_dim}")
    on = _On(stream, *tensors)
    ref = lambda t, n: None if t is None else ctypes.byref(_heads(t, n))  # noqa: E731
    on.call("lora_kv_append", ref(q, "q"), ref(q_out, "q_out"), ref(k, "k"), ref(v, "v"),
            None if positions is None else positions.data_ptr(), slots.data_ptr(), T, code,
            None if rope is None else rope.ref, cache.ref, None if batch is None else batch.flags.data_ptr())


def lora_kv_gather(cache: Cache, slots: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor, stream=None) -> None:
    """The cached K and V at slots as values (n, kv heads, head_dim)."""
    _ints(slots, "slots")
    n = slots.numel()
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        _rows(name, t, n)
        if t.dim() != 3 or t.shape[2] != cache.head_dim:
            raise ValueError(f"{name} must have the cache's head_dim {cache.head_dim}")
    code = _same_type(("k_out", k_out), ("v_out", v_out))
    on = _On(stream, slots, cache.data, k_out, v_out)
    on.call("lora_kv_gather", cache.ref, slots.data_ptr(), n, ctypes.byref(_heads(k_out, "k_out")),
            ctypes.byref(_heads(v_out, "v_out")), code)


def lora_kv_attend(q: torch.Tensor, out: torch.Tensor, batch: Batch, block_table: torch.Tensor, cache: Cache,
                   scale: float, ws: torch.Tensor, stream=None) -> None:
    """Attention of the batch's rows q (T, heads, head_dim) over the cache."""
    _ints(block_table, "block_table", 2)
    for name, t in (("q", q), ("out", out)):
        _rows(name, t, batch.T)
        if t.dim() != 3 or t.shape[2] != cache.head_dim:
            raise ValueError(f"{name} must have the cache's head_dim {cache.head_dim}")
    _rows("block_table", block_table, batch.B)
    code = _same_type(("q", q), ("out", out))
    on = _On(stream, q, out, batch.buf, block_table, cache.data, ws)
    on.call("lora_kv_attend", ctypes.byref(_heads(q, "q")), ctypes.byref(_heads(out, "out")), batch.T, batch.B, code,
            batch.ref, block_table.data_ptr(), max(block_table.stride(0), block_table.shape[1]), block_table.shape[1],
            cache.ref, scale, ws.data_ptr(), ws.numel() * ws.element_size())


def lora_prompt_attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, indptr: torch.Tensor,
                       scale: float, stream=None) -> None:
    """Causal attention of packed prompts: rows indptr[i]..indptr[i+1]-1 of q,
    k, v and out (T, heads, head_dim) are prompt i."""
    _ints(indptr, "indptr")
    if indptr.numel() < 1:
        raise ValueError("indptr has one entry more than prompts")
    T = q.shape[0]
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        _rows(name, t, T)
        if t.dim() != 3 or t.shape[2] != q.shape[2]:
            raise ValueError("q, k, v and out must have the same head_dim")
    code = _same_type(("q", q), ("k", k), ("v", v), ("out", out))
    on = _On(stream, q, k, v, out, indptr)
    on.call("lora_prompt_attend", *(ctypes.byref(_heads(t, n)) for n, t in (("q", q), ("k", k), ("v", v), ("out", out))),
            indptr.data_ptr(), indptr.numel() - 1, T, q.shape[2], code, scale)
