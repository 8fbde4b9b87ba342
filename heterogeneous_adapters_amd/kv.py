"""Python binding of the attention operators (``include/lora_kv.h``): argument
marshalling only.

Everything between the q/k/v projections and the o projection of a mixed
multi-LoRA batch: block tables and slot maps (``lora_kv_build``), rotary
positions (``lora_rope``), the paged 4-bit cache (``lora_kv_append``,
``lora_kv_gather``), attention over it (``lora_kv_attend``), over it where
requests share their first tokens (``lora_kv_share``,
``lora_kv_attend_shared``) and over whole prompts (``lora_prompt_attend``).  The steps run in liblora.so's HIP kernels;
this module checks tensors, fills the C structs and raises on a non-zero
status.  All tensors of a call must be on one GPU; the call runs on that GPU's
current stream, or on ``stream``.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

from . import lora

ROPE_HALF, ROPE_INTERLEAVED = 0, 1
SCALING_NONE, SCALING_LINEAR, SCALING_NTK, SCALING_YARN, SCALING_BANDS = range(5)
COUNT_TOKENS, COUNT_NEW_BLOCKS, COUNT_ITEMS, COUNT_PARTS, COUNT_CHUNK, COUNT_MID, COUNT_WIDE = range(7)
COUNT_FLAGS = 8
FLAG_LENGTH, FLAG_TOKENS, FLAG_FREE_LIST, FLAG_BLOCK_RANGE, FLAG_NONFINITE, FLAG_BATCH, FLAG_GROUPS = 1, 2, 4, 8, 16, 32, 64
N_COUNTS = 16
MAX_SEQS = 1 << 16
EXPORTS = ("lora_kv_block_bytes", "lora_kv_batch_size", "lora_kv_batch_init", "lora_kv_build", "lora_rope_frequencies",
           "lora_rope", "lora_kv_append", "lora_kv_gather", "lora_kv_workspace_size", "lora_kv_attend",
           "lora_kv_share_size", "lora_kv_share_init", "lora_kv_share", "lora_kv_share_workspace_size",
           "lora_kv_attend_shared", "lora_prompt_attend")

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


class lora_kv_share_t(ctypes.Structure):
    _fields_ = [("max_groups", _i32), ("counts", _vp), ("plan", _vp)]


class lora_rope_t(ctypes.Structure):
    _fields_ = [("inv_freq", _vp), ("rot_dim", _i32), ("layout", _i32), ("scale", _f64)]


_bound = None


def lib() -> dict:
    """liblora.so's attention functions by name, declared."""
    global _bound
    if _bound is None:
        L, sz = lora.lib(), ctypes.c_size_t
        sigs = {
            "lora_kv_block_bytes": (sz, [_i32] * 3),
            "lora_kv_batch_size": (sz, [_i32] * 5),
            "lora_kv_batch_init": (_i32, [_vp, sz] + [_i32] * 5 + [_vp]),
            "lora_kv_build": (_i32, [_vp, _vp, _i32, _i32, _vp, _i64, _i32, _vp, _i32, _i32, _i32, _vp, _vp]),
            "lora_rope_frequencies": (_i32, [_i32, _f64, _i32, _f64, _f64, _f64, _f64, _vp, _vp]),
            "lora_rope": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp]),
            "lora_kv_append": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp]),
            "lora_kv_gather": (_i32, [_vp, _vp, _i32, _vp, _vp, _i32, _vp]),
            "lora_kv_workspace_size": (sz, [_vp]),
            "lora_kv_attend": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _i64, _i32, _vp, ctypes.c_float, _vp, sz, _vp]),
            "lora_kv_share_size": (sz, [_vp, _i32]),
            "lora_kv_share_init": (_i32, [_vp, sz, _vp, _i32, _vp]),
            "lora_kv_share": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp]),
            "lora_kv_share_workspace_size": (sz, [_vp, _vp]),
            "lora_kv_attend_shared": (_i32, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _i64, _i32, _vp,
                                             ctypes.c_float, _vp, sz, _vp]),
            "lora_prompt_attend": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, ctypes.c_float, _vp]),
        }
        fns = {}
        for name, (res, args) in sigs.items():
            fns[name] = f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _bound = fns
    return _bound


# ------------------------------------------------------------------ checking
# These run on every call of a decode step's many small launches, so they keep
# to the cheapest accessors, and descriptors are packed bytes, not ctypes
# structures.
_pack_heads = struct.Struct("@Pqqi4x").pack  # lora_heads_t
assert struct.calcsize("@Pqqi4x") == ctypes.sizeof(lora_heads_t)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_CODES = {torch.bfloat16: lora.LORA_DTYPE_BF16, torch.float32: lora.LORA_DTYPE_F32}


def _heads(t: torch.Tensor, name: str, rows: int, dim: int, dtype: torch.dtype) -> bytes:
    """Packed lora_heads_t of t (rows, heads, dim)."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (stride[2] != 1 and shape[2] > 1):
        raise ValueError(f"{name} must have shape (tokens, heads, head_dim) with contiguous dims")
    if shape[0] != rows:
        raise ValueError(f"{name} has {shape[0]} rows, not {rows}")
    if shape[2] != dim:
        raise ValueError(f"{name} must have the call's head_dim {dim}, not {shape[2]}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has type {t.dtype}, not {dtype}")
    return _pack_heads(t.data_ptr(), stride[0], stride[1], shape[1])


def _code(dtype: torch.dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    return code


def _ints(t: torch.Tensor, name: str, dim: int = 1) -> int:
    """Address of an int32 tensor."""
    if t.dtype != torch.int32 or t.dim() != dim or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name} must be int32 with {dim} dimension(s), its last one contiguous")
    return t.data_ptr()


def _table(t: torch.Tensor):
    """(address, row stride, width) of a block table."""
    at, (rows, width), stride = _ints(t, "block_table", 2), t.shape, t.stride(0)
    if stride < width:
        if rows > 1:
            raise ValueError(f"block_table's rows overlap: {stride} entries apart, {width} wide")
        stride = width
    return at, stride, width


def _call(name: str, stream, tensors, *args, fns=None) -> None:
    """The C call (of `fns`, or this module's) on the tensors' device and its
    current stream (or `stream`)."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"{name}: tensors of one call on {tensors[0].device} and {t.device}")
    if dev < 0:
        raise ValueError(f"{name} needs GPU tensors")
    if stream is None:
        s = _raw_stream(dev)
    elif stream.device_index != dev:
        raise ValueError(f"{name}: a stream of {stream.device} for tensors on {tensors[0].device}")
    else:
        s = stream.cuda_stream
    fn = (fns or _bound or lib())[name]
    if _current() == dev:
        st = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, s)
    if st != 0:
        raise lora.LoraError(name, st)


# ------------------------------------------------------------------ handles
def block_bytes(block_tokens: int, num_kv_heads: int, head_dim: int) -> int:
    """Bytes of one cache block (0: unsupported geometry)."""
    return int(lib()["lora_kv_block_bytes"](block_tokens, num_kv_heads, head_dim))


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
        self.ref = ctypes.addressof(self.c)

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
        self.ref = ctypes.addressof(self.c)

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
        n = L["lora_kv_batch_size"](max_tokens, max_seqs, num_q_heads, num_kv_heads, head_dim)
        if n == 0:
            raise ValueError("unsupported batch capacity or head geometry")
        # zeroed: a buffer that was never built must not look like one that was
        self.buf = torch.zeros(n, dtype=torch.uint8, device=device)
        self.c = lora_kv_batch_t()
        self.ref = ctypes.addressof(self.c)
        st = L["lora_kv_batch_init"](self.buf.data_ptr(), n, max_tokens, max_seqs, num_q_heads, num_kv_heads, head_dim, self.ref)
        if st != 0:
            raise lora.LoraError("lora_kv_batch_init", st)
        self._all = {name: self._view(name, size) for name, size in
                     (("q_indptr", max_seqs + 1), ("kv_len", max_seqs), ("token_seq", max_tokens),
                      ("positions", max_tokens), ("slots", max_tokens), ("counts", N_COUNTS))}
        self.counts = self._all["counts"]
        self.flags = self.counts[COUNT_FLAGS:COUNT_FLAGS + 1]
        self.new_blocks = self.counts[COUNT_NEW_BLOCKS:COUNT_NEW_BLOCKS + 1]
        self._resize(0, 0)

    def _view(self, field: str, n: int) -> torch.Tensor:
        off = getattr(self.c, field) - self.buf.data_ptr()
        return self.buf[off:off + 4 * n].view(torch.int32)

    def _resize(self, T: int, B: int) -> None:
        """The arrays' views for a build of T rows and B requests."""
        self.T, self.B = T, B
        self.q_indptr, self.kv_len = self._all["q_indptr"][:B + 1], self._all["kv_len"][:B]
        self.token_seq, self.positions, self.slots = (self._all[n][:T] for n in ("token_seq", "positions", "slots"))


def attend_workspace(batch: Batch) -> torch.Tensor:
    """Workspace of lora_kv_attend for a batch buffer (one serves every layer)."""
    n = lib()["lora_kv_workspace_size"](batch.ref)
    return torch.empty(n, dtype=torch.uint8, device=batch.buf.device)


class Shared:
    """Device buffer of a batch's shared plan, for up to max_groups groups of
    requests that begin with the same cached tokens."""

    def __init__(self, batch: Batch, max_groups: int):
        L = lib()
        n = L["lora_kv_share_size"](batch.ref, max_groups)
        if n == 0:
            raise ValueError("unsupported number of groups")
        # zeroed, as a batch's buffer is
        self.buf = torch.zeros(n, dtype=torch.uint8, device=batch.buf.device)
        self.c = lora_kv_share_t()
        self.ref = ctypes.addressof(self.c)
        st = L["lora_kv_share_init"](self.buf.data_ptr(), n, batch.ref, max_groups, self.ref)
        if st != 0:
            raise lora.LoraError("lora_kv_share_init", st)
        self.batch, self.groups = batch, 0


def shared_workspace(batch: Batch, shared: Shared) -> torch.Tensor:
    """Workspace of lora_kv_attend_shared (one serves every layer)."""
    n = lib()["lora_kv_share_workspace_size"](batch.ref, shared.ref)
    return torch.empty(n, dtype=torch.uint8, device=batch.buf.device)


# ------------------------------------------------------- the C entry points
def lora_rope_frequencies(rot_dim: int, theta: float = 10000.0, scaling: int = SCALING_NONE, factor: float = 1.0,
                          original: float = 0.0, low: float = 0.0, high: float = 0.0):
    """(frequencies as a list of floats, scale of cos and sin)."""
    out, scale = (_f64 * max(rot_dim // 2, 1))(), _f64()
    st = lib()["lora_rope_frequencies"](rot_dim, theta, scaling, factor, original, low, high, out, ctypes.byref(scale))
    if st != 0:
        raise lora.LoraError("lora_rope_frequencies", st)
    return list(out), scale.value


def lora_kv_build(ctx_len: torch.Tensor, new_len: torch.Tensor, T: int, block_table: torch.Tensor,
                  free_blocks: torch.Tensor, num_blocks: int, block_tokens: int, batch: Batch, stream=None) -> None:
    """Rows, positions, slots and plan of a step from request lengths; new
    blocks go from free_blocks into block_table (B, width)."""
    (table, stride, width), B = _table(block_table), ctx_len.shape[0]
    if new_len.shape[0] != B or block_table.shape[0] != B:
        raise ValueError("one length of each kind and one table row per request")
    _call("lora_kv_build", stream, (ctx_len, new_len, block_table, free_blocks, batch.buf),
          _ints(ctx_len, "ctx_len"), _ints(new_len, "new_len"), B, T, table, stride, width, _ints(free_blocks, "free_blocks"),
          free_blocks.shape[0], num_blocks, block_tokens, batch.ref)
    if batch.T != T or batch.B != B:
        batch._resize(T, B)


def lora_rope(q: Optional[torch.Tensor], q_out: Optional[torch.Tensor], k: Optional[torch.Tensor],
              k_out: Optional[torch.Tensor], positions: torch.Tensor, rope: Rope, stream=None) -> None:
    """Rotate q and k (T, heads, head_dim; either may be None) into q_out and
    k_out, which may be q and k."""
    if (q is None and k is None) or (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("q with q_out, k with k_out, or both")
    pos, T = _ints(positions, "positions"), positions.shape[0]
    lead = k if q is None else q
    D, dtype = lead.shape[-1], lead.dtype
    tensors, ref = [positions, rope.inv_freq], []
    for name, t in (("q", q), ("q_out", q_out), ("k", k), ("k_out", k_out)):
        ref.append(None if t is None else _heads(t, name, T, D, dtype))
        if t is not None:
            tensors.append(t)
    _call("lora_rope", stream, tensors, *ref, pos, T, D, _code(dtype), rope.ref)


def lora_kv_append(q: Optional[torch.Tensor], q_out: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                   positions: Optional[torch.Tensor], slots: torch.Tensor, rope: Optional[Rope], cache: Cache,
                   batch: Optional[Batch] = None, stream=None) -> None:
    """Rotate q into q_out and put rotated k, and v, into the cache at slots.
    rope None: no rotation.  batch: whose flags take FLAG_NONFINITE."""
    slot, T = _ints(slots, "slots"), slots.shape[0]
    if rope is None and q is not None:
        raise ValueError("q is only rotated: pass rope, or no q")
    if rope is not None and positions is None:
        raise ValueError("rope needs positions")
    if (q is None) != (q_out is None):
        raise ValueError("q with q_out")
    D, dtype = cache.head_dim, k.dtype
    tensors = [slots, cache.data, k, v]
    kr, vr = _heads(k, "k", T, D, dtype), _heads(v, "v", T, D, dtype)
    qr = qo = pos = flags = None
    if q is not None:
        qr, qo = _heads(q, "q", T, D, dtype), _heads(q_out, "q_out", T, D, dtype)
        tensors += (q, q_out)
    if positions is not None:
        pos = _ints(positions, "positions")
        if positions.shape[0] != T:
            raise ValueError("one position per slot")
        tensors.append(positions)
    if rope is not None:
        tensors.append(rope.inv_freq)
    if batch is not None:
        flags = batch.c.counts + 4 * COUNT_FLAGS
        tensors.append(batch.buf)
    _call("lora_kv_append", stream, tensors, qr, qo, kr, vr, pos, slot, T, _code(dtype),
          None if rope is None else rope.ref, cache.ref, flags)


def lora_kv_gather(cache: Cache, slots: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor, stream=None) -> None:
    """The cached K and V at slots as values (n, kv heads, head_dim)."""
    slot, n, dtype = _ints(slots, "slots"), slots.shape[0], k_out.dtype
    _call("lora_kv_gather", stream, (slots, cache.data, k_out, v_out), cache.ref, slot, n,
          _heads(k_out, "k_out", n, cache.head_dim, dtype), _heads(v_out, "v_out", n, cache.head_dim, dtype), _code(dtype))


def lora_kv_attend(q: torch.Tensor, out: torch.Tensor, batch: Batch, block_table: torch.Tensor, cache: Cache,
                   scale: float, ws: torch.Tensor, stream=None) -> None:
    """Attention of the batch's rows q (T, heads, head_dim) over the cache."""
    (table, stride, width), dtype = _table(block_table), q.dtype
    if block_table.shape[0] != batch.B:
        raise ValueError(f"block_table has {block_table.shape[0]} rows, not {batch.B}")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    _call("lora_kv_attend", stream, (q, out, batch.buf, block_table, cache.data, ws),
          _heads(q, "q", batch.T, cache.head_dim, dtype), _heads(out, "out", batch.T, cache.head_dim, dtype), batch.T, batch.B,
          _code(dtype), batch.ref, table, stride, width, cache.ref, scale, ws.data_ptr(),
          ws.numel() * ws.element_size())


def lora_kv_share(group_indptr: torch.Tensor, shared_len: torch.Tensor, batch: Batch, shared: Shared, stream=None) -> None:
    """Plan of a built batch whose requests group_indptr[g]..group_indptr[g+1]-1
    begin with the same shared_len[g] cached tokens."""
    groups = shared_len.shape[0]
    if group_indptr.shape[0] != groups + 1:
        raise ValueError("group_indptr has one entry more than shared_len")
    if shared.batch is not batch:
        raise ValueError("shared was made for another batch buffer")
    _call("lora_kv_share", stream, (group_indptr, shared_len, batch.buf, shared.buf), _ints(group_indptr, "group_indptr"),
          _ints(shared_len, "shared_len"), groups, batch.T, batch.B, batch.ref, shared.ref)
    shared.groups = groups


def lora_kv_attend_shared(q: torch.Tensor, out: torch.Tensor, batch: Batch, shared: Shared, block_table: torch.Tensor,
                          cache: Cache, scale: float, ws: torch.Tensor, stream=None) -> None:
    """lora_kv_attend, with the tokens that groups share attended to together, by
    the plan that lora_kv_share made of the batch's last build."""
    (table, stride, width), dtype = _table(block_table), q.dtype
    if block_table.shape[0] != batch.B:
        raise ValueError(f"block_table has {block_table.shape[0]} rows, not {batch.B}")
    if shared.batch is not batch:
        raise ValueError("shared was made for another batch buffer")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    _call("lora_kv_attend_shared", stream, (q, out, batch.buf, shared.buf, block_table, cache.data, ws),
          _heads(q, "q", batch.T, cache.head_dim, dtype), _heads(out, "out", batch.T, cache.head_dim, dtype), batch.T, batch.B,
          shared.groups, _code(dtype), batch.ref, shared.ref, table, stride, width, cache.ref, scale, ws.data_ptr(),
          ws.numel() * ws.element_size())


def lora_prompt_attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, indptr: torch.Tensor,
                       scale: float, stream=None) -> None:
    """Causal attention of packed prompts: rows indptr[i]..indptr[i+1]-1 of q,
    k, v and out (T, heads, head_dim) are prompt i."""
    ptr, B = _ints(indptr, "indptr"), indptr.shape[0] - 1
    if B < 0:
        raise ValueError("indptr has one entry more than prompts")
    T, D, dtype = q.shape[0], q.shape[-1], q.dtype
    _call("lora_prompt_attend", stream, (q, k, v, out, indptr), _heads(q, "q", T, D, dtype), _heads(k, "k", T, D, dtype),
          _heads(v, "v", T, D, dtype), _heads(out, "out", T, D, dtype), ptr, B, T, D, _code(dtype), scale)
