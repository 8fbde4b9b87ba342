"""Python binding of the beam search operators (``include/lora_beam.h``):
argument marshalling only.

A search's step over the paged cache of ``kv``: the best continuations of every
request's beams from the step's logits (``lora_beam_select``), the survivors'
block tables (``lora_beam_reorder``) and the copies of blocks that two of them
would write to, in every layer (``lora_beam_copy``).  Beam w of request b is
row ``b*beams + w`` of every tensor.  Tensors, streams and errors as in ``kv``.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import kv, lora

MAX_BEAMS, MAX_VOCAB, MAX_LAYERS, MAX_PENALTY = 32, 1 << 24, 1024, 16
FLAG_LOGITS, FLAG_PARENT, FLAG_LENGTH, FLAG_FREE_LIST, FLAG_BLOCK_RANGE = 1, 2, 4, 8, 16
COUNT_COPIES, COUNT_FREED, COUNT_FLAGS = 0, 1, 8
N_COUNTS = 16
EXPORTS = ("lora_beam_select_workspace", "lora_beam_select", "lora_beam_moves_size", "lora_beam_moves_init",
           "lora_beam_reorder", "lora_beam_copy")

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class lora_beams_t(ctypes.Structure):
    _fields_ = [("score", _vp), ("length", _vp), ("done", _vp)]


class lora_beam_moves_t(ctypes.Structure):
    _fields_ = [("max_rows", _i32), ("table_width", _i32), ("source", _vp), ("target", _vp), ("tokens", _vp),
                ("freed", _vp), ("counts", _vp), ("scratch", _vp)]


_bound = None


def lib() -> dict:
    """liblora.so's beam search functions by name, declared."""
    global _bound
    if _bound is None:
        L, sz = lora.lib(), ctypes.c_size_t
        sigs = {
            "lora_beam_select_workspace": (sz, [_i32] * 3),
            "lora_beam_select": (_i32, [_vp, _i64, _i32, _i32, _i32, _i32, _vp, ctypes.c_float, _i32, _vp, _vp, _vp, _vp, _vp, sz, _vp]),
            "lora_beam_moves_size": (sz, [_i32] * 2),
            "lora_beam_moves_init": (_i32, [_vp, sz, _i32, _i32, _vp]),
            "lora_beam_reorder": (_i32, [_vp, _vp, _i32, _i32, _vp, _i64, _vp, _i64, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _vp]),
            "lora_beam_copy": (_i32, [_vp, _vp, _i32, _vp]),
        }
        fns = {}
        for name, (res, args) in sigs.items():
            fns[name] = f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _bound = fns
    return _bound


def _call(name: str, stream, tensors, *args) -> None:
    kv._call(name, stream, tensors, *args, fns=_bound or lib())


# ------------------------------------------------------------------ handles
class Beams:
    """The beams' state, one entry per row: score (float32), length and done
    (int32)."""

    def __init__(self, score: torch.Tensor, length: torch.Tensor, done: torch.Tensor):
        for name, t, dtype in (("score", score, torch.float32), ("length", length, torch.int32), ("done", done, torch.int32)):
            if t.dtype != dtype or t.dim() != 1 or not t.is_contiguous() or t.shape != score.shape:
                raise ValueError(f"{name} must be a contiguous vector of {dtype}, one entry per row")
        self.score, self.length, self.done = score, length, done
        self.c = lora_beams_t(score.data_ptr(), length.data_ptr(), done.data_ptr())
        self.ref = ctypes.addressof(self.c)

    @classmethod
    def start(cls, num_requests: int, beams: int, device="cuda") -> "Beams":
        """A search's first state: one beam per request, of score 0."""
        score = torch.full((num_requests, beams), -float("inf"), device=device)
        score[:, 0] = 0.0
        zeros = lambda: torch.zeros(num_requests * beams, dtype=torch.int32, device=device)  # noqa: E731
        return cls(score.flatten(), zeros(), zeros())


class Moves:
    """Copies and freed blocks of a reorder, for up to max_rows rows and tables
    of up to table_width entries."""

    def __init__(self, max_rows: int, table_width: int, device="cuda"):
        n = lib()["lora_beam_moves_size"](max_rows, table_width)
        if n == 0:
            raise ValueError("unsupported number of rows or table width")
        # zeroed: no copies before the first reorder
        self.buf = torch.zeros(n, dtype=torch.uint8, device=device)
        self.c = lora_beam_moves_t()
        self.ref = ctypes.addressof(self.c)
        st = lib()["lora_beam_moves_init"](self.buf.data_ptr(), n, max_rows, table_width, self.ref)
        if st != 0:
            raise lora.LoraError("lora_beam_moves_init", st)
        view = lambda field, n: self._view(field, n)  # noqa: E731
        self.source, self.target, self.tokens = view("source", max_rows), view("target", max_rows), view("tokens", max_rows)
        self.freed, self.counts = view("freed", max_rows * table_width), view("counts", N_COUNTS)
        self.copies = self.counts[COUNT_COPIES:COUNT_COPIES + 1]
        self.given_back = self.counts[COUNT_FREED:COUNT_FREED + 1]
        self.flags = self.counts[COUNT_FLAGS:COUNT_FLAGS + 1]

    def _view(self, field: str, n: int) -> torch.Tensor:
        off = getattr(self.c, field) - self.buf.data_ptr()
        return self.buf[off:off + 4 * n].view(torch.int32)


class Layers:
    """The caches of all layers, of one geometry."""

    def __init__(self, caches: Sequence["kv.Cache"]):
        self.caches = tuple(caches)
        self.array = (kv.lora_kv_cache_t * max(len(self.caches), 1))(*(c.c for c in self.caches))
        self.ref, self.n = ctypes.addressof(self.array), len(self.caches)


def select_workspace(num_requests: int, beams: int, vocab: int, device="cuda") -> torch.Tensor:
    """Workspace of lora_beam_select."""
    n = lib()["lora_beam_select_workspace"](num_requests, beams, vocab)
    if n == 0:
        raise ValueError("unsupported number of requests, beams or tokens")
    return torch.empty(n, dtype=torch.uint8, device=device)


# ------------------------------------------------------- the C entry points
def lora_beam_select(logits: torch.Tensor, beams: int, state: Beams, parent: torch.Tensor, token: torch.Tensor,
                     out: Beams, ws: torch.Tensor, length_penalty: float = 0.0, eos: int = -1,
                     flags: Optional[torch.Tensor] = None, stream=None) -> None:
    """The best continuations of every request's beams: logits (rows, vocab)
    into parent and token (rows) and the new state `out`, which may be `state`."""
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must have shape (rows, vocab) with contiguous tokens")
    rows, vocab = logits.shape
    if beams < 1 or rows % beams:
        raise ValueError(f"{rows} rows are not a whole number of requests of {beams} beams")
    for name, n in (("state", state.score.shape[0]), ("out", out.score.shape[0]), ("parent", parent.shape[0]), ("token", token.shape[0])):
        if n != rows:
            raise ValueError(f"{name} has {n} rows, not {rows}")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    tensors = [logits, state.score, state.length, state.done, parent, token, out.score, out.length, out.done, ws]
    fl = None
    if flags is not None:
        fl = kv._ints(flags, "flags")
        if flags.numel() < 1:
            raise ValueError("flags must have an entry")
        tensors.append(flags)
    _call("lora_beam_select", stream, tensors, logits.data_ptr(), logits.stride(0) if rows > 1 else vocab, kv._code(logits.dtype),
          rows // beams, beams, vocab, state.ref, length_penalty, eos, kv._ints(parent, "parent"), kv._ints(token, "token"), out.ref,
          fl, ws.data_ptr(), ws.numel() * ws.element_size())


def lora_beam_reorder(parent: torch.Tensor, beams: int, kv_len: torch.Tensor, block_table: torch.Tensor,
                      new_len: torch.Tensor, new_table: torch.Tensor, free_blocks: torch.Tensor, num_blocks: int,
                      block_tokens: int, moves: Moves, stream=None) -> None:
    """Block tables of the rows that go on from `parent` into new_table and
    new_len; copies and freed blocks into moves."""
    (table, stride, width), (new, new_stride, new_width) = kv._table(block_table), kv._table(new_table)
    rows = parent.shape[0]
    if beams < 1 or rows % beams:
        raise ValueError(f"{rows} rows are not a whole number of requests of {beams} beams")
    for name, t in (("kv_len", kv_len), ("block_table", block_table), ("new_len", new_len), ("new_table", new_table)):
        if t.shape[0] != rows:
            raise ValueError(f"{name} has {t.shape[0]} rows, not {rows}")
    if new_width != width:
        raise ValueError(f"new_table is {new_width} wide, not {width}")
    _call("lora_beam_reorder", stream, (parent, kv_len, block_table, new_len, new_table, free_blocks, moves.buf),
          kv._ints(parent, "parent"), kv._ints(kv_len, "kv_len"), rows // beams, beams, table, stride, new, new_stride, width,
          kv._ints(new_len, "new_len"), kv._ints(free_blocks, "free_blocks"), free_blocks.shape[0], num_blocks, block_tokens,
          moves.ref)


def lora_beam_copy(moves: Moves, layers: Layers, stream=None) -> None:
    """The copies of a reorder, in every layer's cache."""
    _call("lora_beam_copy", stream, [moves.buf] + [c.data for c in layers.caches], moves.ref, layers.ref, layers.n)
