"""Host-side tests of beam search and of shared plans: exports, sizes, refusals
before any device work, the plain references themselves (no GPU)."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import beam_reference as BR
from heterogeneous_adapters_amd import beam, kv, lora

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lora_beam.h")


def test_library_exports_every_declared_function():
    txt = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    fns = set(re.findall(r"^(?:size_t|lora_status_t)\s+(lora_[a-z_]+)\s*\(", txt, flags=re.M))
    assert fns == set(beam.EXPORTS) == set(beam.lib())


def test_binding_constants_match_header():
    defs = dict(re.findall(r"^#define (LORA_BEAM_[A-Z_0-9]+) \(?([^/\n]*?)\)?\s*(?:/\*.*)?$", open(HEADER).read(), flags=re.M))
    want = {"MAX": beam.MAX_BEAMS, "MAX_VOCAB": beam.MAX_VOCAB, "MAX_LAYERS": beam.MAX_LAYERS, "MAX_PENALTY": beam.MAX_PENALTY}
    want.update({f"FLAG_{n}": getattr(beam, f"FLAG_{n}") for n in ("LOGITS", "PARENT", "LENGTH", "FREE_LIST", "BLOCK_RANGE")})
    want.update({f"COUNT_{n}": getattr(beam, f"COUNT_{n}") for n in ("COPIES", "FREED", "FLAGS")})
    assert set(want) == {n[len("LORA_BEAM_"):] for n in defs}
    for name, v in want.items():
        assert eval(defs["LORA_BEAM_" + name].strip()) == v, name


def test_structs_match_the_header(tmp_path):
    import subprocess
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "lora_beam.h"\nint main(void){printf("%zu %zu %zu",sizeof(lora_beams_t),'
                   'sizeof(lora_beam_moves_t),sizeof(lora_kv_share_t));return 0;}\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout
    assert got == " ".join(str(ctypes.sizeof(c)) for c in (beam.lora_beams_t, beam.lora_beam_moves_t, kv.lora_kv_share_t))


def ref(x):
    return None if x is None else ctypes.byref(x)


class Buf:
    """Aligned host memory that no kernel may touch: a refusal comes before any launch."""

    def __init__(self, n=1 << 16):
        self.raw = ctypes.create_string_buffer(n + 256)
        self.p = (ctypes.addressof(self.raw) + 255) // 256 * 256

    def at(self, k):
        return self.p + 1024 * k


def beams_at(b, k):
    return beam.lora_beams_t(b.at(k), b.at(k + 1), b.at(k + 2))


@pytest.mark.parametrize("case,code", [
    ("null_logits", -1), ("null_parent", -1), ("null_token", -1), ("null_in", -1), ("null_out", -1), ("null_score", -1), ("null_done_out", -1),
    ("null_ws", -1), ("requests", -1), ("beams", -1), ("many_beams", -6), ("vocab", -1), ("large_vocab", -6), ("rows", -6), ("stride", -1),
    ("far", -6), ("penalty", -1), ("penalty_inf", -1), ("penalty_large", -1), ("eos", -1), ("eos_low", -1), ("dtype", -6), ("align", -7), ("ws_align", -7), ("ws", -4),
    ("same_out", -1), ("out_in", -1), ("crossed", -1), ("shifted", -1), ("out_logits", -1),
])
def test_select_refusals(case, code):
    b = Buf()
    logits, stride, dt, B, W, V = b.at(0), 100, lora.LORA_DTYPE_F32, 2, 3, 100
    i, o, parent, token, ws, pen, eos = beams_at(b, 10), beams_at(b, 20), b.at(30), b.at(31), b.at(40), 0.0, 5
    n = beam.lib()["lora_beam_select_workspace"](B, W, V)
    assert n > 0
    if case == "null_logits":
        logits = None
    if case == "null_parent":
        parent = None
    if case == "null_token":
        token = None
    if case == "null_in":
        i = None
    if case == "null_out":
        o = None
    if case == "null_score":
        i.score = None
    if case == "null_done_out":
        o.done = None
    if case == "null_ws":
        ws = None
    if case == "requests":
        B = -1
    if case == "beams":
        W = 0
    if case == "many_beams":
        W = 33
    if case == "vocab":
        V = 0
    if case == "large_vocab":
        V = stride = (1 << 24) + 1
    if case == "rows":
        B = 30000
    if case == "stride":
        stride = 99
    if case == "far":
        stride = 1 << 41
    if case == "penalty":
        pen = math.nan
    if case == "penalty_inf":
        pen = math.inf
    if case == "penalty_large":
        pen = -16.5
    if case == "eos":
        eos = 100
    if case == "eos_low":
        eos = -2
    if case == "dtype":
        dt = 7
    if case == "align":
        logits += 2
    if case == "ws_align":
        ws += 8
    if case == "ws":
        n -= 1
    if case == "same_out":
        parent = token
    if case == "out_in":
        parent = i.score
    if case == "crossed":
        o.length = i.done
    if case == "shifted":
        o.score = i.score + 4
    if case == "out_logits":
        token = logits + 400
    assert beam.lib()["lora_beam_select"](logits, stride, dt, B, W, V, ref(i), pen, eos, parent, token, ref(o), None, ws, n, None) == code


@pytest.mark.parametrize("case,code", [
    ("null_parent", -1), ("null_len", -1), ("null_table", -1), ("null_new", -1), ("null_new_len", -1), ("null_free", -1), ("null_moves", -1),
    ("moves", -1), ("requests", -1), ("beams", -1), ("many_beams", -6), ("num_free", -1), ("num_blocks", -1), ("width", -1), ("stride", -1),
    ("new_stride", -1), ("block_tokens", -6), ("blocks_range", -6), ("width_range", -6), ("rows", -4), ("wide", -4), ("same_table", -1),
    ("len_len", -1), ("in_moves", -1), ("free_new", -1),
])
def test_reorder_refusals(case, code):
    b = Buf()
    L = beam.lib()
    m = beam.lora_beam_moves_t()
    n = L["lora_beam_moves_size"](8, 10)
    store = Buf(n)
    assert L["lora_beam_moves_init"](store.p, n, 8, 10, ctypes.byref(m)) == 0
    parent, lens, B, W, table, stride, new, new_stride, width, new_len, free, nfree, nblocks, bt = (
        b.at(0), b.at(1), 2, 3, b.at(2), 10, b.at(3), 10, 10, b.at(4), b.at(5), 6, 100, 16)
    if case == "null_parent":
        parent = None
    if case == "null_len":
        lens = None
    if case == "null_table":
        table = None
    if case == "null_new":
        new = None
    if case == "null_new_len":
        new_len = None
    if case == "null_free":
        free = None
    if case == "null_moves":
        m = None
    if case == "moves":
        m.freed = None
    if case == "requests":
        B = -1
    if case == "beams":
        W = 0
    if case == "many_beams":
        W = 33
    if case == "num_free":
        nfree = -1
    if case == "num_blocks":
        nblocks = 0
    if case == "width":
        width = 0
    if case == "stride":
        stride = 9
    if case == "new_stride":
        new_stride = 9
    if case == "block_tokens":
        bt = 24
    if case == "blocks_range":
        nblocks = 1 << 27
    if case == "width_range":
        width = stride = new_stride = (1 << 26) + 1
    if case == "rows":
        B = 3
    if case == "wide":
        width = stride = new_stride = 11
    if case == "same_table":
        new = table
    if case == "len_len":
        new_len = lens
    if case == "in_moves":
        parent = store.p
    if case == "free_new":
        free = new + 8
    assert L["lora_beam_reorder"](parent, lens, B, W, table, stride, new, new_stride, width, new_len, free, nfree, nblocks, bt, ref(m), None) == code


@pytest.mark.parametrize("case,code", [("null_moves", -1), ("null_caches", -1), ("layers", -1), ("many", -6), ("base", -1), ("geometry", -6),
                                       ("stride", -1), ("differ", -1), ("differ_dim", -1), ("align", -7), ("base_align", -7)])
def test_copy_refusals(case, code):
    b = Buf()
    L = beam.lib()
    m = beam.lora_beam_moves_t()
    n = L["lora_beam_moves_size"](8, 10)
    store = Buf(n)
    assert L["lora_beam_moves_init"](store.p, n, 8, 10, ctypes.byref(m)) == 0
    nb = kv.block_bytes(16, 2, 64)
    caches = (kv.lora_kv_cache_t * 2)(*(kv.lora_kv_cache_t(b.at(i), nb, 4, 16, 2, 64) for i in range(2)))
    layers = 2
    if case == "null_moves":
        m = None
    if case == "null_caches":
        caches = None
    if case == "layers":
        layers = -1
    if case == "many":
        layers = 1025
    if case == "base":
        caches[1].base = None
    if case == "geometry":
        caches[0].block_tokens = 17
    if case == "stride":
        caches[0].block_stride = nb - 16
    if case == "differ":
        caches[1].num_blocks = 5
    if case == "differ_dim":
        caches[1].head_dim = 32
    if case == "align":
        caches[0].block_stride = caches[1].block_stride = nb + 8
    if case == "base_align":
        caches[1].base = b.at(1) + 4
    assert L["lora_beam_copy"](ref(m), caches, layers, None) == code


def test_sizes_and_carving():
    L = beam.lib()
    assert L["lora_beam_select_workspace"](0, 4, 10) > 0
    for bad in ((-1, 4, 10), (1, 0, 10), (1, 33, 10), (1, 4, 0), (1, 4, (1 << 24) + 1), (65537, 1, 10)):
        assert L["lora_beam_select_workspace"](*bad) == 0
    for bad in ((0, 4), (4, 0), (65537, 4), (1 << 16, 1 << 14)):
        assert L["lora_beam_moves_size"](*bad) == 0
    b, m = Buf(), beam.lora_beam_moves_t()
    n = L["lora_beam_moves_size"](5, 7)
    for args, code in (((None, n, 5, 7), -1), ((b.p, n - 1, 5, 7), -4), ((b.p + 8, n, 5, 7), -7), ((b.p, n, 0, 7), -1), ((b.p, n, 1 << 17, 7), -6)):
        assert L["lora_beam_moves_init"](*args, ctypes.byref(m)) == code
    assert L["lora_beam_moves_init"](b.p, n, 5, 7, ctypes.byref(m)) == 0
    at = [m.source, m.target, m.tokens, m.freed, m.counts, m.scratch, b.p + n]
    need = [20, 20, 20, 140, 64, 40]
    assert at[0] == b.p and all(at[i] + need[i] <= at[i + 1] and at[i] % 16 == 0 for i in range(6))


# --------------------------------------------------------------- shared plans
class Plan:
    def __init__(self):
        self.L, self.b = kv.lib(), Buf()
        self.batch = kv.lora_kv_batch_t()
        n = self.L["lora_kv_batch_size"](64, 8, 8, 2, 64)
        self.store = Buf(n)
        assert self.L["lora_kv_batch_init"](self.store.p, n, 64, 8, 8, 2, 64, ctypes.byref(self.batch)) == 0
        self.n = self.L["lora_kv_share_size"](ref(self.batch), 3)
        self.buf, self.share = Buf(self.n), kv.lora_kv_share_t()
        assert self.L["lora_kv_share_init"](self.buf.p, self.n, ref(self.batch), 3, ctypes.byref(self.share)) == 0


def test_shared_sizes_and_carving():
    p = Plan()
    assert p.n > 0 and p.L["lora_kv_share_workspace_size"](ref(p.batch), ref(p.share)) > 0
    for bad in (-1, 9):
        assert p.L["lora_kv_share_size"](ref(p.batch), bad) == 0
    assert p.L["lora_kv_share_size"](None, 1) == 0 and p.L["lora_kv_share_size"](ref(p.batch), 0) > 0
    f = p.L["lora_kv_share_init"]
    for args, code in (((None, p.n, ref(p.batch), 3), -1), ((p.buf.p, p.n - 1, ref(p.batch), 3), -4), ((p.buf.p + 4, p.n, ref(p.batch), 3), -7),
                       ((p.buf.p, p.n, None, 3), -1), ((p.buf.p, p.n, ref(p.batch), -1), -1), ((p.buf.p, p.n, ref(p.batch), 9), -6)):
        assert f(*args, ctypes.byref(p.share)) == code
    assert f(p.buf.p, p.n, ref(p.batch), 3, None) == -1


@pytest.mark.parametrize("case,code", [("null_groups", -1), ("null_len", -1), ("groups", -1), ("many", -4), ("T", -1), ("large_T", -4), ("B", -4),
                                       ("batch", -1), ("share", -1), ("null_share", -1), ("in_batch", -1), ("in_plan", -1), ("len_in_batch", -1)])
def test_share_refusals(case, code):
    p = Plan()
    groups, lens, n, T, B, batch, share = p.b.at(0), p.b.at(1), 2, 8, 4, p.batch, p.share
    if case == "null_groups":
        groups = None
    if case == "null_len":
        lens = None
    if case == "groups":
        n = -1
    if case == "many":
        n = 4
    if case == "T":
        T = -1
    if case == "large_T":
        T = 65
    if case == "B":
        B = 9
    if case == "batch":
        batch.counts = None
    if case == "share":
        share.plan = None
    if case == "null_share":
        share = None
    if case == "in_batch":
        groups = batch.kv_len
    if case == "in_plan":
        groups = share.plan
    if case == "len_in_batch":
        lens = batch.positions
    assert p.L["lora_kv_share"](groups, lens, n, T, B, ref(batch), ref(share), None) == code


@pytest.mark.parametrize("case,code", [("groups", -1), ("many", -4), ("share", -1), ("ws", -4), ("null_ws", -1), ("ws_align", -7), ("scale", -1),
                                       ("heads", -1), ("same", -1), ("T", -4), ("dtype", -6), ("null_table", -1), ("dim", -1)])
def test_attend_shared_refusals(case, code):
    p = Plan()
    heads = lambda k: kv.lora_heads_t(p.b.at(k), 512, 64, 8)  # noqa: E731
    q, o, T, B, n, dt, scale = heads(0), heads(20), 8, 4, 2, lora.LORA_DTYPE_BF16, 0.1
    cache = kv.lora_kv_cache_t(p.b.at(40), kv.block_bytes(16, 2, 64), 4, 16, 2, 64)
    table, ws, size = p.b.at(50), p.b.at(51), p.L["lora_kv_share_workspace_size"](ref(p.batch), ref(p.share))
    if case == "groups":
        n = -1
    if case == "many":
        n = 4
    if case == "share":
        p.share.counts = None
        size = 1 << 40
    if case == "ws":
        size -= 1
    if case == "null_ws":
        ws = None
    if case == "ws_align":
        ws += 4
    if case == "scale":
        scale = -0.5
    if case == "heads":
        q.heads = o.heads = 4
    if case == "same":
        o = q
    if case == "T":
        T = 65
    if case == "dtype":
        dt = 5
    if case == "null_table":
        table = None
    if case == "dim":
        cache.head_dim = 32
    assert p.L["lora_kv_attend_shared"](ref(q), ref(o), T, B, n, dt, ref(p.batch), ref(p.share), table, 4, 4, ref(cache), scale, ws, size, None) == code


def test_nothing_to_do_needs_no_device():
    p, b = Plan(), Buf()
    q, o = kv.lora_heads_t(b.at(0), 512, 64, 8), kv.lora_heads_t(b.at(9), 512, 64, 8)
    cache = kv.lora_kv_cache_t(b.at(20), kv.block_bytes(16, 2, 64), 4, 16, 2, 64)
    size = p.L["lora_kv_share_workspace_size"](ref(p.batch), ref(p.share))
    assert p.L["lora_kv_attend_shared"](ref(q), ref(o), 0, 0, 0, 1, ref(p.batch), ref(p.share), None, 0, 0, ref(cache), 0.1, b.at(30), size, None) == 0
    i = beams_at(b, 0)
    n = beam.lib()["lora_beam_select_workspace"](0, 4, 10)
    assert beam.lib()["lora_beam_select"](None, 10, 0, 0, 4, 10, ref(i), 0.0, -1, None, None, ref(i), None, None, n, None) == 0


# ----------------------------------------------------------- binding's checks
def test_binding_refusals():
    z = lambda *n, t=torch.int32: torch.zeros(n, dtype=t)  # noqa: E731
    with pytest.raises(ValueError, match="contiguous vector"):
        beam.Beams(z(4), z(4), z(4))
    with pytest.raises(ValueError, match="contiguous vector"):
        beam.Beams(z(4, t=torch.float32), z(3), z(4))
    s = beam.Beams(z(6, t=torch.float32), z(6), z(6))
    x, ws = z(6, 10, t=torch.float32), z(64, t=torch.uint8)
    with pytest.raises(ValueError, match="whole number"):
        beam.lora_beam_select(x, 4, s, z(6), z(6), s, ws)
    with pytest.raises(ValueError, match="rows"):
        beam.lora_beam_select(x, 3, s, z(5), z(6), s, ws)
    with pytest.raises(ValueError, match="contiguous tokens"):
        beam.lora_beam_select(x.t().contiguous().t(), 3, s, z(6), z(6), s, ws)
    with pytest.raises(ValueError, match="GPU"):
        beam.lora_beam_select(x, 3, s, z(6), z(6), s, ws)
    with pytest.raises(ValueError, match="dtype"):
        beam.lora_beam_select(x.double(), 3, s, z(6), z(6), s, ws)
    with pytest.raises(ValueError, match="unsupported"):
        beam.select_workspace(1, 40, 10, device="cpu")
    with pytest.raises(ValueError, match="unsupported"):
        beam.Moves(0, 3, device="cpu")
    m = beam.Moves(6, 4, device="cpu")
    with pytest.raises(ValueError, match="wide"):
        beam.lora_beam_reorder(z(6), 3, z(6), z(6, 4), z(6), z(6, 5), z(3), 9, 16, m)
    with pytest.raises(ValueError, match="rows"):
        beam.lora_beam_reorder(z(6), 3, z(6), z(5, 4), z(6), z(6, 4), z(3), 9, 16, m)
    with pytest.raises(ValueError, match="GPU"):
        beam.lora_beam_reorder(z(6), 3, z(6), z(6, 4), z(6), z(6, 4), z(3), 9, 16, m)
    b, other = kv.Batch(8, 4, 4, 2, 64, device="cpu"), kv.Batch(8, 4, 4, 2, 64, device="cpu")
    sh = kv.Shared(b, 2)
    with pytest.raises(ValueError, match="one entry more"):
        kv.lora_kv_share(z(2), z(2), b, sh)
    with pytest.raises(ValueError, match="another batch"):
        kv.lora_kv_share(z(3), z(2), other, sh)
    with pytest.raises(ValueError, match="unsupported"):
        kv.Shared(b, 5)


# ------------------------------------------------------- the plain references
def test_plain_selection_by_hand():
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.8, 0.1]]))
    p, t, s, n, d, _ = BR.select(x, 2, np.array([-1.0, -1.2]), np.array([3, 3]), np.array([0, 0]), 1, 0.0)
    assert list(p) == [1, 0] and list(t) == [1, 0] and list(d) == [1, 0] and list(n) == [4, 4]
    np.testing.assert_allclose(s, [-1.2 + math.log(0.8), -1.0 + math.log(0.5)])
    p, t, s, n, d, _ = BR.select(x, 2, np.array([-1.0, -1.2]), np.array([3, 3]), np.array([1, 0]), 1, 0.0)
    assert list(p) == [0, 1] and list(t) == [1, 1] and list(n) == [3, 4] and list(d) == [1, 1]


def test_plain_reorder_by_hand():
    table = np.array([[1, 2, -1], [1, 3, -1]])
    r = BR.reorder([1, 1], 2, np.array([20, 20]), table, [9], 10, 16)
    assert r["table"].tolist() == [[1, 3, -1], [1, 9, -1]] and r["copies"] == [(3, 9, 4)] and r["freed"] == [2]
    r = BR.reorder([0, -1], 2, np.array([32, 32]), table, [], 10, 16)
    assert r["table"].tolist() == [[1, 2, -1], [-1, -1, -1]] and not r["copies"] and r["freed"] == [3] and r["flags"] == 0
