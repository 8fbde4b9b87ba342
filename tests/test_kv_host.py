"""Host-side tests of the attention operators: exports, sizes, frequencies and
refusals before any device work, and the plain reference itself (no GPU)."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import kv_reference as R
from heterogeneous_adapters_amd import kv, lora

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lora_kv.h")


def test_library_exports_every_declared_function():
    txt = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    fns = sorted(set(re.findall(r"^(?:size_t|lora_status_t)\s+(lora_[a-z_]+)\s*\(", txt, flags=re.M)))
    assert set(fns) == set(kv.EXPORTS) == set(kv.lib())


def test_binding_constants_match_header():
    defs = dict(re.findall(r"^#define (LORA_[A-Z_0-9]+) \(?([^/\n]*?)\)?\s*(?:/\*.*)?$", open(HEADER).read(), flags=re.M))
    want = {"LORA_KV_MAX_SEQS": kv.MAX_SEQS, "LORA_ROPE_HALF": kv.ROPE_HALF, "LORA_ROPE_INTERLEAVED": kv.ROPE_INTERLEAVED}
    want.update({f"LORA_KV_COUNT_{n}": getattr(kv, f"COUNT_{n}")
                 for n in ("TOKENS", "NEW_BLOCKS", "ITEMS", "PARTS", "CHUNK", "MID", "WIDE", "FLAGS")})
    want.update({f"LORA_KV_FLAG_{n}": getattr(kv, f"FLAG_{n}")
                 for n in ("LENGTH", "TOKENS", "FREE_LIST", "BLOCK_RANGE", "NONFINITE", "BATCH")})
    want.update({f"LORA_ROPE_SCALING_{n}": getattr(kv, f"SCALING_{n}") for n in ("NONE", "LINEAR", "NTK", "YARN", "BANDS")})
    for name, v in want.items():
        assert eval(defs[name].strip()) == v, name


def test_block_bytes():
    for bt in (16, 32, 64, 128, 256):
        for heads in (1, 8, 32):
            for D in range(32, 257, 32):
                assert kv.block_bytes(bt, heads, D) == R.block_bytes(bt, heads, D)
    for bad in ((8, 1, 32), (17, 1, 32), (512, 1, 32), (16, 0, 32), (16, 1, 48), (16, 1, 288), (16, 1, 0), (16, 1025, 32)):
        assert kv.block_bytes(*bad) == 0


def test_batch_limits():
    f = kv.lib()["lora_kv_batch_size"]
    assert f(1024, 1024, 32, 8, 128) > 4 * (1024 * 4)
    for bad in ((-1, 4, 8, 8, 64), (4, 0, 8, 8, 64), (4, (1 << 16) + 1, 8, 8, 64), (4, 4, 8, 3, 64), (4, 4, 4, 8, 64),
                (4, 4, 2048, 8, 64), (4, 4, 8, 8, 40), (lora.LORA_MAX_TOKENS, 4, 64, 8, 64), (lora.LORA_MAX_TOKENS + 1, 4, 8, 8, 64)):
        assert f(*bad) == 0, bad


KINDS = ["none", "linear", "ntk", "yarn", "bands"]


@pytest.mark.parametrize("kind", range(5))
@pytest.mark.parametrize("rot,theta,factor,original", [(128, 1e4, 8.0, 4096.0), (64, 5e5, 32.0, 8192.0), (2, 1e4, 2.0, 64.0),
                                                       (20, 1e6, 1.0, 2048.0), (256, 1e4, 1.5, 100.0)])
def test_frequencies(kind, rot, theta, factor, original):
    got, scale = kv.lora_rope_frequencies(rot, theta, kind, factor, original)
    want, wscale = R.frequencies(rot, theta, KINDS[kind], factor, original)
    assert len(got) == rot // 2
    np.testing.assert_allclose(got, want, rtol=1e-13)
    assert scale == pytest.approx(wscale, rel=1e-15)
    if factor == 1.0:
        np.testing.assert_allclose(got, R.frequencies(rot, theta, "none", 1.0, 0)[0], rtol=1e-13)


@pytest.mark.parametrize("args", [(0, 1e4, 0, 1.0, 1.0), (3, 1e4, 0, 1.0, 1.0), (258, 1e4, 0, 1.0, 1.0), (64, 1.0, 0, 1.0, 1.0),
                                  (64, 1e4, 5, 1.0, 1.0), (64, 1e4, 1, 0.5, 1.0), (64, 1e4, 1, math.nan, 1.0),
                                  (64, 1e4, 3, 2.0, 0.0), (64, 1e4, 4, 2.0, 100.0, 4.0, 2.0), (64, 1e4, 2, math.inf, 1.0)])
def test_frequencies_refusals(args):
    with pytest.raises(lora.LoraError) as e:
        kv.lora_rope_frequencies(*args)
    assert e.value.status == -1


# ---------------------------------------------------------------- refusals
class Args:
    """Valid arguments on host memory that stands in for device memory: every
    call below is refused before anything is enqueued."""

    def __init__(self):
        self.mem = np.zeros(1 << 16, np.uint8)
        base = self.mem.ctypes.data
        self.p = base + (-base) % 256
        self.batch = kv.lora_kv_batch_t()
        f = kv.lib()["lora_kv_batch_init"]
        assert f(self.p, 1 << 30, 64, 8, 8, 2, 64, ctypes.addressof(self.batch)) == 0
        self.cache = kv.lora_kv_cache_t(self.p, R.block_bytes(16, 2, 64), 16, 16, 2, 64)
        self.rope = kv.lora_rope_t(self.p, 64, 0, 1.0)

    def heads(self, n, off=0, ts=None, hs=64):
        return kv.lora_heads_t(self.p + 4096 * off, n * 64 if ts is None else ts, hs, n)


def ref(x):
    return None if x is None else ctypes.addressof(x)


def test_batch_init_refusals():
    a, f = Args(), kv.lib()["lora_kv_batch_init"]
    out = kv.lora_kv_batch_t()
    n = kv.lib()["lora_kv_batch_size"](64, 8, 8, 2, 64)
    assert f(a.p, n, 64, 8, 8, 2, 64, ref(out)) == 0
    assert f(None, n, 64, 8, 8, 2, 64, ref(out)) == -1
    assert f(a.p, n, 64, 8, 8, 2, 64, None) == -1
    assert f(a.p, n, -1, 8, 8, 2, 64, ref(out)) == -1
    assert f(a.p, n - 1, 64, 8, 8, 2, 64, ref(out)) == -4
    assert f(a.p + 4, n, 64, 8, 8, 2, 64, ref(out)) == -7
    assert f(a.p, n, 64, 8, 8, 3, 64, ref(out)) == -6


def build_args(a, **kw):
    d = dict(ctx=a.p, new=a.p, B=4, T=16, table=a.p, stride=8, width=8, free=a.p, nfree=4, nb=16, bt=16, batch=ref(a.batch))
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw,code", [
    (dict(ctx=None), -1), (dict(new=None), -1), (dict(table=None), -1), (dict(batch=None), -1), (dict(B=-1), -1), (dict(T=-1), -1),
    (dict(free=None), -1), (dict(nfree=-1), -1), (dict(width=0), -1), (dict(stride=7), -1), (dict(nb=0), -1), (dict(bt=24), -6),
    (dict(bt=0), -6), (dict(nb=1 << 28, bt=16), -6), (dict(B=9), -4), (dict(T=65), -4),
])
def test_build_refusals(kw, code):
    assert kv.lib()["lora_kv_build"](*build_args(Args(), **kw)) == code


@pytest.mark.parametrize("which", ["ctx", "new", "table", "free"])
def test_build_refuses_inputs_in_its_own_batch(which):
    a = Args()
    outside = a.p + (1 << 15)
    # the batch of Args starts at a.p: a copy of it elsewhere leaves the other inputs outside
    assert kv.lib()["lora_kv_batch_init"](outside, 1 << 30, 64, 8, 8, 2, 64, ctypes.addressof(a.batch)) == 0
    assert kv.lib()["lora_kv_build"](*build_args(a, **{which: a.batch.kv_len})) == -1


@pytest.mark.parametrize("case,code", [
    ("null_q", -1), ("null_pos", -1), ("neg_T", -1), ("dtype", -6), ("dim", -6), ("odd_rot", -1), ("rot_past", -1), ("layout", -6),
    ("null_freq", -1), ("stride", -7), ("short_stride", -1), ("base", -7), ("heads", -1), ("out_missing", -1), ("in_place", -1),
    ("many_heads", -6), ("null_rope", -1),
])
def test_rope_refusals(case, code):
    a = Args()
    q, qo, pos, T, D, dt, rope = a.heads(4), a.heads(4, 1), a.p, 8, 64, lora.LORA_DTYPE_BF16, a.rope
    if case == "null_q":
        q.data = None
    if case == "null_pos":
        pos = None
    if case == "neg_T":
        T = -1
    if case == "dtype":
        dt = 2
    if case == "dim":
        D = 60
    if case == "odd_rot":
        rope.rot_dim = 7
    if case == "rot_past":
        rope.rot_dim = 66
    if case == "layout":
        rope.layout = 2
    if case == "null_freq":
        rope.inv_freq = None
    if case == "stride":
        q.token_stride = 260
    if case == "short_stride":
        q.token_stride = 56
    if case == "base":
        qo.data = a.p + 8
    if case == "heads":
        qo.heads = 3
    if case == "out_missing":
        qo = None
    if case == "in_place":
        qo = a.heads(4, 0, ts=512)
    if case == "many_heads":
        q.heads = qo.heads = 1025
    if case == "null_rope":
        rope = None
    assert kv.lib()["lora_rope"](ref(q), ref(qo), None, None, pos, T, D, dt, ref(rope), None) == code


@pytest.mark.parametrize("case,code", [
    ("null_k", -1), ("null_slots", -1), ("null_pos", -1), ("null_cache", -1), ("kv_heads", -1), ("v_heads", -1), ("dtype", -6),
    ("block_tokens", -6), ("cache_dim", -6), ("short_block", -1), ("block_align", -7), ("base_align", -7), ("slots_range", -6),
    ("q_stride", -7), ("q_out", -1), ("T", -1),
])
def test_append_and_gather_refusals(case, code):
    a = Args()
    q, qo, k, v, pos, slots, T, dt, rope, cache = (a.heads(4), a.heads(4, 1), a.heads(2, 2), a.heads(2, 3), a.p, a.p, 8,
                                                   lora.LORA_DTYPE_BF16, a.rope, a.cache)
    if case == "null_k":
        k = None
    if case == "null_slots":
        slots = None
    if case == "null_pos":
        pos = None
    if case == "null_cache":
        cache = None
    if case == "kv_heads":
        k.heads = 3
    if case == "v_heads":
        v.heads = 1
    if case == "dtype":
        dt = -1
    if case == "block_tokens":
        cache.block_tokens = 48
    if case == "cache_dim":
        cache.head_dim = 80
    if case == "short_block":
        cache.block_stride -= 16
    if case == "block_align":
        cache.block_stride += 8
    if case == "base_align":
        cache.base = a.p + 8
    if case == "slots_range":
        cache.num_blocks, cache.block_tokens, cache.block_stride = 1 << 27, 16, 1 << 20
    if case == "q_stride":
        q.token_stride = 258
    if case == "q_out":
        qo = None
    if case == "T":
        T = -5
    assert kv.lib()["lora_kv_append"](ref(q), ref(qo), ref(k), ref(v), pos, slots, T, dt, ref(rope), ref(cache), None, None) == code
    if case not in ("null_pos", "q_stride", "q_out"):
        assert kv.lib()["lora_kv_gather"](ref(cache), slots, T, ref(k), ref(v), dt, None) == code


@pytest.mark.parametrize("case,code", [
    ("null_q", -1), ("heads", -1), ("kv_heads", -1), ("dim", -1), ("same", -1), ("scale", -1), ("scale_nan", -1), ("scale_inf", -1),
    ("null_ws", -1), ("ws", -4), ("ws_align", -7), ("T", -4), ("B", -4), ("null_table", -1), ("width", -1), ("dtype", -6),
    ("batch", -1), ("stride", -7),
])
def test_attend_refusals(case, code):
    a = Args()
    q, o, T, B, dt, batch, table, stride, width, cache, scale, ws = (a.heads(8), a.heads(8, 1), 8, 4, lora.LORA_DTYPE_BF16, a.batch,
                                                                    a.p, 4, 4, a.cache, 0.1, a.p)
    n = kv.lib()["lora_kv_workspace_size"](ref(batch))
    assert n > 0
    if case == "null_q":
        q = None
    if case == "heads":
        q.heads = o.heads = 4
    if case == "kv_heads":
        cache.num_kv_heads = 1
    if case == "dim":
        cache.head_dim = 32
    if case == "same":
        o = q
    if case == "scale":
        scale = 0.0
    if case == "scale_nan":
        scale = math.nan
    if case == "scale_inf":
        scale = math.inf
    if case == "null_ws":
        ws = None
    if case == "ws":
        n -= 1
    if case == "ws_align":
        ws = a.p + 4
    if case == "T":
        T = 65
    if case == "B":
        B = 9
    if case == "null_table":
        table = None
    if case == "width":
        stride = 3
    if case == "dtype":
        dt = 3
    if case == "batch":
        batch.plan = None
    if case == "stride":
        o.head_stride = 68
    assert kv.lib()["lora_kv_attend"](ref(q), ref(o), T, B, dt, ref(batch), table, stride, width, ref(cache), scale, ws, n, None) == code


@pytest.mark.parametrize("case,code", [
    ("null_v", -1), ("kv", -1), ("group", -1), ("o_heads", -1), ("same", -1), ("indptr", -1), ("B", -1), ("T", -1), ("dim", -6),
    ("big_dim", -6), ("seqs", -6), ("scale", -1), ("dtype", -6), ("align", -7), ("far", -6),
])
def test_prompt_refusals(case, code):
    a = Args()
    q, k, v, o, ptr, B, T, D, dt, scale = (a.heads(8), a.heads(2, 1), a.heads(2, 2), a.heads(8, 3), a.p, 2, 8, 64,
                                           lora.LORA_DTYPE_BF16, 0.1)
    if case == "null_v":
        v.data = None
    if case == "kv":
        v.heads = 4
    if case == "group":
        k.heads = v.heads = 3
    if case == "o_heads":
        o.heads = 4
    if case == "same":
        o = q
    if case == "indptr":
        ptr = None
    if case == "B":
        B = -1
    if case == "T":
        T = -1
    if case == "dim":
        D = 48
    if case == "big_dim":
        D = 288
    if case == "seqs":
        B = (1 << 16) + 1
    if case == "scale":
        scale = -1.0
    if case == "dtype":
        dt = 9
    if case == "align":
        k.data = a.p + 2
    if case == "far":
        k.token_stride = 1 << 25
    assert kv.lib()["lora_prompt_attend"](ref(q), ref(k), ref(v), ref(o), ptr, B, T, D, dt, scale, None) == code


def test_nothing_to_do_needs_no_device():
    a, L = Args(), kv.lib()
    q, k, o = a.heads(8), a.heads(2), a.heads(8, 1)
    assert L["lora_rope"](ref(q), ref(o), None, None, None, 0, 64, 1, ref(a.rope), None) == 0
    assert L["lora_rope"](None, None, None, None, a.p, 4, 64, 1, ref(a.rope), None) == 0
    assert L["lora_kv_append"](None, None, ref(k), ref(k), None, None, 0, 1, None, ref(a.cache), None, None) == 0
    assert L["lora_kv_gather"](ref(a.cache), None, 0, ref(k), ref(k), 1, None) == 0
    assert L["lora_prompt_attend"](ref(q), ref(k), ref(k), ref(o), None, 0, 0, 64, 1, 0.1, None) == 0
    n = L["lora_kv_workspace_size"](ref(a.batch))
    assert L["lora_kv_attend"](ref(q), ref(o), 0, 0, 1, ref(a.batch), None, 0, 0, ref(a.cache), 0.1, a.p, n, None) == 0


# ------------------------------------------------------------- the binding
def test_binding_refuses_host_tensors_and_wrong_shapes():
    q, pos = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    rope = kv.Rope(torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="GPU"):
        kv.lora_rope(q, q, None, None, pos, rope)
    with pytest.raises(ValueError, match="rows"):
        kv.lora_rope(q, q, None, None, pos[:3], rope)
    with pytest.raises(ValueError, match="int32"):
        kv.lora_rope(q, q, None, None, pos.long(), rope)
    with pytest.raises(ValueError, match="type"):
        kv.lora_rope(q, q.float(), None, None, pos, rope)
    with pytest.raises(ValueError, match="unsupported dtype"):
        kv.lora_rope(q.half(), q.half(), None, None, pos, rope)
    with pytest.raises(ValueError, match="contiguous"):
        kv.lora_rope(q.transpose(1, 2), q, None, None, pos, rope)
    with pytest.raises(ValueError, match="q_out"):
        kv.lora_rope(q, None, None, None, pos, rope)
    with pytest.raises(ValueError, match="head_dim"):
        kv.lora_prompt_attend(q, q[..., :32], q, torch.empty_like(q), pos, 0.1)
    with pytest.raises(ValueError, match="GPU"):
        kv.lora_prompt_attend(q, q, q, torch.empty_like(q), pos, 0.1)
    with pytest.raises(ValueError):
        kv.Rope(torch.zeros(32))
    data = torch.zeros((4, kv.block_bytes(16, 2, 64)), dtype=torch.uint8)
    cache = kv.Cache(data, 16, 2, 64)
    with pytest.raises(ValueError, match="rope, or no q"):
        kv.lora_kv_append(q, q, q, q, None, pos, None, cache)
    with pytest.raises(ValueError, match="positions"):
        kv.lora_kv_append(None, None, q, q, None, pos, rope, cache)
    with pytest.raises(ValueError, match="GPU"):
        kv.lora_kv_append(None, None, q, q, None, pos, None, cache)
    with pytest.raises(ValueError):
        kv.Cache(data, 32, 2, 64)
    with pytest.raises(ValueError):
        kv.Cache(data.int(), 16, 2, 64)
    with pytest.raises(ValueError):
        kv.Cache(data, 24, 2, 64)
    with pytest.raises(ValueError):
        kv.Batch(4, 4, 8, 3, 64, device="cpu")
    b = kv.Batch(8, 4, 4, 2, 64, device="cpu")
    table = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        kv.lora_kv_build(pos[:2], pos[:2], 4, table, pos, 4, 16, b)
    with pytest.raises(ValueError, match="one table row"):
        kv.lora_kv_build(pos[:3], pos[:3], 4, table, pos, 4, 16, b)
    with pytest.raises(ValueError, match="rows"):
        kv.lora_kv_attend(q, q, b, table, cache, 0.1, data)


def test_a_pool_gives_a_cache():
    pool = lora.Pool(torch.zeros((6, 16 * 128), dtype=torch.bfloat16), 128)
    c = kv.Cache.in_pool(pool, 16, 1, 64)
    assert c.num_blocks == 6 and c.c.block_stride == 16 * 128 * 2 and c.c.base == pool.base.data_ptr()
    with pytest.raises(ValueError):
        kv.Cache.in_pool(pool, 256, 8, 256)


# ----------------------------------------------------------- the reference
def test_reference_codes():
    """Every code is the nearest of its scale, ties to the even code, scales the least that hold the group."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 32)) * 2.0 ** rng.integers(-60, 60, (200, 1))
    code, byte = R.quantise(x)
    v = R.values(code, byte)
    scale = 2.0 ** (byte[:, None] - 127.0)
    grid = np.concatenate([-R.CODES[::-1], R.CODES])
    best = np.abs(x[..., None] / scale[..., None] - grid).min(-1)
    assert np.allclose(np.abs(x - v) / scale, best, rtol=1e-12)
    most = np.abs(x).max(1)
    assert np.all(most <= 7 * scale[:, 0]) and np.all(most > 7 * scale[:, 0] / 2)
    assert list(R.quantise(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0] * 4))[0][:8]) == [0, 2, 2, 4, 4, 6, 6, 7]


def test_reference_cache_round_trip():
    rng = np.random.default_rng(1)
    for D in (32, 96, 128, 256):
        k, v = rng.standard_normal((20, 2, D)), rng.standard_normal((20, 2, D))
        data = rng.integers(0, 256, (4, R.block_bytes(32, 2, D))).astype(np.uint8)
        slots = rng.permutation(128)[:20]
        R.put(data, slots, k, v, 32)
        gk, gv = R.get(data, slots, 2, D, 32)
        for x, g in ((k, gk), (v, gv)):
            c, b = R.quantise(x.reshape(20, 2, -1, 32))
            assert np.array_equal(g.reshape(20, 2, -1, 32), R.values(c, b))


def test_binding_refuses_block_tables_whose_rows_overlap():
    """A row stride below the width (an expanded row, overlapping rows) would address rows behind the tensor."""
    pos, b = torch.zeros(4, dtype=torch.int32), kv.Batch(8, 4, 4, 2, 64, device="cpu")
    data = torch.zeros((4, kv.block_bytes(16, 2, 64)), dtype=torch.uint8)
    cache, ws = kv.Cache(data, 16, 2, 64), kv.attend_workspace(b)
    b._resize(4, 4)
    q = torch.zeros((4, 4, 64), dtype=torch.bfloat16)
    row = torch.zeros((1, 8), dtype=torch.int32)
    for bad in (row.expand(4, 8), torch.as_strided(torch.zeros(32, dtype=torch.int32), (4, 8), (7, 1))):
        with pytest.raises(ValueError, match="block_table"):
            kv.lora_kv_build(pos, pos, 4, bad, pos, 4, 16, b)
        with pytest.raises(ValueError, match="block_table"):
            kv.lora_kv_attend(q, torch.empty_like(q), b, bad, cache, 0.1, ws)
    # rows apart, and a single row of any stride, go on to the check of the device
    for good in (torch.zeros((4, 8), dtype=torch.int32), torch.zeros((4, 11), dtype=torch.int32)[:, :8]):
        with pytest.raises(ValueError, match="GPU"):
            kv.lora_kv_build(pos, pos, 4, good, pos, 4, 16, b)
        with pytest.raises(ValueError, match="GPU"):
            kv.lora_kv_attend(q, torch.empty_like(q), b, good, cache, 0.1, ws)
    one = torch.as_strided(torch.zeros(8, dtype=torch.int32), (1, 8), (0, 1))
    with pytest.raises(ValueError, match="GPU"):
        kv.lora_kv_build(pos[:1], pos[:1], 4, one, pos, 4, 16, b)


def test_binding_refuses_workspaces_that_are_not_contiguous():
    """An expanded tensor counts more elements than it has memory for."""
    b = kv.Batch(8, 4, 4, 2, 64, device="cpu")
    data = torch.zeros((4, kv.block_bytes(16, 2, 64)), dtype=torch.uint8)
    cache, ws, table = kv.Cache(data, 16, 2, 64), kv.attend_workspace(b), torch.zeros((4, 8), dtype=torch.int32)
    b._resize(4, 4)
    q = torch.zeros((4, 4, 64), dtype=torch.bfloat16)
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(ws.numel()), torch.zeros(2 * ws.numel(), dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="ws"):
            kv.lora_kv_attend(q, torch.empty_like(q), b, table, cache, 0.1, bad)
    with pytest.raises(ValueError, match="GPU"):
        kv.lora_kv_attend(q, torch.empty_like(q), b, table, cache, 0.1, ws)


@pytest.mark.parametrize("which,count", [("ctx", 4), ("new", 4), ("table", 3 * 8 + 8), ("free", 4)])
def test_build_refuses_inputs_that_reach_into_its_batch(which, count):
    """Not only those that start there.  `count`: entries that the call may touch."""
    a = Args()
    outside = a.p + (1 << 15)
    assert kv.lib()["lora_kv_batch_init"](outside, 1 << 30, 64, 8, 8, 2, 64, ctypes.addressof(a.batch)) == 0
    n = kv.lib()["lora_kv_batch_size"](64, 8, 8, 2, 64)
    for at in (outside - 4, outside - 4 * (count - 1), outside + n - 4):
        assert kv.lib()["lora_kv_build"](*build_args(a, **{which: at})) == -1
    # one that ends where the batch begins passes this check and is refused for T alone


@pytest.mark.parametrize("bt", [16, 64, 256])
def test_build_refuses_rows_of_more_than_2_30_tokens(bt):
    """The kernels count a request's tokens, and steps past its last, in 32 bits."""
    width = (1 << 30) // bt
    for w, code in ((width, -4), (width + 1, -6), (1 << 30, -6)):  # the first is refused for its B alone
        assert kv.lib()["lora_kv_build"](*build_args(Args(), B=9, width=w, stride=1 << 30, nb=16, bt=bt)) == code


# ----------------------------------------------------- the plan's arithmetic
PLAN = r"""
#include "lora_kv_plan.h"
using namespace lora::kv;
extern "C" {
long long plan_item_cap(long long T, long long B, long long hkv, long long G) { return item_cap(T, B, hkv, G); }
long long plan_class_cap(int c, long long T, long long B, long long hkv, long long G) { return class_cap(c, T, B, hkv, G); }
int plan_even_chunk(int kv, int chunk) { return even_chunk(kv, chunk); }
int plan_last_row(int first, int rows, int len) { return last_row(first, rows, len); }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(PLAN)
    csrc = os.path.join(ROOT, "heterogeneous_adapters_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{csrc}", str(at / "plan.cpp"), "-o", str(at / "plan.so")], check=True)
    lib = ctypes.CDLL(str(at / "plan.so"))
    lib.plan_item_cap.restype = lib.plan_class_cap.restype = ctypes.c_longlong
    lib.plan_item_cap.argtypes, lib.plan_class_cap.argtypes = [ctypes.c_longlong] * 4, [ctypes.c_int] + [ctypes.c_longlong] * 4
    return lib


@pytest.mark.parametrize("hkv,G", [(1, 1), (8, 1), (8, 4), (2, 17), (32, 1), (1, 32), (128, 2), (1, 1024), (1024, 1)])
def test_a_launch_stays_within_its_list_of_items(plan, hkv, G):
    """Each class's grid is no longer than the list its descriptors are read from, whatever the step and the batch's capacity."""
    for B in (1, 2, 3, 17, 100, 1000, 5000):
        for T in (1, 2, B - 1, B, B + 1, B + 17, 2 * B, 16 * B, 1000 * B):
            if T < 1:
                continue
            for most_t, most_b in ((T, B), (T + 5, B), (T, B + 9)):
                room = plan.plan_item_cap(most_t, most_b, hkv, G)
                for c in range(3) if T > B else (0,):  # the launches of the step
                    assert plan.plan_class_cap(c, T, B, hkv, G) <= room, (c, T, B)


@pytest.mark.parametrize("seed", range(40))
def test_a_launch_covers_its_items(plan, seed):
    """The items of a step, by the plan's rules, are no more than the work-groups of each class's launch."""
    rng = np.random.default_rng(seed)
    for _ in range(30):
        hkv, G = int(rng.choice([1, 2, 8, 32, 128])), int(rng.choice([1, 2, 4, 7, 16, 33]))
        B = int(np.exp(rng.uniform(0, 6)))
        new = np.floor(np.exp(rng.uniform(0, rng.choice([0.1, 2.0, 6.0]), B)) - rng.choice([0.0, 0.6])).astype(np.int64)
        ctx = np.floor(np.exp(rng.uniform(0, 10, B)) - 1).astype(np.int64)
        T = int(rng.integers(1, max(new.sum(), 1) + 2)) if rng.random() < 0.3 else int(new.sum()) + int(rng.integers(0, 3))
        add = np.minimum(new, T)
        many = T > B
        last = np.minimum(np.cumsum(add), T)
        rows = np.diff(np.concatenate([[0], last])) * G
        cls = np.where((add * G <= 16) | (not many), 0, np.where(add * G <= 64, 1, 2))
        per = np.array([16, 32, 128])[cls]
        chunk = np.zeros(3, np.int64)
        for group, target in (((0, 1), 1024), ((2,), 512)):
            mine = np.isin(cls, group)
            reads = int((-(-(add * G) // per) * (ctx + add))[mine].sum())
            chunk[list(group)] = max(-(-(-(-reads * hkv // target)) // 256) * 256, 1024)
        items = np.zeros(3, np.int64)
        for i in range(B):
            kv_i = int(ctx[i] + rows[i] // G)
            even = plan.plan_even_chunk(kv_i, int(chunk[cls[i]]))
            items[cls[i]] += -(-int(rows[i]) // per[i]) * max(-(-kv_i // even), 1)
        for c in range(3):
            if c == 0 or many:
                assert items[c] <= plan.plan_class_cap(c, T, B, hkv, G), (c, T, B, hkv, G)
            else:
                assert items[c] == 0


def test_waves_without_rows_take_no_keys(plan):
    """The steps over a prompt's keys that its waves of 32 rows take: those of the rows that are there."""
    for n in (1, 5, 31, 32, 33, 64, 65, 97, 127, 128, 129, 4097):
        for tile in range(-(-n // 128)):
            for wave in range(4):
                first = 128 * tile + 32 * wave
                rows = min(max(n - first, 0), 32)
                last = plan.plan_last_row(first, 32, n)
                assert len(range(0, last + 1, 32)) == (-(-(first + rows) // 32) if rows else 0), (n, first)
                assert [r for r in range(first, first + 32) if r <= last] == list(range(first, first + rows))
