"""The attention operators on the GPU against their plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import kv_reference as R
from heterogeneous_adapters_amd import kv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device=DEV)


def tdt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def to_dev(x, dtype):
    return torch.tensor(np.asarray(x, np.float32)).to(tdt(dtype)).to(DEV)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def normal(rng, shape, dtype):
    return R.round_to(rng.standard_normal(shape), dtype)


def make_table(rng, ctx, new, bt, slack=2):
    """Table with cached blocks filled in, free list, number of blocks."""
    ctx, new = np.asarray(ctx), np.asarray(new)
    need = -(-(ctx + new) // bt)
    num = int(need.sum()) + 3
    ids = rng.permutation(num)
    table = np.full((len(ctx), int(need.max(initial=0)) + slack), -7)
    at = 0
    for i in range(len(ctx)):
        h = -(-int(ctx[i]) // bt)
        table[i, :h] = ids[at:at + h]
        at += h
    return table, ids[at:], num


# -------------------------------------------------------------------- build
def run_build(ctx, new, T, table, free, num_blocks, bt, hq=8, hkv=2, cap=None):
    b = kv.Batch(cap or max(T, 1), max(len(ctx), 1), hq, hkv, 64)
    tab = i32(table)
    kv.lora_kv_build(i32(ctx), i32(new), T, tab, i32(free), num_blocks, bt, b)
    torch.cuda.synchronize()
    return b, tab


def check_build(ctx, new, T, table, free, num_blocks, bt, **kw):
    ref = R.build(ctx, new, T, table, free, num_blocks, bt)
    b, tab = run_build(ctx, new, T, table, free, num_blocks, bt, **kw)
    for name in ("q_indptr", "kv_len", "token_seq", "positions", "slots"):
        assert np.array_equal(getattr(b, name).cpu().numpy(), ref[name]), name
    assert np.array_equal(tab.cpu().numpy(), ref["table"])
    c = b.counts.cpu().numpy()
    assert (c[kv.COUNT_TOKENS], c[kv.COUNT_NEW_BLOCKS], c[kv.COUNT_FLAGS]) == (ref["tokens"], ref["new_blocks"], ref["flags"])
    return ref


@pytest.mark.parametrize("B,hi,most_new,bt", [(1, 1, 1, 16), (1, 40, 40, 16), (3, 33, 7, 32), (65, 300, 1, 16),
                                              (1025, 50, 3, 64), (2300, 20, 5, 128), (40, 3000, 1500, 256)])
def test_build_against_plain(B, hi, most_new, bt):
    rng = np.random.default_rng(B + bt)
    total = rng.integers(0, hi + 1, B)
    new = np.minimum(rng.integers(0, most_new + 1, B), total)
    ctx = total - new
    table, free, num = make_table(rng, ctx, new, bt)
    T = int(new.sum())
    check_build(ctx, new, T, table, free, num, bt)
    check_build(ctx, new, T + 77, table, free, num, bt)  # a padded batch


def test_build_of_nothing():
    check_build([], [], 0, np.zeros((0, 1)), [], 1, 16)
    check_build([], [], 5, np.zeros((0, 1)), [], 1, 16)
    check_build([5, 0], [0, 0], 0, [[3], [-1]], [], 4, 16)


@pytest.mark.parametrize("case", ["negative", "past_row", "tokens", "free", "free_mid", "bad_free", "bad_cached"])
def test_build_flags(case):
    ctx, new, T, width, num = [20, 0, 31, 7], [5, 40, 2, 0], 47, 3, 12
    table = np.array([[0, 1, -1], [-1, -1, -1], [2, 3, -1], [4, -1, -1]])
    free = [5, 6, 7, 8, 9]
    if case == "negative":
        ctx, new = [20, 0, 31, -3], [5, 40, 2, -9]
    if case == "past_row":
        ctx, new, T = [20, 0, 31, 7], [5, 400, 60, 0], 465
    if case == "tokens":
        T = 30
    if case == "free":
        free = []
    if case == "free_mid":
        free = [5, 6]
    if case == "bad_free":
        free = [5, 12, -1, 8, 9]
    if case == "bad_cached":
        table[0, 1] = 99
    ref = check_build(ctx, new, T, table, free, num, 16, cap=600)
    assert ref["flags"] != 0


def test_build_again_gives_the_same_and_smaller_steps_reuse_the_buffer():
    rng = np.random.default_rng(3)
    ctx, new = rng.integers(0, 100, 50), rng.integers(0, 9, 50)
    table, free, num = make_table(rng, ctx, new, 16)
    T = int(new.sum())
    b = kv.Batch(T + 100, 80, 4, 4, 32)
    for B in (50, 50, 7, 50):
        tab = i32(table[:B])
        t = int(new[:B].sum())
        ref = R.build(ctx[:B], new[:B], t, table[:B], free, num, 16)
        for _ in range(2):
            kv.lora_kv_build(i32(ctx[:B]), i32(new[:B]), t, tab, i32(free), num, 16, b)
            assert np.array_equal(b.slots.cpu().numpy(), ref["slots"]) and np.array_equal(tab.cpu().numpy(), ref["table"])


# --------------------------------------------------------------------- rope
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,rot", [(1, 1, 1, 32, 32), (5, 3, 2, 64, 64), (17, 4, 1, 96, 48), (9, 8, 8, 128, 64),
                                           (3, 2, 2, 256, 256), (6, 2, 3, 64, 20), (4, 5, 1, 40, 2), (33, 1, 0, 128, 128)])
def test_rope_against_plain(dtype, interleaved, T, hq, hk, D, rot):
    rng = np.random.default_rng(T * D + rot)
    q, k = normal(rng, (T, hq, D), dtype), normal(rng, (T, hk, D), dtype)
    pos = rng.integers(0, 1 << 20, T)
    pos[0] = 0
    freq, scale = R.frequencies(rot, 10000.0, "none", 1.0, 4096)
    rope = kv.Rope(torch.tensor(freq, dtype=torch.float64, device=DEV), int(interleaved), 1.25)
    dq = to_dev(q, dtype)
    qo = torch.full_like(dq, 9.0)
    dk = to_dev(k, dtype) if hk else None
    kv.lora_rope(dq, qo, dk, dk, i32(pos), rope)  # k in place
    torch.cuda.synchronize()
    rq = R.rotate(q, pos, freq, 1.25, interleaved)
    # fp32 cos and sin (2^-24 each), two products and a sum, one rounding of the result
    mag = 1.25 * 1.5 * max(1.0, np.abs(q).max())
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    assert np.all(np.abs(host(qo) - rq) <= half * np.abs(rq) + 6 * 2.0 ** -24 * mag)
    if hk:
        rk = R.round_to(R.rotate(k, pos, freq, 1.25, interleaved), dtype)
        # one rounding of a 64-bit value: the same but for values within 2^-48 of a border
        got = host(dk)
        assert np.all(np.abs(got - rk) <= 2 * half * np.abs(rk)) and np.mean(got != rk) < 1e-3


def test_rope_skips_padded_rows_and_passes_the_tail():
    q = torch.randn((4, 2, 64), device=DEV).bfloat16()
    freq, _ = R.frequencies(32, 10000.0, "none", 1.0, 4096)
    rope = kv.Rope(torch.tensor(freq, dtype=torch.float64, device=DEV))
    out = torch.full_like(q, 3.0)
    kv.lora_rope(q, out, None, None, i32([5, -1, 0, -1]), rope)
    torch.cuda.synchronize()
    assert bool((out[[1, 3]] == 3.0).all())
    assert torch.equal(out[[0, 2]][..., 32:], q[[0, 2]][..., 32:]) and torch.equal(out[2], q[2])


# -------------------------------------------------------------------- cache
def strided(x, dtype, pad_heads):
    """A view with other heads behind each row (a fused projection's rows)."""
    T, H, D = x.shape
    big = torch.full((T, H + pad_heads, D), float("nan"), dtype=tdt(dtype), device=DEV)
    big[:, :H] = to_dev(x, dtype)
    return big[:, :H]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D,bt,scatter", [(1, 1, 32, 16, True), (7, 2, 64, 16, False), (40, 3, 96, 32, False),
                                              (35, 5, 128, 64, True), (70, 8, 128, 16, False), (19, 2, 160, 128, True),
                                              (18, 1, 192, 16, False), (21, 3, 224, 32, False), (33, 2, 256, 256, False)])
def test_append_writes_the_exact_bytes(dtype, T, H, D, bt, scatter):
    rng = np.random.default_rng(T * D)
    blocks = -(-T // bt) * (4 if scatter else 1) + 3
    k, v = normal(rng, (T, H, D), dtype), normal(rng, (T, H, D), dtype) * 2.0 ** rng.integers(-9, 9, (T, H, 1))
    k[0, 0, :32] = 0.0
    if scatter:
        slots = rng.permutation(blocks * bt)[:T]
    else:  # neighbours from an odd place on
        perm = rng.permutation(blocks)
        at = np.arange(5, 5 + T)
        slots = perm[at // bt] * bt + at % bt
    slots = slots.copy()
    if T > 3:
        slots[2], slots[3] = -1, blocks * bt + 5
    nbytes = R.block_bytes(bt, H, D)
    stride = nbytes + 48
    fill = rng.integers(0, 256, (blocks, stride)).astype(np.uint8)
    data = torch.tensor(fill, device=DEV)
    cache = kv.Cache(data, bt, H, D)
    kv.lora_kv_append(None, None, strided(k, dtype, 2), strided(v, dtype, 1), None, i32(slots), None, cache)
    torch.cuda.synchronize()
    want = fill.copy()
    R.put(want, slots, k, v, bt)
    assert np.array_equal(data.cpu().numpy(), want)
    # and back
    ko = torch.full((T, H, D), 7.0, dtype=tdt(dtype), device=DEV)
    vo = torch.full_like(ko, 7.0)
    kv.lora_kv_gather(cache, i32(slots), ko, vo)
    torch.cuda.synchronize()
    rk, rv = R.get(want, slots, H, D, bt)
    assert np.array_equal(host(ko), rk) and np.array_equal(host(vo), rv)


def test_append_of_borders_infinities_and_nan():
    """Every border between codes, largest and smallest scales, values that are none."""
    D = 128
    x = np.zeros((6, 1, D))
    borders = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]
    x[0, 0, :32] = (borders + [-b for b in borders]) * 2
    x[0, 0, 32:64] = [b * 2.0 ** -90 for b in borders] * 4
    x[0, 0, 64:96] = [b * 2.0 ** -120 for b in borders] * 4  # below the smallest scale
    x[0, 0, 96:] = 7.0
    x[1, 0, :32] = 7.0000001 * np.ones(32)
    x[1, 0, 32:64] = R.round_to(3.3e38, "f32")
    x[1, 0, 64] = 7.5
    x[1, 0, 96] = 3.5 + 2.0 ** -21
    x[2, 0, 3], x[2, 0, 4], x[2, 0, 5] = np.nan, 1.0, -2.0
    x[3, 0, 40], x[3, 0, 41], x[3, 0, 42] = np.inf, -np.inf, 0.3
    x[4, 0, :] = np.nan
    x[5, 0, :] = -np.inf
    x = np.where(np.isnan(x) | np.isinf(x), x, x.astype(np.float32).astype(np.float64))
    blocks, bt = 1, 16
    data = torch.zeros((blocks, R.block_bytes(bt, 1, D)), dtype=torch.uint8, device=DEV)
    b = kv.Batch(8, 1, 1, 1, D)
    dev = torch.tensor(x.astype(np.float32), device=DEV)
    kv.lora_kv_append(None, None, dev[:2], dev[:2], None, i32([0, 1]), None, kv.Cache(data, bt, 1, D), b)
    torch.cuda.synchronize()
    assert int(b.flags) == 0
    kv.lora_kv_append(None, None, dev, dev, None, i32(range(6)), None, kv.Cache(data, bt, 1, D), b)
    torch.cuda.synchronize()
    assert int(b.flags) == kv.FLAG_NONFINITE
    want = np.zeros((blocks, R.block_bytes(bt, 1, D)), np.uint8)
    R.put(want, np.arange(6), x, x, bt)
    k, v = R.get(data.cpu().numpy(), np.arange(6), 1, D, bt)
    wk, wv = R.get(want, np.arange(6), 1, D, bt)
    assert np.array_equal(k, wk) and np.array_equal(v, wv) and np.isfinite(k).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,D,rot", [(1, 4, 1, 64, 64), (21, 4, 2, 128, 128), (37, 6, 3, 96, 48), (40, 4, 4, 128, 64),
                                            (18, 2, 1, 256, 256), (20, 5, 5, 160, 80), (9, 1, 1, 64, 30)])
def test_append_with_rope_is_rope_then_append(dtype, interleaved, T, hq, hkv, D, rot):
    rng = np.random.default_rng(T + D)
    q, k, v = (to_dev(rng.standard_normal((T, h, D)), dtype) for h in (hq, hkv, hkv))
    pos = rng.integers(0, 100000, T)
    if T > 4:
        pos[4] = -1
    rope = kv.Rope.scaled(rot, scaling=kv.SCALING_YARN, factor=4.0, original=4096.0, layout=int(interleaved), device=DEV)
    bt, blocks = 16, T + 2
    slots = rng.permutation(blocks * bt)[:T]
    nbytes = R.block_bytes(bt, hkv, D)
    one, two = (torch.zeros((blocks, nbytes), dtype=torch.uint8, device=DEV) for _ in range(2))
    q1, q2, k2 = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k)
    kv.lora_kv_append(q, q1, k, v, i32(pos), i32(slots), rope, kv.Cache(one, bt, hkv, D))
    kv.lora_rope(q, q2, k, k2, i32(pos), rope)
    kv.lora_kv_append(None, None, k2, v, None, i32(np.where(pos < 0, -1, slots)), None, kv.Cache(two, bt, hkv, D))
    torch.cuda.synchronize()
    assert torch.equal(one, two) and torch.equal(q1, q2)
    qin = q.clone()
    kv.lora_kv_append(qin, qin, k, v, i32(pos), i32(slots), rope, kv.Cache(two, bt, hkv, D))
    torch.cuda.synchronize()
    keep = torch.tensor(pos >= 0, device=DEV)
    assert torch.equal(qin[keep], q1[keep]) and torch.equal(qin[~keep], q[~keep])


# ----------------------------------------------------------- cache attention
class Step:
    """A step over a random cache; the plain result of each row."""

    def __init__(self, seed, ctx, new, hq, hkv, D, bt, dtype, pad=0, k_scale=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.ctx, self.new, self.hq, self.hkv, self.D, self.bt, self.dtype = ctx, new, hq, hkv, D, bt, dtype
        table, free, num = make_table(rng, ctx, new, bt)
        self.num, self.free = num, free
        self.T = int(np.sum(new)) + pad
        self.ref = R.build(ctx, new, self.T, table, free, num, bt)
        # every byte of the cache random, scales of unused places too (255: NaN)
        nb = R.block_bytes(bt, hkv, D)
        data = rng.integers(0, 256, (num, nb)).astype(np.uint8)
        used = []
        for i in range(len(ctx)):
            for p in range(int(ctx[i] + new[i])):
                used.append(self.ref["table"][i, p // bt] * bt + p % bt)
        k = R.round_to(rng.standard_normal((len(used), hkv, D)) * k_scale, "bf16")
        v = R.round_to(rng.standard_normal((len(used), hkv, D)), "bf16")
        R.put(data, np.array(used, np.int64), k, v, bt)
        self.data = data
        self.k, self.v = R.get(data, used, hkv, D, bt)
        self.q = normal(rng, (self.T, hq, D), dtype)
        self.table = table

    def rows(self):
        at = 0
        for i in range(len(self.ctx)):
            L = int(self.ctx[i] + self.new[i])
            yield i, slice(int(self.ref["q_indptr"][i]), int(self.ref["q_indptr"][i + 1])), at, L
            at += L

    def run(self, scale, stream=None):
        self.cache = kv.Cache(torch.tensor(self.data, device=DEV), self.bt, self.hkv, self.D)
        self.batch = kv.Batch(self.T + 3, len(self.ctx) + 2, self.hq, self.hkv, self.D)
        self.tab = i32(self.table)
        self.dq = to_dev(self.q, self.dtype)
        self.out = torch.full_like(self.dq, 5.0)
        self.ws = kv.attend_workspace(self.batch)
        kv.lora_kv_build(i32(self.ctx), i32(self.new), self.T, self.tab, i32(self.free), self.num, self.bt, self.batch)
        kv.lora_kv_attend(self.dq, self.out, self.batch, self.tab, self.cache, scale, self.ws)
        torch.cuda.synchronize()
        return host(self.out)

    def check(self, got, scale):
        for i, rows, at, L in self.rows():
            n = rows.stop - rows.start
            sees = self.ctx[i] + np.arange(n) + 1
            o, a, s_abs = R.attend_rows(self.q[rows], self.k[at:at + L], self.v[at:at + L], sees, scale)
            bound = R.attend_bound(o, a, s_abs, L, self.D, self.dtype)
            err = np.abs(got[rows] - o)
            assert np.all(err <= bound), (i, L, float((err / bound).max()))
        end = int(self.ref["q_indptr"][-1])
        assert np.all(got[end:] == 5.0)  # rows behind the last request


ATTEND = [
    # ctx, new, hq, hkv, D, bt
    ([0], [1], 1, 1, 32, 16), ([0, 15, 16, 31, 32, 127, 128], [1] * 7, 4, 1, 64, 16),
    ([300, 5, 0, 129], [1, 1, 1, 1], 8, 8, 128, 32), ([700, 3], [1, 1], 32, 2, 128, 64),
    ([50, 0, 200], [3, 17, 40], 6, 3, 96, 16), ([90, 10], [1, 33], 20, 1, 64, 128), ([130, 0, 7], [1, 1, 0], 5, 5, 160, 16),
    ([260], [5], 7, 1, 192, 256), ([40, 140], [1, 2], 2, 1, 224, 16), ([33, 400], [1, 1], 4, 2, 256, 32),
    ([1500], [1], 2, 1, 64, 16), ([3, 0, 0, 900], [0, 0, 5, 1], 3, 1, 128, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend_against_plain(case, dtype):
    ctx, new, hq, hkv, D, bt = ATTEND[case]
    s = Step(case, np.array(ctx), np.array(new), hq, hkv, D, bt, dtype, pad=case % 3)
    scale = 1.0 / math.sqrt(D)
    s.check(s.run(scale), scale)
    assert int(s.batch.flags) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_peaked_scores(dtype):
    """Scores that grow along the keys and far apart: the running maximum moves often."""
    s = Step(5, np.array([600, 250]), np.array([1, 20]), 4, 2, 64, 16, dtype, k_scale=6.0)
    s.check(s.run(0.9), 0.9)


def test_attend_many_requests():
    rng = np.random.default_rng(9)
    ctx = rng.integers(0, 60, 1100)
    s = Step(11, ctx, np.ones(1100, np.int64), 2, 1, 32, 16, "bf16")
    s.check(s.run(0.3), 0.3)
