"""The attention operators over the rest of their range: weights that sum to
one, scores far from zero, fp32 queries rotated in 64 bits,
every head dim of the 128-row kernel, rows in several tiles of a decode step,
items without room for partial results."""
import math

import numpy as np
import pytest
import torch

import kv_reference as R
from heterogeneous_adapters_amd import kv
from test_gpu_kv import DEV, Step, host, i32, make_table, normal, to_dev
from test_gpu_prompt import run_prompt

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ sums of weights
# The second product takes weights rounded to bf16 (bf16 q, k and v), and the
# sum that divides it is of the same rounded weights.  With every visible V
# the same bf16 number v the result is v * S / S: each product is exact in
# fp32, the two sums of n terms, the reciprocal and the last product are off by
# (2 n + 2) * 2^-24 of it, below the 2^-9 that rounding back to v allows while
# n < 2^14.
#
# The keys make one weight count: the first token's score is 0, the others'
# -20, but for token 130, whose score of just over 7 leaves the running maximum
# where it is and has a weight of 128.4 to 131.6, far from the bf16 numbers 128,
# 129, ..  Sums of the unrounded weights would be off by up to 0.38 % of it, more
# than half a step of v.
STAR = 130
TWISTS = [0.42, 0.58, 1.42, 1.58, 2.42, 2.58, 3.42, 3.58]  # over 128


def star(rows, heads, hkv, dim):
    """q (rows, heads, dim) and k (rows, hkv, dim) of such scores in powers of two."""
    q, k = np.zeros((rows, heads, dim)), np.zeros((rows, hkv, dim))
    q[..., 0], q[..., 1], q[..., 2] = 7.0, R.bf16([math.log2(1 + TWISTS[h % 8] / 128) for h in range(heads)]), 5.0
    k[..., 2] = -4.0
    k[0] = 0.0
    if rows > STAR:
        k[STAR] = 0.0
        k[STAR, :, :2] = 1.0
    return q, k


def test_star_weights_lie_between_bf16_numbers():
    q, _ = star(1, 8, 1, 32)
    p = 2.0 ** (q[0, :, 0] + q[0, :, 1])
    off = np.abs(R.bf16(p) - p) / p
    assert np.all((p > 128.4) & (p < 131.6)) and np.all(off > 0.0025)


@pytest.mark.parametrize("lens,hq,hkv,D", [([140], 8, 2, 32), ([150, 5], 8, 8, 64), ([133], 8, 1, 96), ([300, 200], 8, 2, 128),
                                           ([140], 8, 1, 160), ([132], 8, 2, 192), ([140], 8, 1, 224), ([160], 8, 2, 256)])
def test_prompt_weights_sum_to_one(lens, hq, hkv, D):
    indptr = np.concatenate([[0], np.cumsum(lens)])
    parts = [star(n, hq, hkv, D) for n in lens]
    q, k = (np.concatenate([p[i] for p in parts]) for i in (0, 1))
    v = np.broadcast_to(1.9921875 * 2.0 ** (np.arange(D) % 17 - 8), k.shape).copy()
    v[..., 1::3] *= -1
    got = run_prompt(q, k, v, indptr, math.log(2.0), "bf16")
    assert np.array_equal(got, np.repeat(v, hq // hkv, axis=1))


def put_step(s, q, k, v):
    """Queries and cached keys and values of a Step, which 4 bits hold exactly."""
    slots = np.array([s.ref["table"][i, p // s.bt] * s.bt + p % s.bt for i in range(len(s.ctx)) for p in range(int(s.ctx[i] + s.new[i]))])
    s.q, s.k, s.v = q, k, np.broadcast_to(v, k.shape).copy()
    R.put(s.data, slots, s.k, s.v, s.bt)
    for got, want in zip(R.get(s.data, slots, s.hkv, s.D, s.bt), (s.k, s.v)):
        assert np.array_equal(got, want)


@pytest.mark.parametrize("ctx,new,hq,hkv,D,bt", [([STAR, 200, 3], [1] * 3, 8, 2, 64, 16), ([2500], [1], 8, 1, 128, 32), ([STAR], [1], 8, 2, 160, 16),
                                                 ([140, 5], [4, 1], 8, 1, 96, 16), ([100, 3], [80, 1], 8, 8, 128, 64), ([1500], [20], 8, 1, 64, 16),
                                                 ([120], [70], 8, 8, 256, 16), ([STAR], [1], 8, 8, 256, 16)])
def test_cache_weights_sum_to_one(ctx, new, hq, hkv, D, bt):
    s = Step(60 + D, np.array(ctx), np.array(new), hq, hkv, D, bt, "bf16")
    k = np.concatenate([star(c + n, hq, hkv, D)[1] for c, n in zip(ctx, new)])
    v = np.tile([6.0, -3.0, 1.5, 6.0], D // 4)
    put_step(s, star(s.T, hq, 1, D)[0], k, v)
    got = s.run(math.log(2.0))
    assert np.array_equal(got, np.broadcast_to(v, got.shape))


# ------------------------------------------------------- scores far from zero
# Scores of +-2^60 and beyond, up to the end of fp32: q has one dim that is not
# zero, so that every score is one exact product.  At these sizes the weights
# are 1 for the largest score and 0 for every lower one (steps of a factor of
# 1.5), so a row is the mean of V over the keys that share the largest score:
# sums of at most n equal weights, one reciprocal and one product, (n + 4)
# roundings of 2^-24 of the mean of |V|, and one rounding of the result.
FAR = [(30, 1), (31, -1), (33, 1), (47, -1), (60, 1), (106, -1), (106, 1), (124, -1), (124, 1)]


def far_rows(level, v, sees, G):
    """Mean of V over the keys of the highest level, and the mean of |V|.  level (L,), v (L, hkv, D)."""
    o, a = (np.zeros((len(sees), v.shape[1] * G, v.shape[2])) for _ in range(2))
    for j, n in enumerate(sees):
        best = level[:n] == level[:n].max()
        o[j], a[j] = np.repeat(v[:n][best].mean(0), G, axis=0), np.repeat(np.abs(v[:n][best]).mean(0), G, axis=0)
    return o, a


def far_check(got, o, a, n, dtype):
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    bad = ~(np.abs(got - o) <= half * np.abs(o) + (n + 4) * 2.0 ** -24 * a * (1 + half))
    assert not bad.any(), np.argwhere(bad)[:5]


@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("power,sign", FAR)
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_prompt_scores_far_from_zero(dtype, D, power, sign, order):
    rng = np.random.default_rng(power)
    T, hq, hkv = 150, 2, 1
    c = rng.choice([1.0, 1.5, 2.0, 3.0], T)
    if order != "mixed":
        c = np.sort(c)[:: 1 if order == "up" else -1]
    q, k = np.zeros((T, hq, D)), np.zeros((T, hkv, D))
    q[..., 0] = sign * 2.0 ** (power // 2)
    k[..., 0] = c[:, None] * 2.0 ** (power - power // 2)
    v = normal(rng, (T, hkv, D), dtype)
    got = run_prompt(q, k, v, [0, T], 1.0, dtype)
    o, a = far_rows(sign * c, v, np.arange(1, T + 1), hq // hkv)
    far_check(got, o, a, T, dtype)


@pytest.mark.parametrize("power,sign", FAR)
@pytest.mark.parametrize("ctx,new,D,dtype", [([0, 2100, 40], [1, 1, 1], 64, "bf16"), ([70, 2], [30, 1], 128, "bf16"),
                                             ([1200, 0], [90, 1], 64, "bf16"), ([30, 0], [70, 1], 256, "bf16"),
                                             ([0, 1100], [1, 1], 64, "f32"), ([60], [50], 96, "f32")])
def test_cache_scores_far_from_zero(ctx, new, D, dtype, power, sign):
    s = Step(70 + D, np.array(ctx), np.array(new), 2, 1, D, 16, dtype)
    level = s.rng.choice([1.0, 1.5, 2.0, 3.0], len(s.k))
    k = np.zeros_like(s.k)
    k[..., 0] = level[:, None] * 2.0 ** (power - power // 2)
    q = np.zeros_like(s.q)
    q[..., 0] = sign * 2.0 ** (power // 2)
    put_step(s, q, k, s.v)
    got = s.run(1.0)
    for i, rows, at, L in s.rows():
        o, a = far_rows(sign * level[at:at + L], s.v[at:at + L], s.ctx[i] + np.arange(rows.stop - rows.start) + 1, 2)
        far_check(got[rows], o, a, L, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_with_ordinary_and_far_scores_side_by_side(dtype):
    """Query heads of one tile: one with scores of 2^100, one of ordinary size, one that is all zeros."""
    D, T = 64, 100
    rng = np.random.default_rng(2)
    q, k, v = normal(rng, (T, 3, D), dtype), normal(rng, (T, 1, D), dtype), normal(rng, (T, 1, D), dtype)
    q[:, 2] = 0.0
    far = q.copy()
    far[:, 0] *= 2.0 ** 100
    scale = 1.0 / math.sqrt(D)
    got, want = run_prompt(far, k, v, [0, T], scale, dtype), run_prompt(q, k, v, [0, T], scale, dtype)
    assert np.array_equal(got[:, 1:], want[:, 1:]) and np.isfinite(got).all()
    s = Step(90, np.array([90]), np.array([5]), 3, 1, D, 16, dtype)
    plain = s.run(scale)
    s.q[:, 0] *= 2.0 ** 100
    mixed = s.run(scale)
    # a tile's rows share the form of their weights, which differs by one rounding of the score
    o, a, s_abs = R.attend_rows(s.q[:, 1:], np.repeat(s.k, 2, 1), np.repeat(s.v, 2, 1), 91 + np.arange(5), scale)
    extra = 2.0 ** -8 * np.abs(o) if dtype == "bf16" else 0.0  # the sum is of rounded weights too
    assert np.all(np.abs(mixed[:, 1:] - o) <= R.attend_bound(o, a, s_abs, 95, D, dtype) + extra)
    assert np.isfinite(mixed).all() and np.isfinite(plain).all()


# ---------------------------------------------------------- rotation in 64 bits
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,rot", [(9, 8, 2, 128, 128), (5, 3, 0, 64, 20), (17, 4, 4, 256, 128), (1, 1, 1, 32, 32)])
def test_fp32_queries_are_rotated_in_64_bits_and_rounded_once(T, hq, hk, D, rot, interleaved):
    rng = np.random.default_rng(T + D)
    q, k, v = (normal(rng, (T, max(h, 1), D), "f32") for h in (hq, hk, hk))
    pos = rng.integers(0, 1 << 16, T)
    freq, scale = R.frequencies(rot, 10000.0, "yarn", 8.0, 4096)
    rope = kv.Rope(torch.tensor(freq, dtype=torch.float64, device=DEV), int(interleaved), scale)
    want = R.round_to(R.rotate(q, pos, freq, scale, interleaved), "f32")
    dq, outs = to_dev(q, "f32"), []
    outs.append(torch.zeros_like(dq))
    kv.lora_rope(dq, outs[0], to_dev(k, "f32") if hk else None, to_dev(k, "f32") if hk else None, i32(pos), rope)
    data = torch.zeros((T, R.block_bytes(16, k.shape[1], D)), dtype=torch.uint8, device=DEV)
    outs.append(torch.zeros_like(dq))
    kv.lora_kv_append(dq, outs[1], to_dev(k, "f32"), to_dev(v, "f32"), i32(pos), i32(np.arange(T) * 16), rope, kv.Cache(data, 16, k.shape[1], D))
    torch.cuda.synchronize()
    for got in outs:
        # the same but for values next to a border: the plain form's angles are off by up to 2^-53 * 2^16 radians
        # (a turn rounded to 53 bits), 2^-13 of half a step
        got = host(got)
        assert np.all(np.abs(got - want) <= 2 * 2.0 ** -24 * np.abs(want)) and np.mean(got != want) < 1e-3


# ------------------------------------------------- head dims, tiles and splits
class Big:
    """A step over a cache of random bytes; the plain result in 64 bits on the GPU from the gathered values."""

    def __init__(self, seed, ctx, new, hq, hkv, D, bt, dtype="bf16", pad=0):
        rng = np.random.default_rng(seed)
        self.ctx, self.new, self.hq, self.hkv, self.D = np.array(ctx), np.array(new), hq, hkv, D
        table, free, num = make_table(rng, ctx, new, bt)
        self.T = int(np.sum(new)) + pad
        nc = D // 32
        data = rng.integers(0, 256, (num, hkv * bt // 16, 544 * nc)).astype(np.uint8)
        data[..., 512 * nc:] = 125 + data[..., 512 * nc:] % 3
        self.cache = kv.Cache(torch.tensor(data.reshape(num, -1), device=DEV), bt, hkv, D)
        self.batch = kv.Batch(self.T, len(ctx), hq, hkv, D)
        self.table = i32(table)
        self.q = to_dev(rng.standard_normal((self.T, hq, D)), dtype)
        self.ws = kv.attend_workspace(self.batch)
        kv.lora_kv_build(i32(ctx), i32(new), self.T, self.table, i32(free), num, bt, self.batch)
        self.bt, self.dtype = bt, dtype

    def check(self, q, out, scale):
        kv.lora_kv_attend(q, out, self.batch, self.table, self.cache, scale, self.ws)
        torch.cuda.synchronize()
        assert int(self.batch.flags) == 0
        begin, G = 0, self.hq // self.hkv
        for i, (c, n) in enumerate(zip(self.ctx.tolist(), self.new.tolist())):
            L = c + n
            p = torch.arange(L, device=DEV)
            slots = (self.table[i].long()[p // self.bt] * self.bt + p % self.bt).int()
            k = torch.zeros((L, self.hkv, self.D), dtype=torch.float32, device=DEV)
            v = torch.zeros_like(k)
            kv.lora_kv_gather(self.cache, slots, k, v)
            hide = p[None, :] > torch.arange(c, L, device=DEV)[:, None]
            for h in range(self.hkv):
                qq = self.q[begin:begin + n, h * G:(h + 1) * G].double().transpose(0, 1).contiguous()
                kk, vv = k[:, h].double(), v[:, h].double()
                x = (qq @ kk.T.contiguous() * scale).masked_fill(hide, -math.inf)
                w = torch.softmax(x, -1)
                o, a = w @ vv, w @ vv.abs()
                s_abs = (qq.abs() @ kk.abs().T.contiguous() * scale).masked_fill(hide, 0.0).amax(-1, keepdim=True)
                o, a, s_abs = (y.cpu().numpy() for y in (o, a, s_abs))
                got = host(out[begin:begin + n, h * G:(h + 1) * G].transpose(0, 1))
                bound = R.attend_bound(o, a, s_abs, L, self.D, self.dtype)
                if self.dtype == "bf16":  # the sum is of rounded weights too
                    bound = bound + 2.0 ** -8 * np.abs(o)
                assert np.all(np.abs(got - o) <= bound), (i, h)
            begin += n
        return begin


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("D,hq,hkv,bt", [(128, 8, 2, 16), (128, 2, 2, 256), (160, 4, 2, 32), (192, 3, 1, 16), (224, 2, 1, 64), (256, 4, 2, 128)])
def test_requests_of_many_rows_at_every_wide_head_dim(D, hq, hkv, bt, split, dtype):
    ctx, new = ([2300, 0, 77], [131, 66, 1]) if split else ([150, 0, 77], [131, 66, 1])
    s = Big(D + split, ctx, new, hq, hkv, D, bt, dtype, pad=3)
    assert int(s.batch.counts[kv.COUNT_WIDE]) > 0 and (int(s.batch.counts[kv.COUNT_PARTS]) > 0) == split
    out = torch.full_like(s.q, 5.0)
    end = s.check(s.q, out, D ** -0.5)
    assert bool((out[end:] == 5.0).all())


@pytest.mark.parametrize("D,hq,hkv", [(64, 4, 2), (128, 8, 1), (256, 2, 1)])
def test_requests_of_many_rows_with_strided_queries_and_outputs(D, hq, hkv):
    s = Big(D, [1300, 20], [100, 70], hq, hkv, D, 16)
    assert int(s.batch.counts[kv.COUNT_WIDE]) > 0
    fused = torch.full((s.T, hq + 3, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    fused[:, 1:1 + hq] = s.q
    out = torch.full((s.T, hq + 2, D), 5.0, dtype=torch.bfloat16, device=DEV)
    s.check(fused[:, 1:1 + hq], out[:, :hq], D ** -0.5)
    assert bool((out[:, hq:] == 5.0).all())
    first = torch.zeros((hq, s.T, D), dtype=torch.bfloat16, device=DEV).transpose(0, 1)  # heads first
    s.check(s.q, first, D ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ctx,hq,hkv,D", [([5000, 3, 0], 32, 1, 64), ([4100, 900], 40, 1, 128), ([3000], 34, 2, 96), ([2100, 17], 17, 1, 256)])
def test_decode_steps_with_more_query_heads_than_a_tile(ctx, hq, hkv, D, dtype):
    s = Big(hq + D, ctx, [1] * len(ctx), hq, hkv, D, 16, dtype)
    c = s.batch.counts
    assert int(c[kv.COUNT_PARTS]) > 1 and int(c[kv.COUNT_MID]) + int(c[kv.COUNT_WIDE]) == 0
    s.check(s.q, torch.zeros_like(s.q), D ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_long_chunk_among_idle_requests(dtype):
    """As many requests as tokens: the step is planned as a decode step, in items of 16 rows."""
    new = [0] * 100 + [60, 1]
    s = Big(3, [20] * 100 + [1500, 40], new, 4, 2, 64, 16, dtype)
    assert s.T <= len(new) and int(s.batch.counts[kv.COUNT_WIDE]) == 0
    s.check(s.q, torch.zeros_like(s.q), 0.125)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_requests_without_room_for_partial_results_are_not_split(dtype):
    hkv = 32
    s = Big(4, [947, 1035] * 14 + [1035], [128, 40] * 14 + [40], hkv, hkv, 64, 16, dtype)
    room = 8 * (1024 // hkv + 1)
    assert int(s.batch.counts[kv.COUNT_PARTS]) > room
    s.check(s.q, torch.zeros_like(s.q), 0.125)
