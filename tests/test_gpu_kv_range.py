"""The attention operators over the rest of their range: weights that sum to one."""
import math

import numpy as np
import pytest

import kv_reference as R
from test_gpu_kv import Step
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
