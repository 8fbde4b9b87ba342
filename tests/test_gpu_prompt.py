"""Prompt attention on the GPU against its plain 64-bit form."""
import math

import numpy as np
import pytest
import torch

import kv_reference as R
from heterogeneous_adapters_amd import kv
from test_gpu_kv import DEV, host, i32, normal, to_dev

pytestmark = pytest.mark.gpu


def run_prompt(q, k, v, indptr, scale, dtype):
    dq, dk, dv = (to_dev(x, dtype) for x in (q, k, v))
    out = torch.full_like(dq, 5.0)
    kv.lora_prompt_attend(dq, dk, dv, out, i32(indptr), scale)
    torch.cuda.synchronize()
    return host(out)


def check_prompt(got, q, k, v, indptr, scale, dtype):
    D, inside = q.shape[2], np.zeros(q.shape[0], bool)
    for a, b in zip(indptr, indptr[1:]):
        inside[a:b] = True
        n = b - a
        o, w, s_abs = R.attend_rows(q[a:b], k[a:b], v[a:b], np.arange(1, n + 1), scale)
        bound = R.attend_bound(o, w, s_abs, n, D, dtype)
        err = np.abs(got[a:b] - o)
        assert np.all(err <= bound), (a, b, float((err / bound).max()))
    assert np.all(got[~inside] == 5.0)


PROMPTS = [
    ([1], 1, 1, 32), ([2, 1, 3], 2, 1, 64), ([31, 32, 33], 4, 2, 128), ([63, 64, 65, 0, 1], 2, 2, 96), ([127, 128, 129], 3, 1, 64),
    ([200], 6, 2, 128), ([257, 5], 4, 4, 160), ([130, 70], 5, 1, 192), ([100, 300], 2, 1, 224), ([190], 2, 2, 256),
    ([1] * 300, 1, 1, 32), ([400], 16, 2, 32),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_prompt_against_plain(case, dtype):
    lens, hq, hkv, D = PROMPTS[case]
    rng = np.random.default_rng(case)
    gap = case % 3  # rows before the first and behind the last prompt
    indptr = gap + np.concatenate([[0], np.cumsum(lens)])
    T = int(indptr[-1]) + gap
    q, k, v = normal(rng, (T, hq, D), dtype), normal(rng, (T, hkv, D), dtype), normal(rng, (T, hkv, D), dtype)
    scale = 1.0 / math.sqrt(D)
    check_prompt(run_prompt(q, k, v, indptr, scale, dtype), q, k, v, indptr, scale, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_peaked_scores(dtype):
    rng = np.random.default_rng(1)
    T = 210
    q, v = normal(rng, (T, 2, 64), dtype), normal(rng, (T, 1, 64), dtype)
    k = R.round_to(normal(rng, (T, 1, 64), dtype) * np.linspace(0.1, 8.0, T)[:, None, None], dtype)
    check_prompt(run_prompt(q, k, v, [0, T], 0.9, dtype), q, k, v, [0, T], 0.9, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 96])
def test_prompt_values_that_are_not_finite_stay_with_the_rows_that_see_them(dtype, D):
    """NaN and infinities in V (and NaN in K) behind a row's last key, of its own prompt or the next one, change nothing."""
    rng = np.random.default_rng(D)
    lens = [150, 77]
    indptr = np.concatenate([[0], np.cumsum(lens)])
    T = int(indptr[-1])
    q, k, v = normal(rng, (T, 2, D), dtype), normal(rng, (T, 1, D), dtype), normal(rng, (T, 1, D), dtype)
    v[70, 0, 3], v[75, 0, 5], v[90, 0, 5], v[100, 0, 7] = np.nan, np.inf, -np.inf, np.inf
    v[150, 0, :] = np.nan  # the second prompt's first token: all of its rows
    k[120] = np.nan  # rows from 120 on of the first prompt are NaN
    scale = 1.0 / math.sqrt(D)
    got = run_prompt(q, k, v, indptr, scale, dtype)
    clean_v, clean_k = np.where(np.isfinite(v), v, 0.0), np.where(np.isfinite(k), k, 0.0)
    o, w, s_abs = R.attend_rows(q[:150], clean_k[:150], clean_v[:150], np.arange(1, 151), scale)
    bound = R.attend_bound(o, w, s_abs, 150, D, dtype)
    want = o.copy()
    want[70:, :, 3] = np.nan
    want[75:, :, 5] = np.inf
    want[90:, :, 5] = np.nan
    want[100:, :, 7] = np.inf
    want[120:] = np.nan
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got[:150]), np.isnan(want)) and np.array_equal(np.isposinf(got[:150]), np.isposinf(want))
    assert np.all(np.abs(got[:150] - want)[fine] <= bound[fine])
    assert np.isnan(got[150:]).all()
