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
