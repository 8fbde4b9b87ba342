"""Selection from logits of any finite size: vocabularies masked with large
negative numbers, rows far from zero, against the plain 64-bit form.

The tolerance is that of Select.check: weights are e^(x - r) with x - r formed
to 2^-24 of itself whatever the size of x and r, so the count of roundings
there holds for every finite logit."""
import numpy as np
import pytest
import torch

from test_gpu_beam import Select

pytestmark = pytest.mark.gpu
MASKS = [-1e4, -7e4, -1e6, -1e7, -1e9, -1e10, -1e12, -1e20, -1e30, -1e37]
SCORES = [-1.0, -1.1, -1.2, -1.3]


def masked(mask, V=6001, W=4):
    """Three requests: parts of rows masked, and a whole one; a few tokens left in every row; nothing left."""
    rng = np.random.default_rng(7)
    x = rng.standard_normal((3 * W, V)).astype(np.float32) * 2.5
    x[0, :2500] = mask  # whole chunks before the others
    x[1] = mask
    x[2, np.arange(V) % 97 != 5] = mask
    x[3, 300:] = mask
    for w in range(W):
        left = rng.choice(V, 6, replace=False)
        keep = x[W + w, left]
        x[W + w] = mask
        x[W + w, left] = keep
    x[2 * W:] = mask
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mask", MASKS)
def test_masks_of_any_size(mask, dtype):
    s = Select(masked(mask), 4, np.tile(SCORES, 3), np.arange(12), np.zeros(12), -1, 0.0, dtype)
    got = s.run()
    assert np.all(np.isfinite(got[2])) and int(s.flags) == 0
    s.check(got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mask", MASKS)
def test_masks_where_a_wave_takes_a_whole_row(mask, dtype):
    """4200 rows: each wave goes from masked chunks to others and back."""
    n, rows = 350, 12
    x = masked(mask)
    one = Select(x, 4, np.tile(SCORES, 3), np.arange(rows), np.zeros(rows), -1, 0.0, dtype)
    s = Select(np.tile(x, (n, 1)), 4, np.tile(SCORES, 3 * n), np.tile(np.arange(rows), n), np.zeros(rows * n), -1, 0.0, dtype)
    got = [g.reshape(n, rows) for g in s.run()]
    assert int(s.flags) == 0
    got[0] = got[0] - np.arange(n)[:, None] * rows
    for i in (0, 1, n // 2, n - 1):
        one.check([g[i] for g in got])
    for g in (got[0], got[1], got[3], got[4]):
        assert np.all(g == g[0])
    # the same sums, cut at other places
    assert np.all(np.abs(got[2] - got[2][0]) <= 2 * (64 * 2.0 ** -24 + 2.0 ** -24 * np.abs(got[2][0])))


@pytest.mark.parametrize("W", [1, 3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e4, 1e5, 1e6, 1e7, 3e7, 1e9, 1e12, 1e20, 1e30, 1e37])
def test_rows_of_any_size(size, dtype, W):
    """Neighbouring numbers of the type around +-size, next to an ordinary row."""
    rng = np.random.default_rng(3)
    V = 5000
    step = torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).eps
    x = np.stack([size * (1 + step * rng.integers(0, 20, V)), -size * (1 + step * rng.integers(0, 20, V)), rng.standard_normal(V) * 2.5])
    s = Select(x, W, [-1.0, -1.37, -1.9], [1, 2, 3], [0, 0, 0], -1, 0.0, dtype)
    got = s.run()
    assert np.all(np.isfinite(got[2])) and int(s.flags) == 0
    s.check(got)


@pytest.mark.parametrize("W", [1, 4])
@pytest.mark.parametrize("centre", [32768.0, 65520.0, 65536.0, 65552.0, 131072.0, 1e6])
def test_spread_rows_far_from_zero(centre, W):
    """fp32 rows around a far centre that keep some of their spread."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 7000)) * 2.5 + centre * np.array([[1.0], [-1.0], [1.0], [-1.0]])
    x[2, 100] = 5.0
    x[3, 6000] = 5.0
    s = Select(x, W, SCORES, [1, 2, 3, 4], [0] * 4, -1, 0.0, "f32")
    s.check(s.run())
    assert int(s.flags) == 0
