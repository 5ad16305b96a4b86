"""LayerNorm of rows whose values are nearly equal and far from zero, where what m0's rounding leaves is as large as the
deviation itself, or larger; and of the largest eps.  Tolerances as in test_gpu_mx_layernorm."""
import numpy as np
import pytest

import mx_block_scaled_x128_amd as mx
from test_gpu_mx_layernorm import T, U, check_codes, close, given, normalised, tensor, xh_error

pytestmark = pytest.mark.gpu


def nearly_equal(rows, cols, seed, top=2 ** 24):
    """fp32 rows of one value each, 1 to 5 elements of which are one or two steps higher."""
    rng = np.random.default_rng(seed)
    x = np.repeat(rng.uniform(1e3, top, rows).astype(np.float32)[:, None], cols, axis=1)
    x[0], x[1] = np.float32(7377776.5), np.float32(15792095)
    for row in x:
        up = rng.choice(cols, rng.integers(1, 6), replace=False)
        row[up] = np.nextafter(row[up], np.float32(np.inf))
        row[up[:len(up) // 3]] = np.nextafter(row[up[:len(up) // 3]], np.float32(np.inf))
    return x


@pytest.mark.parametrize("eps", [0.0, 1e-5, 1e-3])
# one, two and four units a lane; 600 rows of 3584 are taken two at a time
@pytest.mark.parametrize("rows,cols", [(40, 64), (40, 3584), (600, 3584), (40, 7168), (40, 9216), (24, 20480)])
def test_equal_but_for_a_few_steps(rows, cols, eps):
    x = nearly_equal(rows, cols, rows + cols)
    xh, r = normalised(x.astype(np.float64), eps)
    y, ys, kept = mx.layernorm_mx(tensor(x, "f32"), None, None, eps)
    close(kept.rstd, r, (T / 2 + 4) * U * r)
    check_codes(y, ys, xh, xh_error(xh), mx.E4M3, mx.RULE_CEIL)


@pytest.mark.parametrize("rows,cols", [(16, 3584), (1100, 3584), (16, 9216)])
def test_equal_but_for_a_few_steps_of_bf16(rows, cols):
    rng = np.random.default_rng(cols)
    x = np.repeat(rng.integers(128, 255, rows)[:, None] * 2.0 ** rng.integers(-3, 9, rows)[:, None], cols, axis=1)
    for row in x:
        row[rng.choice(cols, 3, replace=False)] *= 1 + 2.0 ** -7
    x = tensor(x.astype(np.float32), "bf16")
    x64 = x.double().cpu().numpy()
    for eps in (0.0, 1e-5):
        xh, r = normalised(x64, eps)
        y, ys, kept = mx.layernorm_mx(x, None, None, eps)
        close(kept.rstd, r, (T / 2 + 4) * U * r)
        check_codes(y, ys, xh, xh_error(xh), mx.E4M3, mx.RULE_CEIL)


@pytest.mark.parametrize("rows,cols", [(5, 64), (1100, 3584), (5, 9216)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_largest_eps(rows, cols, dtype):
    """eps = 3.4e38, the largest that is taken: the variance of some rows takes the sum past fp32's range."""
    x = given((rows, cols), 2.0 ** np.array([0, 40, 58, 59, 60] * rows)[:rows, None], 7, dtype)
    xh, r = normalised(x.astype(np.float64), float(np.float32(3.4e38)))
    y, ys, kept = mx.layernorm_mx(tensor(x, dtype), None, None, 3.4e38)
    close(kept.rstd, r, (T / 2 + 4) * U * r)
    check_codes(y, ys, xh, xh_error(xh), mx.E4M3, mx.RULE_CEIL)
