"""moe_norm and moe_norm_backward on rows whose mean, size or entries are out of the ordinary."""
import numpy as np
import pytest
import torch

from oracle import train_step as S
from routing_dispatch_grouped_gb300 import moe, synth
from tests.helpers import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
bf16, f32 = torch.bfloat16, torch.float32
U = 2.0 ** -24                                     # fp32 unit roundoff
OUT = {bf16: 2.0 ** -8, f32: 2.0 ** -24}           # of the stored type
# a warp a row, a block a row, more than 512 threads
SHAPES = [(96, bf16), (2880, bf16), (16384, bf16), (96, f32), (2880, f32), (8192, f32)]


def _normal(shape, dtype, name, sigma=1.0):
    return synth.normal(shape, dtype, 0, name, sigma, device=DEV)


@pytest.mark.parametrize("offset", [0.0, 3.0, 100.0, 3000.0])
@pytest.mark.parametrize("d,dtype", SHAPES)
def test_gradient_of_rows_with_a_large_mean(d, dtype, offset):
    """For given statistics xh = (x - mean) rstd has two roundings, whatever the mean's size."""
    x = (_normal((5, d), f32, "x") + offset).to(dtype)
    dy, w = _normal((5, d), dtype, "dy", 0.1), _normal((d,), f32, "w", 0.3) + 1
    _, _, mean, rstd = moe.moe_norm(x, w)
    dx, _, _ = moe.moe_norm_backward(dy, x, w, mean, rstd)
    x64, dy64, w64, mu, q = f64(x), f64(dy), f64(w), f64(mean)[:, None], f64(rstd)[:, None]
    xh = np.abs((x64 - mu) * q)
    for t in range(5):
        # one row: its product with dy rounds once more, and nothing is added to it
        row = [a[t:t + 1].clone() for a in (dy, x, mean, rstd)]
        dw = moe.moe_norm_backward(row[0], row[1], w, row[2], row[3])[1]
        ref = (dy64 * (x64 - mu) * q)[t]
        assert np.all(np.abs(f64(dw) - ref) <= 3.01 * U * np.abs(ref))
    rx = S.norm_backward(dy64, x64, w64, mu[:, 0], q[:, 0])[0]
    # a mean over a row is a tree of at most 40 additions and a few products
    u = np.abs(dy64 * w64)
    c1, c2 = u.mean(1, keepdims=True), (u * xh).mean(1, keepdims=True)
    err = q * (4 * U * u + xh * 46 * U * c2 + 6 * U * xh * c2 + 48 * U * c1)
    assert np.all(np.abs(f64(dx) - rx) <= OUT[dtype] * np.abs(rx) + err)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_a_row_of_equal_values_is_its_own_mean(dtype):
    """Whatever the width: the sum of a row of one such value is exact, and so is its quotient."""
    values = torch.tensor([1000.0, -100.5, 7.25, 0.1875], device=DEV, dtype=dtype)
    for d in [*range(8, 2048, 8), 5000, 7000, 8192]:
        x = values[:, None].expand(-1, d).contiguous()
        y, _, mean, _ = moe.moe_norm(x)
        assert torch.equal(mean, values.float()) and not y.any(), d


def _bound(s, w, b, mu, q, y, dtype, rms):
    """A row's sums are trees of at most 40 additions, so its mean is off by 40 U mean|s|, rstd by
    half of that relatively, the squares' error and its own roundings."""
    dmu = np.zeros(s.shape[0]) if rms else 42 * U * np.abs(s).mean(1) + U * np.abs(mu)
    xw = np.abs(s - mu[:, None]) * q[:, None] * np.abs(w)
    dq = 50 * U + (dmu * q) ** 2
    return (OUT[dtype] * np.abs(y) + (dq[:, None] + 4 * U) * xw + 2 * U * np.abs(b) +
            (q * dmu)[:, None] * np.abs(w) +
            2 * U * q[:, None] * np.abs(w) * (np.abs(s) + np.abs(mu)[:, None]))


def _check_rows(x, residual, w, b, eps, rms, rows):
    """`rows` of moe_norm against the definition."""
    y, total, mean, rstd = moe.moe_norm(x, w, None if rms else b, eps, rms=rms, residual=residual)
    s = f64(x if residual is None else total)[rows]
    w64, b64 = f64(w), np.zeros(x.shape[1]) if rms else f64(b)
    ref, mu, q = S.norm(s, w64, b64, eps, rms)
    assert np.all(np.abs(f64(y)[rows] - ref) <= _bound(s, w64, b64, mu, q, ref, x.dtype, rms))
    # rstd is a fp32 number, which may be a subnormal one
    dmu = 0 if rms else 42 * U * np.abs(s).mean(1) + U * np.abs(mu)
    assert np.all(np.abs(f64(rstd)[rows] - q) <= q * (52 * U + (dmu * q) ** 2) + 2.0 ** -149)
    if not rms:
        assert np.all(np.abs(f64(mean)[rows] - mu) <= dmu)
    return y, mean, rstd


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("d,dtype", SHAPES + [(1000, bf16), (1000, f32)])
def test_rows_beyond_the_squares_range(d, dtype, residual, rms):
    """Infinities and NaN make their whole row NaN, in both forms; finite rows stay right however
    large; the rows beside them are untouched."""
    w, b = _normal((d,), f32, "w", 0.3) + 1, _normal((d,), f32, "b", 0.3)
    x = _normal((12, d), f32, "x")
    x[1, d // 2], x[2, 0], x[3, d - 1] = float("inf"), -float("inf"), float("nan")
    x[4] *= 1e19                                       # squares above the range, one by one
    x[5] = x[5] * 1e36 + 3e37
    x[6] = 3.3e38 * (1 - (torch.arange(d, device=DEV) % 7) / 64)     # so is the sum
    x[7] = 3.3e38 * torch.sign(x[7])                   # and the distance from the mean
    x[8, 3] = 1e30                                     # one large entry
    x[9] *= 2e-10
    x = x.to(dtype)
    r = None
    if residual:                                       # x / 2 + x / 2: the same rows
        x = x / 2
        r = x.clone()
    y, mean, rstd = _check_rows(x, r, w, b, 1e-5, rms, [0, 4, 5, 6, 7, 8, 9, 10, 11])
    assert y[1:4].isnan().all() and rstd[1:4].isnan().all()
    assert rms or not mean[1:4].isfinite().any()


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("d,dtype", SHAPES)
def test_small_rows_without_an_epsilon(d, dtype, rms):
    w, b = _normal((d,), f32, "w", 0.3) + 1, _normal((d,), f32, "b", 0.3)
    sizes = torch.tensor([1.0, 1e-14, 1e-16, 1e-20, 1e-25, 1e-32], device=DEV)
    x = (_normal((6, d), f32, "x") * sizes[:, None]).to(dtype)
    _check_rows(x, None, w, b, 0.0, rms, list(range(6)))
    _check_rows(x, None, w, b, 1e-38, rms, list(range(6)))
