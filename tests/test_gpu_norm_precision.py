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
