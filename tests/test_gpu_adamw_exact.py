"""moe_adamw with fp32 moments: the parameters bit for bit, as the moments."""
import numpy as np
import pytest
import torch

from routing_dispatch_grouped_gb300 import synth
from tests.test_gpu_adamw import DEV, SIZES, _fp32_step, _step, _tensor

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("pd,gd,copy", [(f32, f32, False), (f32, bf16, True), (bf16, bf16, False),
                                        (bf16, f32, False)])
@pytest.mark.parametrize("n", SIZES)
def test_every_step_of_the_formula_is_rounded_by_itself(n, pd, gd, copy):
    t = _tensor(n, pd, gd, 32, copy)
    # magnitudes over many binades, so that a fused or approximate step shows somewhere
    t["m"].mul_(torch.exp(4 * synth.normal((n,), f32, 0, "spread", 1.0, device=DEV)))
    for step in (1, 7):
        p, _, m, v = _fp32_step(t, step, 0.1, 0.75)
        _step([t], step, grad_scale=torch.full((1,), 0.75, device=DEV))
        assert np.array_equal(t["m"].cpu().numpy(), m) and np.array_equal(t["v"].cpu().numpy(), v)
        ref = torch.from_numpy(p).to(pd)
        assert torch.equal(t["p"].cpu(), ref)
        if copy:
            assert torch.equal(t["c"].cpu(), ref.to(bf16))
