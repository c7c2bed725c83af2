"""The stored numbers of 8-bit moments in a block that holds something not finite."""
import pytest
import torch

from tests.test_gpu_adamw import _step, _tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_numbers_and_scales_of_such_a_block_are_nan(bad):
    t = _tensor(2000, bits=8)
    t["g"][700] = bad                                       # block 2
    _step([t], 5)
    for numbers, scales in ((t["m"], t["ms"]), (t["v"], t["vs"])):
        x = numbers.float()
        assert x[512:768].isnan().all() and scales[2].isnan()
        assert x[:512].isfinite().all() and x[768:].isfinite().all()
        assert scales[:2].isfinite().all() and scales[3:].isfinite().all()
