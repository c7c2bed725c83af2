"""moe_embed_backward past the longest chunks: a run of equal ids over more than a thousand of them."""
import pytest
import torch

from routing_dispatch_grouped_gb300 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T", [524288, 524289, 1100003])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_one_id_and_two_ids_over_all_tokens(T, grad):
    """Whole numbers whose sums fp32 holds: every order gives the same."""
    V, d = 5, 72
    dout = ((torch.arange(T * d, device=DEV) % 7) - 3).view(T, d).to(torch.bfloat16)
    for ids in (torch.full((T,), 3, device=DEV), torch.arange(T, device=DEV) % 2 * 3):
        got = moe.moe_embed_backward(dout, ids, V, grad_dtype=grad)
        ref = torch.zeros(V, d, dtype=torch.float64, device=DEV)
        for v in (0, 3):
            ref[v] = dout[ids == v].double().sum(0)
        assert torch.equal(got, ref.float().to(grad))
