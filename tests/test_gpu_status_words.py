"""The status word of a reused workspace after a call without rows or tokens."""
import pytest
import torch

from routing_dispatch_grouped_gb300 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
BOUNDS = 5


def _norm_backward(ws, d):
    x, s = torch.empty(0, d, dtype=bf16, device=DEV), torch.empty(0, device=DEV)
    moe.moe_norm_backward(x, x, None, s, s, workspace=ws)


def _embed(ws, d):
    moe.moe_embed(torch.empty(0, dtype=i32, device=DEV), torch.ones(5, d, dtype=bf16, device=DEV),
                  workspace=ws)


def _embed_backward(ws, d):
    moe.moe_embed_backward(torch.empty(0, d, dtype=bf16, device=DEV),
                           torch.empty(0, dtype=i32, device=DEV), 5, workspace=ws)


@pytest.mark.parametrize("capture", [False, True])
@pytest.mark.parametrize("call", [_norm_backward, _embed, _embed_backward])
def test_an_empty_call_clears_the_word(call, capture):
    d = 64
    ws = torch.full((moe.moe_embed_backward_workspace_size(8, d),), 77, dtype=torch.uint8,
                    device=DEV)
    graph = torch.cuda.CUDAGraph()
    if capture:
        with torch.cuda.graph(graph):
            call(ws, d)
    run = graph.replay if capture else lambda: call(ws, d)
    run()
    assert moe.moe_read_device_status(ws) == 0
    # an earlier call's error is not reported again
    bad = torch.tensor([0, 9, 1], dtype=i32, device=DEV)
    moe.moe_embed(bad, torch.ones(5, d, dtype=bf16, device=DEV), workspace=ws)
    assert moe.moe_read_device_status(ws) == BOUNDS
    run()
    assert moe.moe_read_device_status(ws) == 0
