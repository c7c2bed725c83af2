"""Calls on another stream than the current one, with a workspace that the call allocates itself."""
import pytest
import torch

from routing_dispatch_grouped_gb300 import moe, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
bf16, f32 = torch.bfloat16, torch.float32


class Recorder:
    """The library, with the pointers of every call kept."""

    def __init__(self, real):
        self.real, self.pointers = real, set()

    def __getattr__(self, name):
        fn = getattr(self.real, name)
        if name.endswith("_size"):
            return fn

        def call(*args):
            for a in args:
                self.pointers.add(getattr(a, "value", a))
            return fn(*args)
        return call


def _like(ts):
    return [torch.empty_like(t) for t in ts]


def _norm_backward():
    T, d = 3000, 1024
    x, dy = (synth.normal((T, d), bf16, 0, n, 1.0, device=DEV) for n in ("x", "dy"))
    _, _, mean, rstd = moe.moe_norm(x)
    size = moe.moe_norm_backward_workspace_size(T, d, bf16)

    def call(out=(None, None, None), **kw):
        return moe.moe_norm_backward(dy, x, None, mean, rstd, dx=out[0], dweight=out[1],
                                     dbias=out[2], **kw)
    return size, call


def _embed_backward():
    T, V, d = 3000, 500, 256
    dout = synth.normal((T, d), bf16, 0, "dout", 1.0, device=DEV)
    ids = (torch.arange(T, device=DEV) * 7919) % V
    size = moe.moe_embed_backward_workspace_size(T, d)
    return size, lambda out=(None,), **kw: (moe.moe_embed_backward(dout, ids, V, d_table=out[0],
                                                                   **kw),)


@pytest.mark.parametrize("make", [_norm_backward, _embed_backward])
def test_the_workspace_is_not_handed_out_while_the_stream_is_busy(make, monkeypatch):
    size, call = make()
    ref = call()
    a = torch.randn(4096, 4096, device=DEV)
    b = a @ a
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    stream = torch.cuda.Stream()
    recorder = Recorder(moe.lib())
    monkeypatch.setattr(moe, "lib", lambda: recorder)
    with torch.cuda.stream(stream):
        for _ in range(40):                     # some tens of milliseconds before the call's turn
            torch.mm(a, a, out=b)
        done = torch.cuda.Event()
    got = call(stream=stream)
    done.record(stream)
    # what the current stream allocates meanwhile, and writes at once
    blocks = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
    busy = not done.query()
    torch.cuda.synchronize()
    assert busy, "the stream was done before the blocks were allocated: nothing was tested"
    assert not any(t.data_ptr() in recorder.pointers for t in blocks)
    assert all(torch.equal(p, q) for p, q in zip(got, ref) if p is not None)


@pytest.mark.parametrize("make", [_norm_backward, _embed_backward])
def test_the_workspace_is_no_block_that_the_current_stream_still_writes(make, monkeypatch):
    size, call = make()
    ref = call()
    out = _like(ref)
    a = torch.randn(4096, 4096, device=DEV)
    b = a @ a
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    stream = torch.cuda.Stream()
    recorder = Recorder(moe.lib())
    monkeypatch.setattr(moe, "lib", lambda: recorder)
    block = torch.empty(size, dtype=torch.uint8, device=DEV)
    address = block.data_ptr()
    for _ in range(40):
        torch.mm(a, a, out=b)
    block.fill_(255)
    late = torch.cuda.Event()
    late.record()
    del block                                   # free for the current stream's next allocation
    call(out=out, stream=stream)                # which this is not
    busy = not late.query()
    torch.cuda.synchronize()
    assert busy, "the current stream was done before the call: nothing was tested"
    assert address not in recorder.pointers
    assert all(torch.equal(p, q) for p, q in zip(out, ref))
