"""What the binding does around a call of the C ABI, without a GPU: stand-ins for CUDA tensors and
for the library record what a call is given."""
import pytest
import torch

from routing_dispatch_grouped_gb300 import moe

bf16, f32 = torch.bfloat16, torch.float32


class Stream:
    cuda_stream = 0x5157


class Current:
    """torch.cuda.stream as far as it goes without a GPU: which stream is current."""
    stack = [None]

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        Current.stack.append(self.stream)

    def __exit__(self, *exc):
        Current.stack.pop()


class Cuda:
    """As much of a contiguous CUDA tensor as the binding looks at."""
    made = 0

    def __init__(self, shape, dtype, index=0):
        Cuda.made += 1
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device = torch.device("cuda", index)
        self.is_cuda, self.address, self.owner = True, 0x100000 * Cuda.made, Current.stack[-1]

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return self.address

    def get_device(self):
        return self.index


class Library:
    """Every call succeeds; the workspaces' sizes are what the real library says."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return getattr(moe._lib, name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    moe.lib()
    fake = Library()
    monkeypatch.setattr(moe, "lib", lambda: fake)
    return fake


@pytest.fixture
def allocated(monkeypatch):
    """The tensors that torch.empty gave out."""
    got = []

    def empty(*shape, dtype=f32, device=None):
        got.append(Cuda(shape[0] if isinstance(shape[0], tuple) else shape, dtype))
        return got[-1]
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", Current)
    return got


@pytest.fixture(autouse=True)
def device_0(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)


def _norm_backward(**kw):
    T, d = 6, 64
    x = Cuda((T, d), bf16)
    return moe.moe_norm_backward(Cuda((T, d), bf16), x, None, Cuda((T,), f32), Cuda((T,), f32),
                                 dx=Cuda((T, d), bf16), dweight=Cuda((d,), f32),
                                 dbias=Cuda((d,), f32), **kw)


def _embed_backward(**kw):
    T, V, d = 6, 10, 64
    return moe.moe_embed_backward(Cuda((T, d), bf16), Cuda((T,), torch.int32), V,
                                  d_table=Cuda((V, d), f32), **kw)


R, d, E, I = 6, 64, 4, 32
GU, DOWN, OFFSETS = Cuda((E, d, 2 * I), bf16), Cuda((E, I, d), bf16), Cuda((E + 1,), torch.int32)
STEPS = {
    "gate_up": lambda **kw: moe.moe_gate_up(Cuda((R, d), bf16), OFFSETS, GU, h=Cuda((R, I), bf16),
                                            **kw),
    "down": lambda **kw: moe.moe_down(Cuda((R, I), bf16), OFFSETS, DOWN,
                                      y_sorted=Cuda((R, d), f32), **kw),
    "experts": lambda **kw: moe.moe_experts(Cuda((R, d), bf16), OFFSETS, GU, DOWN,
                                            h=Cuda((R, I), bf16), y_sorted=Cuda((R, d), f32),
                                            **kw),
    "gate_up_train": lambda **kw: moe.moe_gate_up_train(
        Cuda((R, d), bf16), OFFSETS, GU, h=Cuda((R, I), bf16), ab=Cuda((R, 2 * I), bf16), **kw),
    "down_backward": lambda **kw: moe.moe_down_backward(
        Cuda((R, d), bf16), Cuda((R, 2 * I), bf16), OFFSETS, DOWN, d_ab=Cuda((R, 2 * I), bf16),
        **kw),
    "gate_up_backward": lambda **kw: moe.moe_gate_up_backward(
        Cuda((R, 2 * I), bf16), OFFSETS, GU, dx_sorted=Cuda((R, d), f32), **kw),
    "weight_grad": lambda **kw: moe.moe_weight_grad(
        Cuda((R, d), bf16), Cuda((R, I), bf16), OFFSETS, E, dw=Cuda((E, d, I), f32), **kw),
    # those return their workspace, which a caller may drop at once
    "dispatch": lambda **kw: moe.moe_dispatch(Cuda((R, 2), torch.int32), E, **kw),
    "forward": lambda **kw: moe.moe_forward(Cuda((R, d), bf16), Cuda((R, E), f32), GU, DOWN, 2,
                                            **kw),
    "forward_train": lambda **kw: moe.moe_forward_train(Cuda((R, d), bf16), Cuda((R, E), f32), GU,
                                                        DOWN, 2, **kw),
    "backward": lambda **kw: moe.moe_backward(
        Cuda((R, d), bf16), Cuda((R, d), bf16), Cuda((R, E), f32), GU, DOWN, 2,
        Cuda((R, 2), torch.int32), Cuda((R, 2), f32), Cuda((1 << 20,), torch.uint8), **kw),
}


@pytest.mark.parametrize("call", [_norm_backward, _embed_backward, *STEPS.values()],
                         ids=["norm_backward", "embed_backward", *STEPS])
def test_a_workspace_of_the_call_belongs_to_the_stream_it_was_given(library, allocated, call):
    """Nothing need hold such a workspace after the call has returned, and nothing orders the given
    stream behind the current one: the block has to come from the given stream's own memory, which
    is reused in that stream's order alone."""
    stream = Stream()
    call(stream=stream)
    ws, = [t for t in allocated if t.dtype is torch.uint8]
    assert ws.owner is stream and Current.stack == [None]
    name, args = library.calls[-1]
    args = [getattr(a, "value", a) for a in args]
    assert ws.address in args and args[-1] == stream.cuda_stream
    call()
    assert [t for t in allocated if t.dtype is torch.uint8][1].owner is None


# ------------------------------------------------------------------------------------------------
# The library launches on the current device: a tensor on another one is refused before the call.
# ------------------------------------------------------------------------------------------------
def _operands(call):
    """The stand-ins of a call by name, on device 0."""
    T, V, d = 6, 10, 64
    rows, stat, param = ((T, d), bf16), ((T,), f32), ((d,), f32)
    return {k: Cuda(*v) for k, v in {
        "moe_norm": dict(x=rows, weight=param, bias=param, residual=rows, y=rows, sum=rows,
                         mean=stat, rstd=stat),
        "moe_norm_backward": dict(dy=rows, x=rows, weight=param, mean=stat, rstd=stat,
                                  dresidual=rows, dx=rows, dweight=param, dbias=param,
                                  workspace=((1 << 20,), torch.uint8)),
        "moe_embed": dict(ids=((T,), torch.int32), table=((V, d), bf16), out=rows,
                          workspace=((256,), torch.uint8)),
        "moe_embed_backward": dict(dout=rows, ids=((T,), torch.int32), d_table=((V, d), f32),
                                   workspace=((1 << 20,), torch.uint8)),
    }[call].items()}


@pytest.mark.parametrize("call", ["moe_norm", "moe_norm_backward", "moe_embed",
                                  "moe_embed_backward"])
def test_a_tensor_on_another_device_is_refused(library, monkeypatch, call):
    more = dict(V=10) if call == "moe_embed_backward" else {}
    ops = _operands(call)
    getattr(moe, call)(**ops, **more)
    assert len(library.calls) == 1
    for name in ops:
        ops = _operands(call)
        ops[name].index = 1
        with pytest.raises(ValueError, match=name):
            getattr(moe, call)(**ops, **more)
    # all of them on a device that is not the current one
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="device"):
        getattr(moe, call)(**_operands(call), **more)
    assert len(library.calls) == 1


def test_a_workspace_size_is_kept_by_device(monkeypatch):
    class Sizes:
        """A library on devices of 100 and 200 SMs."""
        def moe_norm_backward_workspace_size(self, T, d, code):
            return 100 * (torch._C._cuda_getDevice() + 1)
    monkeypatch.setattr(moe, "lib", Sizes)
    moe._norm_backward_bytes.cache_clear()
    got = []
    for dev in (0, 1, 0):
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: dev)
        got.append(moe._norm_backward_bytes(7, 64, 1, dev))
    moe._norm_backward_bytes.cache_clear()
    assert got == [100, 200, 100]


def _adamw(monkeypatch, moments=f32, scales=False, elsewhere=None):
    """moe_adamw on three tensors of 300 elements (host memory: only its addresses are taken);
    elsewhere: (argument, index) of the one on another device."""
    n = 3

    def column(dtype, size=300):
        return [torch.zeros(size).to(dtype) for _ in range(n)]
    kw = dict(params=column(f32), grads=column(bf16), exp_avgs=column(moments),
              exp_avg_sqs=column(moments), copies=column(bf16), schedule=torch.zeros(3),
              grad_scale=torch.zeros(1))
    if scales:
        kw.update(exp_avg_scales=column(f32, 2), exp_avg_sq_scales=column(f32, 2))
    odd = None
    if elsewhere:
        odd = kw[elsewhere[0]]
        odd = odd[elsewhere[1]] if isinstance(odd, list) else odd
    monkeypatch.setattr(moe, "_device", lambda t, name: 0)
    monkeypatch.setattr(moe, "_device_of", lambda t: int(t is odd))
    monkeypatch.setattr(moe, "_look", lambda t, name, dev: None)
    return moe.moe_adamw(step=1, **kw)


@pytest.mark.parametrize("name", ["params", "grads", "exp_avgs", "exp_avg_sqs", "copies",
                                  "exp_avg_scales", "exp_avg_sq_scales"])
def test_adamw_refuses_a_list_over_several_devices(library, monkeypatch, name):
    kw = dict(moments=torch.float8_e4m3fn, scales=True)
    _adamw(monkeypatch, **kw)
    assert len(library.calls) == 1
    for i in range(3):
        with pytest.raises(ValueError, match=name):
            _adamw(monkeypatch, **kw, elsewhere=(name, i))
    assert len(library.calls) == 1


@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.int8, torch.bool, f32])
def test_adamw_refuses_8_bit_moments_of_another_kind(library, monkeypatch, dtype):
    """E5M2 numbers or integers would be read as E4M3 numbers."""
    for good in (torch.float8_e4m3fn, torch.uint8):
        _adamw(monkeypatch, moments=good, scales=True)
    assert len(library.calls) == 2
    with pytest.raises(TypeError, match="exp_avgs"):
        _adamw(monkeypatch, moments=dtype, scales=True)
    assert len(library.calls) == 2
