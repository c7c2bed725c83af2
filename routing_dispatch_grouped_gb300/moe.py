"""Python binding of libmoe (ctypes). Argument marshalling only: every step runs in the library's
CUDA kernels. Tensors are PyTorch CUDA tensors (PyTorch provides device memory and streams);
outputs and workspaces not passed in are allocated here with torch.

`stream` is the stream that a call's work is enqueued on (the current one if None). A workspace that
a call allocates belongs to it. Outputs belong to the current stream whatever `stream` is, as with
any PyTorch call: let the given stream wait for the current one first, or pass them in.

The functions keep the C names: moe_route, moe_dispatch, moe_gate_up, moe_down, moe_experts,
moe_combine, moe_forward. A non-zero status raises MoEError. There is no CPU fallback: if the
library is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

SOFTMAX, SIGMOID = 0, 1
RENORMALIZE, SCALE_INPUT, FUSE_COMBINE_WEIGHT, WEIGHTS_PACKED, WGRAD_BF16 = 1, 2, 4, 8, 16
NORM_RMS, IDS_64 = 32, 64
ADAMW_BLOCK = 256  # elements that share one scale of an 8-bit moment
W_GATE_UP, W_DOWN = 0, 1
F32, BF16 = 0, 1
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
          3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_BOUNDS",
          6: "MOE_ERR_TIMEOUT"}

# name -> (restype, argtypes)
_P, _I, _U, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
_F, _D = ctypes.c_float, ctypes.c_double
SIGNATURES = {
    "moe_route": (_I, [_P, _I, _I, _I, _I, _U, _P, _P, _P]),
    "moe_route_hidden": (_I, [_P, _I, _P, _P, _I, _I, _I, _I, _I, _U, _P, _P, _P, _P]),
    "moe_dispatch": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_dispatch_workspace_size": (_S, [_I, _I, _I]),
    "moe_dispatch_noalloc": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "moe_gate_up": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _U, _P, _P, _S, _P]),
    "moe_down": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _U, _P, _P, _S, _P]),
    "moe_experts": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _U, _P, _P, _P, _S, _P]),
    "moe_experts_workspace_size": (_S, []),
    "moe_combine": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "moe_packed_weights_size": (_S, [_I, _I, _I, _I, _I]),
    "moe_pack_weights": (_I, [_I, _P, _P, _I, _I, _I, _I, _P]),
    "moe_forward": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _U, _P, _P, _P, _P, _I, _P, _P,
                         _P, _P, _S, _P]),
    "moe_forward_workspace_size": (_S, [_I, _I, _I, _I, _I, _I, _I]),
    "moe_forward_host": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _U, _P, _P, _P, _P, _I, _P,
                              _P, _S, _P]),
    "moe_forward_host_workspace_size": (_S, [_I, _I, _I, _I, _I, _I, _I]),
    "moe_forward_kernel_count": (_I, [_I, _I, _I, _I]),
    "moe_gemm_kernel_name": (ctypes.c_char_p, [_I, _I, _I, _I]),
    "moe_gate_up_train": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _U, _P, _P, _P, _S,
                               _P]),
    "moe_combine_backward": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P]),
    "moe_down_backward_workspace_size": (_S, [_I, _I, _I]),
    "moe_down_backward": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _U, _P, _P, _P, _S,
                               _P]),
    "moe_gate_up_backward": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _U, _P, _P, _S, _P]),
    "moe_weight_grad": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _S, _P]),
    "moe_weight_grad_bf16": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _S, _P]),
    "moe_route_backward": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _U, _P, _P]),
    "moe_forward_train_workspace_size": (_S, [_I, _I, _I, _I, _I, _I, _I]),
    "moe_forward_train": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _U, _P, _P, _P, _P, _I, _P,
                               _P, _P, _P, _S, _P]),
    "moe_backward_workspace_size": (_S, [_I, _I, _I, _I, _I, _I, _I]),
    "moe_backward": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _U, _P, _P, _P, _P, _I, _P,
                          _P, _P, _S, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_backward_kernel_count": (_I, [_I, _I, _I, _U, _I]),
    "moe_mx_weights_size": (_S, [_I, _I, _I, _I]),
    "moe_quantize_weights_mx": (_I, [_I, _P, _P, _I, _I, _I, _P]),
    "moe_dequantize_weights_mx": (_I, [_I, _P, _P, _I, _I, _I, _P]),
    "moe_quantize_rows_mx": (_I, [_P, _I, _I, _P, _P, _P, _P]),
    "moe_forward_mx_workspace_size": (_S, [_I, _I, _I, _I, _I, _I]),
    "moe_forward_mx": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _U, _P, _P, _P, _P, _I, _P, _P, _P,
                            _P, _S, _P]),
    "moe_mx_tc_weights_size": (_S, [_I, _I, _I, _I]),
    "moe_quantize_weights_mx_tc": (_I, [_I, _P, _P, _I, _I, _I, _P]),
    "moe_dequantize_weights_mx_tc": (_I, [_I, _P, _P, _I, _I, _I, _P]),
    "moe_mx_tc_rows": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_gate_up_mx_tc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _U, _P, _P, _P, _S,
                               _P]),
    "moe_down_mx_tc": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _S, _P]),
    "moe_forward_mx_tc_workspace_size": (_S, [_I, _I, _I, _I, _I, _I]),
    "moe_forward_mx_tc_kernel_count": (_I, [_I, _I, _I, _I, _I]),
    "moe_forward_mx_tc": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _U, _P, _P, _P, _P, _I, _P, _P,
                               _P, _P, _S, _P]),
    "moe_norm": (_I, [_P, _P, _I, _I, _I, _P, _P, _I, _F, _U, _P, _P, _P, _P, _P]),
    "moe_norm_backward_workspace_size": (_S, [_I, _I, _I]),
    "moe_norm_backward": (_I, [_P, _P, _I, _I, _I, _P, _I, _P, _P, _P, _U, _P, _P, _P, _P, _S,
                               _P]),
    "moe_embed": (_I, [_P, _P, _I, _I, _I, _I, _F, _U, _P, _P, _S, _P]),
    "moe_embed_backward_workspace_size": (_S, [_I, _I]),
    "moe_embed_backward": (_I, [_P, _P, _I, _I, _I, _I, _F, _U, _P, _P, _S, _P]),
    "moe_adamw": (_I, [_P, _I, _D, _D, _D, _D, ctypes.c_int64, _P, _P, _P]),
    "moe_read_device_status": (_I, [_P, _P]),
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_debug_set_gemm_stall_ns": (None, [ctypes.c_uint32]),
}

_lib = None


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")


def lib() -> ctypes.CDLL:
    """Load libmoe.so (built in-tree by routing_dispatch_grouped_gb300.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m routing_dispatch_grouped_gb300.build`")
        cdll = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(cdll, name)
            f.restype, f.argtypes = res, args
        _lib = cdll
    return _lib


def _check(fn: str, st: int):
    if st != 0:
        raise MoEError(fn, st)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need(t: torch.Tensor, name: str):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t


class PackedWeights:
    """Expert weights repacked by moe_pack_weights (bf16): `data` is the packed buffer, kind is
    W_GATE_UP (logical [E, K=d, 2I], N = I) or W_DOWN (logical [E, K=I, N=d])."""

    def __init__(self, data: torch.Tensor, kind: int, E: int, K: int, N: int, tc=False):
        self.data, self.kind, self.E, self.K, self.N = data, kind, E, K, N
        self.tc = tc  # True: the MX tensor-core layout (moe_quantize_weights_mx_tc)

    def data_ptr(self):
        return self.data.data_ptr()


def moe_packed_weights_size(kind, E, K, N) -> int:
    return lib().moe_packed_weights_size(kind, E, K, N, BF16)


def pack_weights(w: torch.Tensor, kind: int, stream=None) -> PackedWeights:
    """Repack gate_up ([E, d, 2I] or [d, 2I]) or down ([E, I, d] or [I, d]) bf16 weights."""
    _need(w, "w")
    w3 = w.unsqueeze(0) if w.dim() == 2 else w
    E, K, C = w3.shape
    N = C // 2 if kind == W_GATE_UP else C
    out = torch.empty(moe_packed_weights_size(kind, E, K, N), dtype=torch.uint8,
                      device=w.device)
    _check("moe_pack_weights", lib().moe_pack_weights(kind, _p(w3), _p(out), _dt(w3), E, K, N,
                                                      _stream(stream)))
    return PackedWeights(out, kind, E, K, N)


def _w_dims(w, kind):
    """(E, K, N, flag) of a weight argument, packed or not."""
    if isinstance(w, PackedWeights):
        assert w.kind == kind, "packed weights of the other kind"
        return w.E, w.K, w.N, WEIGHTS_PACKED
    E, K, C = w.shape
    return E, K, (C // 2 if kind == W_GATE_UP else C), 0


def _workspace(nbytes: int, device, stream) -> torch.Tensor:
    """A workspace of one call, from the memory of the stream that the call was given: nothing
    orders that stream behind the current one, whose earlier work may still use a block of its own,
    and whose later work would be given the block, once it is dropped, while the given stream still
    uses it."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _workspace(nbytes, device, None)
    # torch's caching allocator returns blocks aligned to at least 512 bytes
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------------------------------------
def moe_route(logits, k, score_fn=SOFTMAX, renormalize=True, topk_ids=None, topk_weights=None,
              stream=None):
    _need(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    ids = topk_ids if topk_ids is not None else torch.empty(T, k, dtype=torch.int32, device=dev)
    w = topk_weights if topk_weights is not None else torch.empty(T, k, dtype=torch.float32,
                                                                  device=dev)
    _check("moe_route", lib().moe_route(_p(logits), T, E, k, score_fn,
                                        RENORMALIZE if renormalize else 0, _p(ids), _p(w),
                                        _stream(stream)))
    return ids, w


def moe_route_hidden(x, w_router, k, score_fn=SOFTMAX, renormalize=True, bias=None,
                     logits=None, topk_ids=None, topk_weights=None, want_logits=True,
                     stream=None):
    """Router logits x @ w_router (+ bias) and the top-k in one kernel. Returns
    (topk_ids, topk_weights, logits or None)."""
    _need(x, "x")
    _need(w_router, "w_router")
    T, d = x.shape
    E = w_router.shape[1]
    dev = x.device
    ids = topk_ids if topk_ids is not None else torch.empty(T, k, dtype=torch.int32, device=dev)
    w = topk_weights if topk_weights is not None else torch.empty(T, k, dtype=torch.float32,
                                                                  device=dev)
    if logits is None and want_logits:
        logits = torch.empty(T, E, dtype=torch.float32, device=dev)
    _check("moe_route_hidden", lib().moe_route_hidden(
        _p(x), _dt(x), _p(w_router), _p(bias), T, d, E, k, score_fn,
        RENORMALIZE if renormalize else 0, _p(logits), _p(ids), _p(w), _stream(stream)))
    return ids, w, logits


def moe_dispatch_workspace_size(T, E, k) -> int:
    return lib().moe_dispatch_workspace_size(T, E, k)


def moe_dispatch(topk_ids, E, x=None, workspace=None, out=None, stream=None):
    """Returns dict(counts, offsets, sorted_to_slot, slot_to_sorted, x_sorted, workspace)."""
    _need(topk_ids, "topk_ids")
    T, k = topk_ids.shape
    R = T * k
    dev = topk_ids.device
    o = dict(out or {})
    o.setdefault("counts", torch.empty(E, dtype=torch.int32, device=dev))
    o.setdefault("offsets", torch.empty(E + 1, dtype=torch.int32, device=dev))
    o.setdefault("sorted_to_slot", torch.empty(R, dtype=torch.int32, device=dev))
    o.setdefault("slot_to_sorted", torch.empty(R, dtype=torch.int32, device=dev))
    d, dt = 0, BF16
    if x is not None:
        _need(x, "x")
        d, dt = x.shape[1], _dt(x)
        o.setdefault("x_sorted", torch.empty(R, d, dtype=x.dtype, device=dev))
    else:
        o["x_sorted"] = None
    ws = workspace if workspace is not None else _workspace(moe_dispatch_workspace_size(T, E, k),
                                                            dev, stream)
    _check("moe_dispatch", lib().moe_dispatch(
        _p(topk_ids), _p(x), dt, T, d, E, k, _p(o["counts"]), _p(o["offsets"]),
        _p(o["sorted_to_slot"]), _p(o["slot_to_sorted"]), _p(o["x_sorted"]), _p(ws),
        ws.numel(), _stream(stream)))
    o["workspace"] = ws
    return o


def moe_experts_workspace_size() -> int:
    return lib().moe_experts_workspace_size()


def moe_gate_up(x_rows, offsets, w_gate_up, sorted_to_slot=None, topk_weights=None,
                scale_input=False, h=None, workspace=None, stream=None):
    _need(x_rows, "x_rows")
    R, d = x_rows.shape
    E, _, I, pk = _w_dims(w_gate_up, W_GATE_UP)
    dev = x_rows.device
    h = h if h is not None else torch.empty(R, I, dtype=x_rows.dtype, device=dev)
    ws = workspace if workspace is not None else _workspace(moe_experts_workspace_size(), dev,
                                                            stream)
    _check("moe_gate_up", lib().moe_gate_up(
        _p(x_rows), _p(offsets), _p(sorted_to_slot), _p(topk_weights), _dt(x_rows), R, d, E, I,
        _p(w_gate_up), (SCALE_INPUT if scale_input else 0) | pk, _p(h), _p(ws), ws.numel(),
        _stream(stream)))
    return h


def moe_down(h, offsets, w_down, sorted_to_slot=None, topk_weights=None, fuse_weight=False,
             y_sorted=None, workspace=None, stream=None):
    _need(h, "h")
    R, I = h.shape
    E, _, d, pk = _w_dims(w_down, W_DOWN)
    dev = h.device
    y = y_sorted if y_sorted is not None else torch.empty(R, d, dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else _workspace(moe_experts_workspace_size(), dev,
                                                            stream)
    _check("moe_down", lib().moe_down(
        _p(h), _p(offsets), _p(sorted_to_slot), _p(topk_weights), _dt(h), R, d, E, I,
        _p(w_down), (FUSE_COMBINE_WEIGHT if fuse_weight else 0) | pk, _p(y), _p(ws), ws.numel(),
        _stream(stream)))
    return y


def moe_experts(x_sorted, offsets, w_gate_up, w_down, sorted_to_slot=None, topk_weights=None,
                flags=0, h=None, y_sorted=None, workspace=None, stream=None):
    _need(x_sorted, "x_sorted")
    R, d = x_sorted.shape
    E, _, I, pk = _w_dims(w_gate_up, W_GATE_UP)
    flags |= pk
    dev = x_sorted.device
    h = h if h is not None else torch.empty(R, I, dtype=x_sorted.dtype, device=dev)
    y = y_sorted if y_sorted is not None else torch.empty(R, d, dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else _workspace(moe_experts_workspace_size(), dev,
                                                            stream)
    _check("moe_experts", lib().moe_experts(
        _p(x_sorted), _p(offsets), _p(sorted_to_slot), _p(topk_weights), _dt(x_sorted), R, d, E,
        I, _p(w_gate_up), _p(w_down), flags, _p(h), _p(y), _p(ws), ws.numel(), _stream(stream)))
    return h, y


def moe_combine(y_sorted, slot_to_sorted, k, out_dtype, topk_weights=None, y_shared=None,
                out=None, stream=None):
    _need(y_sorted, "y_sorted")
    R, d = y_sorted.shape
    T = slot_to_sorted.numel() // k
    out = out if out is not None else torch.empty(T, d, dtype=out_dtype, device=y_sorted.device)
    _check("moe_combine", lib().moe_combine(
        _p(y_sorted), _p(slot_to_sorted), _p(topk_weights), _p(y_shared), T, d, k, _dt(out),
        _p(out), _stream(stream)))
    return out


def moe_forward_workspace_size(T, d, E, k, I, Is, dtype) -> int:
    return lib().moe_forward_workspace_size(T, d, E, k, I, Is, BF16 if dtype == torch.bfloat16
                                            else F32)


def moe_forward_kernel_count(T, k, Is, dtype=torch.bfloat16) -> int:
    return lib().moe_forward_kernel_count(BF16 if dtype == torch.bfloat16 else F32, T, k, Is)


def moe_gemm_kernel_name(kind, R, E, grouped=True) -> str:
    """The grouped GEMM kernel a bf16 gate_up (kind W_GATE_UP) or down (W_DOWN) call of R rows
    over E experts launches."""
    return lib().moe_gemm_kernel_name(kind, R, E, 1 if grouped else 0).decode()


def moe_forward(x, logits, w_gate_up, w_down, k, score_fn=SOFTMAX, flags=RENORMALIZE,
                w_shared_gate_up=None, w_shared_down=None, out=None, topk_ids=None,
                topk_weights=None, workspace=None, stream=None):
    """The whole layer. Returns (out, topk_ids, topk_weights, workspace)."""
    _need(x, "x")
    _need(logits, "logits")
    T, d = x.shape
    E, _, I, pk = _w_dims(w_gate_up, W_GATE_UP)
    flags |= pk
    Is = 0
    if w_shared_gate_up is not None:
        Is = (w_shared_gate_up.N if isinstance(w_shared_gate_up, PackedWeights)
              else w_shared_gate_up.shape[-1] // 2)
    dev = x.device
    out = out if out is not None else torch.empty(T, d, dtype=x.dtype, device=dev)
    ids = topk_ids if topk_ids is not None else torch.empty(T, k, dtype=torch.int32, device=dev)
    w = topk_weights if topk_weights is not None else torch.empty(T, k, dtype=torch.float32,
                                                                  device=dev)
    ws = workspace if workspace is not None else _workspace(
        moe_forward_workspace_size(T, d, E, k, I, Is, x.dtype), dev, stream)
    _check("moe_forward", lib().moe_forward(
        _p(x), _p(logits), _dt(x), T, d, E, k, I, score_fn, flags, _p(w_gate_up), _p(w_down),
        _p(w_shared_gate_up), _p(w_shared_down), Is, _p(ids), _p(w), _p(out), _p(ws), ws.numel(),
        _stream(stream)))
    return out, ids, w, ws


def moe_forward_host_workspace_size(T, d, E, k, I, Is, dtype) -> int:
    return lib().moe_forward_host_workspace_size(T, d, E, k, I, Is,
                                                 BF16 if dtype == torch.bfloat16 else F32)


def moe_forward_host(x_host, logits_host, w_gate_up, w_down, k, score_fn=SOFTMAX,
                     flags=RENORMALIZE, w_shared_gate_up=None, w_shared_down=None, out=None,
                     workspace=None, stream=None, device=None):
    """The whole layer on host activations (CPU tensors): pinned ones are read and written in
    place by the kernels, pageable ones copied in and out by the library on `stream`. Returns
    (out_host, workspace); synchronise the stream before reading out_host."""
    if x_host.is_cuda or logits_host.is_cuda:
        raise ValueError("moe_forward_host takes host tensors")
    x_host, logits_host = x_host.contiguous(), logits_host.contiguous()
    T, d = x_host.shape
    E, _, I, pk = _w_dims(w_gate_up, W_GATE_UP)
    flags |= pk
    Is = 0
    if w_shared_gate_up is not None:
        Is = (w_shared_gate_up.N if isinstance(w_shared_gate_up, PackedWeights)
              else w_shared_gate_up.shape[-1] // 2)
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    out = out if out is not None else torch.empty(T, d, dtype=x_host.dtype).pin_memory()
    ws = workspace if workspace is not None else _workspace(
        moe_forward_host_workspace_size(T, d, E, k, I, Is, x_host.dtype), dev, stream)
    _check("moe_forward_host", lib().moe_forward_host(
        _p(x_host), _p(logits_host), _dt(x_host), T, d, E, k, I, score_fn, flags,
        _p(w_gate_up), _p(w_down), _p(w_shared_gate_up), _p(w_shared_down), Is, _p(out), _p(ws),
        ws.numel(), _stream(stream)))
    return out, ws


def moe_read_device_status(workspace, stream=None) -> int:
    return lib().moe_read_device_status(_p(workspace), _stream(stream))


def forward_workspace_views(ws: torch.Tensor, T, d, E, k, I, Is, dtype, mx=False):
    """Views of the intermediates moe_forward (moe_forward_mx with mx=True) leaves in its
    workspace (for tests and tools);
    the offsets follow the library's layout rule: 256-byte status word, then (decode batches
    only) the one-kernel layer's counters, counts, offsets,
    dispatch scratch, sorted_to_slot, slot_to_sorted, x_sorted, h, y_sorted, shared h, shared y,
    each rounded up to 256 bytes."""
    R = T * k
    b = 2 if dtype == torch.bfloat16 else 4
    nchunks = (R + 255) // 256
    # decode batches run the one-kernel layer, whose counters follow the status word
    fused = dtype == torch.bfloat16 and Is == 0 and 1 <= T <= 16 and R <= 256
    nbd = (d + 63) // 64
    fcnt = (2 * R * ((I + 63) // 64) + nbd + (nbd + 3) // 4) * 4 if fused else 0
    sizes = [("fused_counters", fcnt), ("counts", E * 4), ("offsets", (E + 1) * 4), ("chunk", nchunks * E * 4),
             ("sorted_to_slot", R * 4), ("slot_to_sorted", R * 4), ("x_sorted", R * d * b),
             ("h", R * I * b), ("y_sorted", R * d * 4), ("h_shared", T * Is * b),
             ("y_shared", T * d * 4 if Is else 0)]
    views, o = {}, 256
    for name, nbytes in sizes:
        views[name] = ws[o:o + nbytes]
        o = (o + nbytes + 255) // 256 * 256
    v = views
    if mx and fused:
        # the one-kernel layer on MX weights: its partial sums, then h's MXFP8 codes and scales
        nbh = (I + 63) // 64
        part_b = ((512 + R * nbh) * T * 128 * 4 + 255) // 256 * 256
        part = part_b + ((512 + nbd) * T * 64 * 4 + 255) // 256 * 256
        if nbh < 512 and nbd * T <= 1024:  # the owner layout's down partials [nbh][R][d]
            part += (nbh * R * d * 4 + 255) // 256 * 256
        o = (o + part + 255) // 256 * 256
        views["h_codes"] = ws[o:o + R * I]
        o = (o + R * I + 255) // 256 * 256
        views["h_scales"] = ws[o:o + R * ((I + 31) // 32)]
    out = {
        "counts": v["counts"].view(torch.int32),
        "offsets": v["offsets"].view(torch.int32),
        "sorted_to_slot": v["sorted_to_slot"].view(torch.int32),
        "slot_to_sorted": v["slot_to_sorted"].view(torch.int32),
        "x_sorted": v["x_sorted"].view(dtype).view(R, d),
        "h": v["h"].view(dtype).view(R, I),
        "y_sorted": v["y_sorted"].view(torch.float32).view(R, d),
    }
    if Is:
        out["h_shared"] = v["h_shared"].view(dtype).view(T, Is)
        out["y_shared"] = v["y_shared"].view(torch.float32).view(T, d)
    if "h_codes" in v:
        out["h_codes"] = v["h_codes"].view(R, I)
        out["h_scales"] = v["h_scales"].view(R, (I + 31) // 32)
    return out


# ------------------------------------------------------------------------------------------------
# training: the forward that keeps what the backward reads, and the backward pass
# ------------------------------------------------------------------------------------------------
def _code(dtype):
    return BF16 if dtype == torch.bfloat16 else F32


def moe_gate_up_train(x_rows, offsets, w_gate_up, sorted_to_slot=None, topk_weights=None,
                      scale_input=False, h=None, ab=None, workspace=None, stream=None):
    """moe_gate_up that also returns ab = [x W_gate | x W_up] (unscaled, layer dtype)."""
    _need(x_rows, "x_rows")
    R, d = x_rows.shape
    E, _, I, pk = _w_dims(w_gate_up, W_GATE_UP)
    dev = x_rows.device
    h = h if h is not None else torch.empty(R, I, dtype=x_rows.dtype, device=dev)
    ab = ab if ab is not None else torch.empty(R, 2 * I, dtype=x_rows.dtype, device=dev)
    ws = workspace if workspace is not None else _workspace(moe_experts_workspace_size(), dev,
                                                            stream)
    _check("moe_gate_up_train", lib().moe_gate_up_train(
        _p(x_rows), _p(offsets), _p(sorted_to_slot), _p(topk_weights), _dt(x_rows), R, d, E, I,
        _p(w_gate_up), (SCALE_INPUT if scale_input else 0) | pk, _p(h), _p(ab), _p(ws),
        ws.numel(), _stream(stream)))
    return h, ab


def moe_combine_backward(dout, slot_to_sorted, k, topk_weights=None, y_sorted=None,
                         want_weight_grad=True, dy_sorted=None, d_topk_weights=None,
                         stream=None):
    """Returns (dy_sorted [R, d] in dout's dtype, d_topk_weights [T, k] fp32 or None)."""
    _need(dout, "dout")
    T, d = dout.shape
    R = slot_to_sorted.numel()
    dev = dout.device
    dy = dy_sorted if dy_sorted is not None else torch.empty(R, d, dtype=dout.dtype, device=dev)
    dw = None
    if want_weight_grad:
        dw = d_topk_weights if d_topk_weights is not None else torch.empty(
            T, k, dtype=torch.float32, device=dev)
    _check("moe_combine_backward", lib().moe_combine_backward(
        _p(dout), _p(y_sorted if want_weight_grad else None), _p(slot_to_sorted),
        _p(topk_weights), _dt(dout), T, d, k, _p(dy), _p(dw), _stream(stream)))
    return dy, dw


def moe_down_backward(dy_sorted, ab, offsets, w_down, sorted_to_slot=None, topk_weights=None,
                      scale_input=False, d_ab=None, d_topk_weights=None, workspace=None,
                      stream=None):
    """Returns (d_ab [R, 2I], d_topk_weights by slot [R] fp32 or None)."""
    _need(dy_sorted, "dy_sorted")
    R, d = dy_sorted.shape
    E, I, _, pk = _w_dims(w_down, W_DOWN)
    dev = dy_sorted.device
    d_ab = d_ab if d_ab is not None else torch.empty(R, 2 * I, dtype=dy_sorted.dtype, device=dev)
    dw = None
    if scale_input:
        dw = d_topk_weights if d_topk_weights is not None else torch.empty(
            R, dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else _workspace(
        lib().moe_down_backward_workspace_size(R, I, _dt(dy_sorted)), dev, stream)
    _check("moe_down_backward", lib().moe_down_backward(
        _p(dy_sorted), _p(ab), _p(offsets), _p(sorted_to_slot), _p(topk_weights), _dt(dy_sorted),
        R, d, E, I, _p(w_down), (SCALE_INPUT if scale_input else 0) | pk, _p(d_ab), _p(dw),
        _p(ws), ws.numel(), _stream(stream)))
    return d_ab, dw


def moe_gate_up_backward(d_ab, offsets, w_gate_up, dx_sorted=None, workspace=None, stream=None):
    """Returns dx_sorted [R, d] fp32."""
    _need(d_ab, "d_ab")
    R = d_ab.shape[0]
    E, d, I, pk = _w_dims(w_gate_up, W_GATE_UP)
    dev = d_ab.device
    dx = dx_sorted if dx_sorted is not None else torch.empty(R, d, dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else _workspace(moe_experts_workspace_size(), dev,
                                                            stream)
    _check("moe_gate_up_backward", lib().moe_gate_up_backward(
        _p(d_ab), _p(offsets), _dt(d_ab), R, d, E, I, _p(w_gate_up), pk, _p(dx), _p(ws),
        ws.numel(), _stream(stream)))
    return dx


def moe_weight_grad(a, b, offsets, E, dw=None, workspace=None, stream=None,
                    out_dtype=torch.float32):
    """dw[e] = a[rows of e]^T b[rows of e]: [E, M, N] fp32, or bf16 (bf16 a, b) with
    out_dtype=torch.bfloat16 (moe_weight_grad_bf16)."""
    _need(a, "a")
    _need(b, "b")
    R, M = a.shape
    N = b.shape[1]
    dev = a.device
    dw = dw if dw is not None else torch.empty(E, M, N, dtype=out_dtype, device=dev)
    ws = workspace if workspace is not None else _workspace(moe_experts_workspace_size(), dev,
                                                            stream)
    if dw.dtype == torch.bfloat16:
        _check("moe_weight_grad_bf16", lib().moe_weight_grad_bf16(
            _p(a), _p(b), _p(offsets), R, M, N, E, _p(dw), _p(ws), ws.numel(), _stream(stream)))
    else:
        _check("moe_weight_grad", lib().moe_weight_grad(
            _p(a), _p(b), _p(offsets), _dt(a), R, M, N, E, _p(dw), _p(ws), ws.numel(),
            _stream(stream)))
    return dw


def moe_route_backward(logits, topk_ids, topk_weights, d_topk_weights, score_fn=SOFTMAX,
                       renormalize=True, d_logits=None, stream=None):
    _need(logits, "logits")
    T, E = logits.shape
    k = topk_ids.shape[1]
    dl = d_logits if d_logits is not None else torch.empty(T, E, dtype=torch.float32,
                                                           device=logits.device)
    _check("moe_route_backward", lib().moe_route_backward(
        _p(logits), _p(topk_ids), _p(topk_weights), _p(d_topk_weights), T, E, k, score_fn,
        RENORMALIZE if renormalize else 0, _p(dl), _stream(stream)))
    return dl


def moe_forward_train_workspace_size(T, d, E, k, I, Is, dtype) -> int:
    return lib().moe_forward_train_workspace_size(T, d, E, k, I, Is, _code(dtype))


def moe_forward_train(x, logits, w_gate_up, w_down, k, score_fn=SOFTMAX, flags=RENORMALIZE,
                      w_shared_gate_up=None, w_shared_down=None, out=None, topk_ids=None,
                      topk_weights=None, workspace=None, stream=None):
    """moe_forward for training. Returns (out, topk_ids, topk_weights, workspace); the
    workspace holds what moe_backward reads."""
    _need(x, "x")
    _need(logits, "logits")
    T, d = x.shape
    E, _, I, pk = _w_dims(w_gate_up, W_GATE_UP)
    flags |= pk
    Is = _shared_width(w_shared_gate_up)
    dev = x.device
    out = out if out is not None else torch.empty(T, d, dtype=x.dtype, device=dev)
    ids = topk_ids if topk_ids is not None else torch.empty(T, k, dtype=torch.int32, device=dev)
    w = topk_weights if topk_weights is not None else torch.empty(T, k, dtype=torch.float32,
                                                                  device=dev)
    ws = workspace if workspace is not None else _workspace(
        moe_forward_train_workspace_size(T, d, E, k, I, Is, x.dtype), dev, stream)
    _check("moe_forward_train", lib().moe_forward_train(
        _p(x), _p(logits), _dt(x), T, d, E, k, I, score_fn, flags, _p(w_gate_up), _p(w_down),
        _p(w_shared_gate_up), _p(w_shared_down), Is, _p(ids), _p(w), _p(out), _p(ws), ws.numel(),
        _stream(stream)))
    return out, ids, w, ws


def _shared_width(w_shared_gate_up):
    if w_shared_gate_up is None:
        return 0
    return (w_shared_gate_up.N if isinstance(w_shared_gate_up, PackedWeights)
            else w_shared_gate_up.shape[-1] // 2)


def moe_backward_workspace_size(T, d, E, k, I, Is, dtype) -> int:
    return lib().moe_backward_workspace_size(T, d, E, k, I, Is, _code(dtype))


def moe_backward_kernel_count(T, k, Is, flags, want_logits=True) -> int:
    return lib().moe_backward_kernel_count(T, k, Is, flags, 1 if want_logits else 0)


def moe_backward(dout, x, logits, w_gate_up, w_down, k, topk_ids, topk_weights, fwd_workspace,
                 score_fn=SOFTMAX, flags=RENORMALIZE, w_shared_gate_up=None, w_shared_down=None,
                 want_logits=True, out=None, workspace=None, stream=None):
    """The whole backward pass for a moe_forward_train call with the same arguments.
    Returns a dict: dx, d_w_gate_up, d_w_down, d_topk_weights, d_logits (None unless
    want_logits) and, with a shared expert, d_w_shared_gate_up, d_w_shared_down. `out` may
    pass preallocated tensors under those names. flags may include WGRAD_BF16: the weight
    gradients are then bf16."""
    _need(dout, "dout")
    T, d = dout.shape
    E, _, I, pk = _w_dims(w_gate_up, W_GATE_UP)
    flags |= pk
    Is = _shared_width(w_shared_gate_up)
    dev = dout.device
    o = dict(out or {})
    f32 = torch.float32

    def get(name, shape, dtype):
        if o.get(name) is None:
            o[name] = torch.empty(*shape, dtype=dtype, device=dev)
        return o[name]

    wdt = torch.bfloat16 if flags & WGRAD_BF16 else f32
    dx = get("dx", (T, d), dout.dtype)
    dwgu = get("d_w_gate_up", (E, d, 2 * I), wdt)
    dwd = get("d_w_down", (E, I, d), wdt)
    dtw = get("d_topk_weights", (T, k), f32)
    dl = get("d_logits", (T, E), f32) if want_logits else None
    o.setdefault("d_logits", dl)
    dsgu = get("d_w_shared_gate_up", (d, 2 * Is), wdt) if Is else None
    dsd = get("d_w_shared_down", (Is, d), wdt) if Is else None
    ws = workspace if workspace is not None else _workspace(
        moe_backward_workspace_size(T, d, E, k, I, Is, dout.dtype), dev, stream)
    _check("moe_backward", lib().moe_backward(
        _p(dout), _p(x), _p(logits), _dt(dout), T, d, E, k, I, score_fn, flags, _p(w_gate_up),
        _p(w_down), _p(w_shared_gate_up), _p(w_shared_down), Is, _p(topk_ids), _p(topk_weights),
        _p(fwd_workspace), fwd_workspace.numel(), _p(dx), _p(dwgu), _p(dwd), _p(dsgu), _p(dsd),
        _p(dtw), _p(dl), _p(ws), ws.numel(), _stream(stream)))
    o["workspace"] = ws
    return o


def backward_workspace_views(ws: torch.Tensor, T, d, k, I, dtype):
    """Views of the intermediates moe_backward leaves in its workspace (for tests): dy_sorted
    [R, d], d_ab [R, 2I] (layer dtype) and dx_sorted [R, d] fp32, after the 256-byte status word,
    each rounded up to 256 bytes."""
    R = T * k
    b = 2 if dtype == torch.bfloat16 else 4
    views, o = {}, 256
    for name, nbytes in [("dy_sorted", R * d * b), ("d_ab", R * 2 * I * b),
                         ("dx_sorted", R * d * 4)]:
        views[name] = ws[o:o + nbytes]
        o = (o + nbytes + 255) // 256 * 256
    return {"dy_sorted": views["dy_sorted"].view(dtype).view(R, d),
            "d_ab": views["d_ab"].view(dtype).view(R, 2 * I),
            "dx_sorted": views["dx_sorted"].view(torch.float32).view(R, d)}


def forward_train_workspace_views(ws: torch.Tensor, T, d, E, k, I, Is, dtype):
    """forward_workspace_views for moe_forward_train's workspace, plus "ab" [R, 2I] and (shared
    expert) "ab_shared" [T, 2Is]."""
    R = T * k
    b = 2 if dtype == torch.bfloat16 else 4
    nchunks = (R + 255) // 256
    sizes = [("counts", E * 4), ("offsets", (E + 1) * 4), ("chunk", nchunks * E * 4),
             ("sorted_to_slot", R * 4), ("slot_to_sorted", R * 4), ("x_sorted", R * d * b),
             ("h", R * I * b), ("y_sorted", R * d * 4), ("h_shared", T * Is * b),
             ("y_shared", T * d * 4 if Is else 0), ("fused", 0), ("ab", R * 2 * I * b),
             ("ab_shared", T * 2 * Is * b)]
    views, o = {}, 256
    for name, nbytes in sizes:
        views[name] = ws[o:o + nbytes]
        o = (o + nbytes + 255) // 256 * 256
    v = views
    out = {
        "counts": v["counts"].view(torch.int32),
        "offsets": v["offsets"].view(torch.int32),
        "sorted_to_slot": v["sorted_to_slot"].view(torch.int32),
        "slot_to_sorted": v["slot_to_sorted"].view(torch.int32),
        "x_sorted": v["x_sorted"].view(dtype).view(R, d),
        "h": v["h"].view(dtype).view(R, I),
        "y_sorted": v["y_sorted"].view(torch.float32).view(R, d),
        "ab": v["ab"].view(dtype).view(R, 2 * I),
    }
    if Is:
        out["h_shared"] = v["h_shared"].view(dtype).view(T, Is)
        out["y_shared"] = v["y_shared"].view(torch.float32).view(T, d)
        out["ab_shared"] = v["ab_shared"].view(dtype).view(T, 2 * Is)
    return out


# ------------------------------------------------------------------------------------------------
# around the layer: norm, embedding, AdamW
# ------------------------------------------------------------------------------------------------
# A decode step's norm or look-up takes the GPU 2 us, so these calls keep the host's part short:
# plain integers as pointers, the stream's handle without a stream object, and one look at each
# tensor that the caller gives.
_CODE = {torch.float32: F32, torch.bfloat16: BF16}


def _device(t, name):
    """The current device, on which the library launches and where every tensor has to be."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return torch._C._cuda_getDevice()


def _current(dev, stream):
    """The stream's handle: the one given, or the current one of the current device."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _dtype_code(t, name):
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} of {name}")
    return code


def _look(t, name, dev):
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor on the current device")


def _ptr(t, name, shape, dtype, dev):
    """t's address (None for None): a contiguous tensor on dev of this shape and dtype."""
    if t is None:
        return None
    _look(t, name, dev)
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must have shape {tuple(shape)} and dtype {dtype}")
    return t.data_ptr()


def _rows(t, name, dev):
    _look(t, name, dev)
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    return t.shape


def moe_norm(x, weight=None, bias=None, eps=1e-5, rms=False, residual=None, want_stats=True,
             y=None, sum=None, mean=None, rstd=None, stream=None):
    """Layer norm (rms: root-mean-square norm) of x + residual; weight and bias float32 or
    bfloat16. Returns (y, sum, mean, rstd): sum is None without a residual, mean with rms, both
    statistics without want_stats (unless they were given)."""
    dev = _device(x, "x")
    shape = _rows(x, "x", dev)
    T, d = shape
    dtype = x.dtype
    code = _dtype_code(x, "x")
    wt = torch.float32 if weight is None and bias is None else \
        (bias if weight is None else weight).dtype
    if wt not in _CODE:
        raise TypeError(f"unsupported dtype {wt} of weight or bias")
    wp, bp = _ptr(weight, "weight", (d,), wt, dev), _ptr(bias, "bias", (d,), wt, dev)
    rp = _ptr(residual, "residual", shape, dtype, dev)
    if y is None:
        y = torch.empty_like(x)
    else:
        _ptr(y, "y", shape, dtype, dev)
    if sum is not None:
        _ptr(sum, "sum", shape, dtype, dev)
    elif residual is not None:
        sum = torch.empty_like(x)
    if mean is not None:
        _ptr(mean, "mean", (T,), torch.float32, dev)
    elif want_stats and not rms:
        mean = torch.empty(T, dtype=torch.float32, device=x.device)
    if rstd is not None:
        _ptr(rstd, "rstd", (T,), torch.float32, dev)
    elif want_stats:
        rstd = torch.empty(T, dtype=torch.float32, device=x.device)
    st = lib().moe_norm(x.data_ptr(), rp, code, T, d, wp, bp, _CODE[wt], eps,
                        NORM_RMS if rms else 0, None if sum is None else sum.data_ptr(),
                        y.data_ptr(), None if mean is None else mean.data_ptr(),
                        None if rstd is None else rstd.data_ptr(), _current(dev, stream))
    if st:
        raise MoEError("moe_norm", st)
    return y, sum, mean, rstd


# of sizes and the device (its SM count) alone; a call across the C ABI takes a microsecond
@functools.lru_cache(maxsize=256)
def _norm_backward_bytes(T, d, code, dev):
    return lib().moe_norm_backward_workspace_size(T, d, code)


@functools.lru_cache(maxsize=256)
def _embed_backward_bytes(T, d):
    return lib().moe_embed_backward_workspace_size(T, d)


def moe_norm_backward_workspace_size(T, d, dtype) -> int:
    return lib().moe_norm_backward_workspace_size(T, d, BF16 if dtype == torch.bfloat16 else F32)


def moe_norm_backward(dy, x, weight, mean, rstd, rms=False, dresidual=None, want_weight=True,
                      want_bias=True, dx=None, dweight=None, dbias=None, workspace=None,
                      stream=None):
    """Gradient of moe_norm; x is what was normed (moe_norm's sum if it had a residual), mean and
    rstd its statistics (mean None with rms). Returns (dx, dweight, dbias): dbias is None with
    rms."""
    dev = _device(dy, "dy")
    shape = _rows(dy, "dy", dev)
    T, d = shape
    dtype, f32 = dy.dtype, torch.float32
    code = _dtype_code(dy, "dy")
    xp = _ptr(x, "x", shape, dtype, dev)
    wt = f32 if weight is None else weight.dtype
    if wt not in _CODE:
        raise TypeError(f"unsupported dtype {wt} of weight")
    wp = _ptr(weight, "weight", (d,), wt, dev)
    mp, qp = _ptr(mean, "mean", (T,), f32, dev), _ptr(rstd, "rstd", (T,), f32, dev)
    rp = _ptr(dresidual, "dresidual", shape, dtype, dev)
    if dx is None:
        dx = torch.empty_like(dy)
    else:
        _ptr(dx, "dx", shape, dtype, dev)
    if dweight is not None:
        _ptr(dweight, "dweight", (d,), f32, dev)
    elif want_weight:
        dweight = torch.empty(d, dtype=f32, device=dy.device)
    if dbias is not None:
        _ptr(dbias, "dbias", (d,), f32, dev)
    elif want_bias and not rms:
        dbias = torch.empty(d, dtype=f32, device=dy.device)
    ws = workspace if workspace is not None else _workspace(
        _norm_backward_bytes(T, d, code, dev), dy.device, stream)
    _look(ws, "workspace", dev)
    st = lib().moe_norm_backward(
        dy.data_ptr(), xp, code, T, d, wp, _CODE[wt], mp, qp, rp, NORM_RMS if rms else 0,
        dx.data_ptr(), None if dweight is None else dweight.data_ptr(),
        None if dbias is None else dbias.data_ptr(), ws.data_ptr(), ws.numel(),
        _current(dev, stream))
    if st:
        raise MoEError("moe_norm_backward", st)
    return dx, dweight, dbias


def _ids(ids, dev):
    """(address, flag) of int32 or int64 token ids."""
    _look(ids, "ids", dev)
    if ids.dtype is torch.int64:
        return ids.data_ptr(), IDS_64
    if ids.dtype is not torch.int32:
        raise TypeError("ids must be int32 or int64")
    return ids.data_ptr(), 0


def moe_embed(ids, table, scale=1.0, out=None, workspace=None, stream=None):
    """scale * table[ids] for int32 or int64 ids of any shape; returns [*ids.shape, d]. An id
    outside the table gives a row of zeros; with a workspace (uint8, 256 bytes) its status word says
    so."""
    dev = _device(table, "table")
    ip, flags = _ids(ids, dev)
    V, d = _rows(table, "table", dev)
    dtype = table.dtype
    code = _dtype_code(table, "table")
    if out is None:
        out = torch.empty((*ids.shape, d), dtype=dtype, device=table.device)
    else:
        _ptr(out, "out", (*ids.shape, d), dtype, dev)
    wp, wb = None, 0
    if workspace is not None:
        _look(workspace, "workspace", dev)
        wp, wb = workspace.data_ptr(), workspace.numel()
    st = lib().moe_embed(ip, table.data_ptr(), code, ids.numel(), V, d, scale, flags,
                         out.data_ptr(), wp, wb, _current(dev, stream))
    if st:
        raise MoEError("moe_embed", st)
    return out


def moe_embed_backward_workspace_size(T, d) -> int:
    return lib().moe_embed_backward_workspace_size(T, d)


def moe_embed_backward(dout, ids, V, scale=1.0, grad_dtype=torch.float32, d_table=None,
                       workspace=None, stream=None):
    """Gradient of moe_embed with respect to the table: [V, d] of grad_dtype (float32 or
    bfloat16; d_table's own when given), rows without a token zero."""
    dev = _device(dout, "dout")
    ip, flags = _ids(ids, dev)
    _look(dout, "dout", dev)
    if dout.shape[:-1] != ids.shape:
        raise ValueError("dout must have one row for each id")
    d, T = dout.shape[-1], ids.numel()
    if d_table is None:
        d_table = torch.empty(V, d, dtype=grad_dtype, device=dout.device)
    else:
        _ptr(d_table, "d_table", (V, d), d_table.dtype, dev)
    if _dtype_code(d_table, "d_table") == BF16:
        flags |= WGRAD_BF16
    ws = workspace if workspace is not None else _workspace(_embed_backward_bytes(T, d),
                                                            dout.device, stream)
    _look(ws, "workspace", dev)
    st = lib().moe_embed_backward(
        dout.data_ptr(), ip, _dtype_code(dout, "dout"), T, V, d, scale, flags, d_table.data_ptr(),
        ws.data_ptr(), ws.numel(), _current(dev, stream))
    if st:
        raise MoEError("moe_embed_backward", st)
    return d_table


class AdamwTensor(ctypes.Structure):
    """moe_adamw_tensor of the C ABI."""
    _fields_ = [("param", _P), ("grad", _P), ("exp_avg", _P), ("exp_avg_sq", _P),
                ("exp_avg_scale", _P), ("exp_avg_sq_scale", _P), ("copy_bf16", _P),
                ("n", ctypes.c_int64), ("param_dt", ctypes.c_int32),
                ("grad_dt", ctypes.c_int32), ("weight_decay", _D)]


def adamw_state(param, bits=32):
    """Zero moments for `param`: (exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale); with 8
    bits E4M3 numbers and the scales of their blocks, with 32 bits fp32 and no scales."""
    if bits == 32:
        z = torch.zeros(param.shape, dtype=torch.float32, device=param.device)
        return z, z.clone(), None, None
    if bits != 8:
        raise ValueError("bits must be 8 or 32")
    z = torch.zeros(param.shape, dtype=torch.float8_e4m3fn, device=param.device)
    s = torch.zeros(-(-param.numel() // ADAMW_BLOCK), dtype=torch.float32, device=param.device)
    return z, z.clone(), s, s.clone()


# a property of every tensor of a list, without a Python frame for each
_T = torch.Tensor
_dtype_of, _device_of = _T.dtype.__get__, _T.get_device
_E4M3 = {torch.float8_e4m3fn, torch.uint8}  # the numbers, or their bytes


def _column(ts, name, counts, dtype, dev):
    """Addresses of a list of contiguous tensors on dev with these element counts and one dtype
    (each None: not looked at)."""
    if set(map(_device_of, ts)) != {dev} or not all(map(_T.is_contiguous, ts)):
        raise ValueError(f"{name} must be contiguous CUDA tensors on the current device")
    if counts is not None and list(map(_T.numel, ts)) != counts:
        raise ValueError(f"{name} must have their parameters' element counts")
    if dtype is not None and set(map(_dtype_of, ts)) != {dtype}:
        raise TypeError(f"{name} must be {dtype}")
    return list(map(_T.data_ptr, ts))


def _codes(ts, name):
    try:
        return list(map(_CODE.__getitem__, map(_dtype_of, ts)))
    except KeyError as e:
        raise TypeError(f"unsupported dtype {e} among {name}") from None


def _where(xs):
    """Indices of the entries that are not None."""
    return [] if xs is None else [i for i, x in enumerate(xs) if x is not None]


def moe_adamw(params, grads, exp_avgs, exp_avg_sqs, step, lr=1e-3, beta1=0.9, beta2=0.999,
              eps=1e-8, weight_decay=0.0, copies=None, exp_avg_scales=None,
              exp_avg_sq_scales=None, schedule=None, grad_scale=None, stream=None):
    """One AdamW step, in place, over lists of tensors of one length. params and grads: float32 or
    bfloat16, each tensor's own; copies: bfloat16 tensors (or None entries) that receive the
    updated float32 parameters; moments: float32, or 8-bit with scales (see adamw_state);
    weight_decay: one number or a list. schedule, grad_scale: float32 CUDA tensors of 3 and 1
    elements or None. step counts from 1."""
    n = len(params)
    if n == 0:
        return
    decay = weight_decay if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
    for x in (grads, exp_avgs, exp_avg_sqs, copies, exp_avg_scales, exp_avg_sq_scales, decay):
        if x is not None and len(x) != n:
            raise ValueError("the lists must have one length")
    dev = _device(params[0], "params")
    counts = list(map(_T.numel, params))
    # moe_adamw_tensor as ten 64-bit words: seven addresses, n, the two dtypes, weight_decay
    words = [0] * (10 * n)
    for k, (xs, name) in enumerate(((params, "params"), (grads, "grads"), (exp_avgs, "exp_avgs"),
                                    (exp_avg_sqs, "exp_avg_sqs"))):
        words[k::10] = _column(xs, name, counts if k else None, None, dev)
    eight = _where(exp_avg_scales)
    if eight != _where(exp_avg_sq_scales):
        raise ValueError("exp_avg_scales and exp_avg_sq_scales must go together")
    if eight:
        blocks = [-(-counts[i] // ADAMW_BLOCK) for i in eight]
        for k, xs, name in ((4, exp_avg_scales, "exp_avg_scales"),
                            (5, exp_avg_sq_scales, "exp_avg_sq_scales")):
            for i, p in zip(eight, _column([xs[i] for i in eight], name, blocks, torch.float32,
                                           dev)):
                words[10 * i + k] = p
    for xs, name in ((exp_avgs, "exp_avgs"), (exp_avg_sqs, "exp_avg_sqs")):
        if eight:
            small = set(eight)
            if not {xs[i].dtype for i in eight} <= _E4M3:
                raise TypeError(f"{name} with scales must be float8_e4m3fn (or its bytes, uint8)")
            xs = [x for i, x in enumerate(xs) if i not in small]
        if set(map(_dtype_of, xs)) - {torch.float32}:
            raise TypeError(f"{name} must be float32, or 8-bit with scales")
    copied = _where(copies)
    if copied:
        for i, p in zip(copied, _column([copies[i] for i in copied], "copies",
                                        [counts[i] for i in copied], torch.bfloat16, dev)):
            words[10 * i + 6] = p
    words[7::10] = counts
    words[8::10] = [p | g << 32 for p, g in zip(_codes(params, "params"), _codes(grads, "grads"))]
    bits = {w: struct.unpack("<q", struct.pack("<d", w))[0] for w in set(decay)}
    words[9::10] = map(bits.__getitem__, decay)
    st = lib().moe_adamw(struct.pack(f"{10 * n}q", *words), n, lr, beta1, beta2, eps, step,
                         _ptr(schedule, "schedule", (3,), torch.float32, dev),
                         _ptr(grad_scale, "grad_scale", (1,), torch.float32, dev),
                         _current(dev, stream))
    if st:
        raise MoEError("moe_adamw", st)


# ------------------------------------------------------------------------------------------------
# MX formats: MXFP4 expert weights, MXFP8 activations
# ------------------------------------------------------------------------------------------------
class MxWeights:
    """Expert weights in the MX buffer layout (moe_quantize_weights_mx): `data` holds the E2M1
    codes then the E8M0 scales; kind W_GATE_UP (logical [E, K=d, 2I], N = I) or W_DOWN
    ([E, K=I, N=d])."""

    def __init__(self, data: torch.Tensor, kind: int, E: int, K: int, N: int, tc=False):
        self.data, self.kind, self.E, self.K, self.N = data, kind, E, K, N
        self.tc = tc  # True: the MX tensor-core layout (moe_quantize_weights_mx_tc)

    def data_ptr(self):
        return self.data.data_ptr()


def quantize_weights_mx(w: torch.Tensor, kind: int, stream=None) -> MxWeights:
    """bf16 gate_up ([E, d, 2I] or [d, 2I]) or down ([E, I, d] or [I, d]) weights to MXFP4."""
    _need(w, "w")
    w3 = w.unsqueeze(0) if w.dim() == 2 else w
    E, K, C = w3.shape
    N = C // 2 if kind == W_GATE_UP else C
    out = torch.empty(lib().moe_mx_weights_size(kind, E, K, N), dtype=torch.uint8,
                      device=w.device)
    _check("moe_quantize_weights_mx", lib().moe_quantize_weights_mx(
        kind, _p(w3), _p(out), E, K, N, _stream(stream)))
    return MxWeights(out, kind, E, K, N)


def dequantize_weights_mx(mx: MxWeights, stream=None) -> torch.Tensor:
    cols = 2 * mx.N if mx.kind == W_GATE_UP else mx.N
    w = torch.empty(mx.E, mx.K, cols, dtype=torch.bfloat16, device=mx.data.device)
    _check("moe_dequantize_weights_mx", lib().moe_dequantize_weights_mx(
        mx.kind, _p(mx.data), _p(w), mx.E, mx.K, mx.N, _stream(stream)))
    return w


def quantize_weights_mx_tc(w: torch.Tensor, kind: int, stream=None) -> MxWeights:
    """bf16 gate_up ([E, d, 2I] or [d, 2I]) or down ([E, I, d] or [I, d]) weights to MXFP4 in
    the MX tensor-core layout (the block-scaled GEMMs of moe_forward_mx_tc read it)."""
    _need(w, "w")
    w3 = w.unsqueeze(0) if w.dim() == 2 else w
    E, K, C = w3.shape
    N = C // 2 if kind == W_GATE_UP else C
    n = lib().moe_mx_tc_weights_size(kind, E, K, N)
    if n == 0:
        raise MoEError("moe_mx_tc_weights_size", 1)
    out = torch.empty(n, dtype=torch.uint8, device=w.device)
    _check("moe_quantize_weights_mx_tc", lib().moe_quantize_weights_mx_tc(
        kind, _p(w3), _p(out), E, K, N, _stream(stream)))
    return MxWeights(out, kind, E, K, N, tc=True)


def dequantize_weights_mx_tc(mx: MxWeights, stream=None) -> torch.Tensor:
    cols = 2 * mx.N if mx.kind == W_GATE_UP else mx.N
    w = torch.empty(mx.E, mx.K, cols, dtype=torch.bfloat16, device=mx.data.device)
    _check("moe_dequantize_weights_mx_tc", lib().moe_dequantize_weights_mx_tc(
        mx.kind, _p(mx.data), _p(w), mx.E, mx.K, mx.N, _stream(stream)))
    return w


def quantize_rows_mx(x: torch.Tensor, want_codes=True, stream=None):
    """bf16 rows [R, K] to MXFP8 along K: (rounded bf16 rows, codes uint8 [R, K] or None,
    scales uint8 [R, ceil(K/32)] or None)."""
    _need(x, "x")
    R, K = x.shape
    xo = torch.empty_like(x)
    codes = torch.empty(R, K, dtype=torch.uint8, device=x.device) if want_codes else None
    scales = (torch.empty(R, (K + 31) // 32, dtype=torch.uint8, device=x.device)
              if want_codes else None)
    _check("moe_quantize_rows_mx", lib().moe_quantize_rows_mx(
        _p(x), R, K, _p(xo), _p(codes), _p(scales), _stream(stream)))
    return xo, codes, scales


def moe_forward_mx_workspace_size(T, d, E, k, I, Is) -> int:
    return lib().moe_forward_mx_workspace_size(T, d, E, k, I, Is)


def moe_forward_mx(x, logits, w_gate_up: MxWeights, w_down: MxWeights, k, score_fn=SOFTMAX,
                   flags=RENORMALIZE, w_shared_gate_up=None, w_shared_down=None, out=None,
                   topk_ids=None, topk_weights=None, workspace=None, stream=None):
    """The MX layer. Returns (out, topk_ids, topk_weights, workspace)."""
    _need(x, "x")
    _need(logits, "logits")
    T, d = x.shape
    E, I = w_gate_up.E, w_gate_up.N
    Is = w_shared_gate_up.N if w_shared_gate_up is not None else 0
    dev = x.device
    out = out if out is not None else torch.empty(T, d, dtype=x.dtype, device=dev)
    ids = topk_ids if topk_ids is not None else torch.empty(T, k, dtype=torch.int32, device=dev)
    w = topk_weights if topk_weights is not None else torch.empty(T, k, dtype=torch.float32,
                                                                  device=dev)
    ws = workspace if workspace is not None else _workspace(
        moe_forward_mx_workspace_size(T, d, E, k, I, Is), dev, stream)
    _check("moe_forward_mx", lib().moe_forward_mx(
        _p(x), _p(logits), T, d, E, k, I, score_fn, flags, _p(w_gate_up), _p(w_down),
        _p(w_shared_gate_up), _p(w_shared_down), Is, _p(ids), _p(w), _p(out), _p(ws), ws.numel(),
        _stream(stream)))
    return out, ids, w, ws


def moe_forward_mx_tc_workspace_size(T, d, E, k, I, Is) -> int:
    return lib().moe_forward_mx_tc_workspace_size(T, d, E, k, I, Is)


def moe_forward_mx_tc_kernel_count(T, d, k, I, Is=0) -> int:
    """Kernels moe_forward_mx_tc launches for these sizes (1: the one-kernel decode layer)."""
    return lib().moe_forward_mx_tc_kernel_count(T, d, k, I, Is)


def moe_forward_mx_tc(x, logits, w_gate_up: MxWeights, w_down: MxWeights, k, score_fn=SOFTMAX,
                      flags=RENORMALIZE, w_shared_gate_up=None, w_shared_down=None, out=None,
                      topk_ids=None, topk_weights=None, workspace=None, stream=None):
    """The MX layer on the block-scaled tensor cores (weights from quantize_weights_mx_tc).
    Returns (out, topk_ids, topk_weights, workspace)."""
    _need(x, "x")
    _need(logits, "logits")
    T, d = x.shape
    E, I = w_gate_up.E, w_gate_up.N
    Is = w_shared_gate_up.N if w_shared_gate_up is not None else 0
    dev = x.device
    out = out if out is not None else torch.empty(T, d, dtype=x.dtype, device=dev)
    ids = topk_ids if topk_ids is not None else torch.empty(T, k, dtype=torch.int32, device=dev)
    w = topk_weights if topk_weights is not None else torch.empty(T, k, dtype=torch.float32,
                                                                  device=dev)
    ws = workspace if workspace is not None else _workspace(
        moe_forward_mx_tc_workspace_size(T, d, E, k, I, Is), dev, stream)
    _check("moe_forward_mx_tc", lib().moe_forward_mx_tc(
        _p(x), _p(logits), T, d, E, k, I, score_fn, flags, _p(w_gate_up), _p(w_down),
        _p(w_shared_gate_up), _p(w_shared_down), Is, _p(ids), _p(w), _p(out), _p(ws), ws.numel(),
        _stream(stream)))
    return out, ids, w, ws


def mx_tc_workspace_views(ws: torch.Tensor, T, d, E, k, I, Is):
    """Views of what moe_forward_mx_tc leaves in its workspace (layout of include/moe.h):
    indices, the padded MXFP8 rows of x and h (codes [Rp, K] uint8, scale atoms
    [Rp / 128, ceil(K / 128), 512] uint8), y_sorted and the shared expert's."""
    R = T * k
    Rp = (R + 127) // 128 * 128 + 128 * E
    Tp = (T + 127) // 128 * 128
    kc = lambda K: (K + 127) // 128
    sizes = [("counts", E * 4), ("offsets", (E + 1) * 4), ("chunk", (R + 255) // 256 * E * 4),
             ("sorted_to_slot", R * 4), ("slot_to_sorted", R * 4), ("x_codes", Rp * d),
             ("x_sf", Rp // 128 * kc(d) * 512), ("h_codes", Rp * I),
             ("h_sf", Rp // 128 * kc(I) * 512), ("y_sorted", R * d * 4),
             ("sx_codes", Tp * d if Is else 0), ("sx_sf", Tp // 128 * kc(d) * 512 if Is else 0),
             ("sh_codes", Tp * Is if Is else 0), ("sh_sf", Tp // 128 * kc(Is) * 512 if Is else 0),
             ("y_shared", T * d * 4 if Is else 0)]
    v, o = {}, 256
    for name, nbytes in sizes:
        v[name] = ws[o:o + nbytes]
        o = (o + nbytes + 255) // 256 * 256
    out = {"counts": v["counts"].view(torch.int32), "offsets": v["offsets"].view(torch.int32),
           "sorted_to_slot": v["sorted_to_slot"].view(torch.int32),
           "slot_to_sorted": v["slot_to_sorted"].view(torch.int32),
           "x_codes": v["x_codes"].view(Rp, d), "x_sf": v["x_sf"].view(Rp // 128, kc(d), 512),
           "h_codes": v["h_codes"].view(Rp, I), "h_sf": v["h_sf"].view(Rp // 128, kc(I), 512),
           "y_sorted": v["y_sorted"].view(torch.float32).view(R, d), "Rp": Rp, "Tp": Tp}
    if Is:
        out.update({"sx_codes": v["sx_codes"].view(Tp, d),
                    "sx_sf": v["sx_sf"].view(Tp // 128, kc(d), 512),
                    "sh_codes": v["sh_codes"].view(Tp, Is),
                    "sh_sf": v["sh_sf"].view(Tp // 128, kc(Is), 512),
                    "y_shared": v["y_shared"].view(torch.float32).view(T, d)})
    return out


def mx_tc_rows(x, topk_ids, slot_to_sorted, offsets, E, codes, sf, codes_sh=None, sf_sh=None,
               stream=None):
    """x [T, d] bf16 to MXFP8 in the padded tensor-core layout (see moe_mx_tc_rows)."""
    T, d = x.shape
    k = topk_ids.shape[1] if topk_ids is not None else 1
    _check("moe_mx_tc_rows", lib().moe_mx_tc_rows(
        _p(x), T, d, k, E, _p(topk_ids), _p(slot_to_sorted), _p(offsets), _p(codes), _p(sf),
        _p(codes_sh), _p(sf_sh), _stream(stream)))


def moe_gate_up_mx_tc(x_codes, x_sf, offsets, w_gate_up: MxWeights, R, h_codes, h_sf,
                      sorted_to_slot=None, topk_weights=None, scale_input=False,
                      workspace=None, stream=None):
    d, E, I = w_gate_up.K, w_gate_up.E, w_gate_up.N
    ws = workspace if workspace is not None else _workspace(256, x_codes.device, stream)
    _check("moe_gate_up_mx_tc", lib().moe_gate_up_mx_tc(
        _p(x_codes), _p(x_sf), _p(offsets), _p(sorted_to_slot), _p(topk_weights), R, d, E, I,
        _p(w_gate_up), SCALE_INPUT if scale_input else 0, _p(h_codes), _p(h_sf), _p(ws),
        ws.numel(), _stream(stream)))
    return ws


def moe_down_mx_tc(h_codes, h_sf, offsets, w_down: MxWeights, R, y_sorted, workspace=None,
                   stream=None):
    I, E, d = w_down.K, w_down.E, w_down.N
    ws = workspace if workspace is not None else _workspace(256, h_codes.device, stream)
    _check("moe_down_mx_tc", lib().moe_down_mx_tc(
        _p(h_codes), _p(h_sf), _p(offsets), R, I, E, d, _p(w_down), _p(y_sorted), _p(ws),
        ws.numel(), _stream(stream)))
    return ws
