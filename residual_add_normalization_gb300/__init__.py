"""Fused residual-add + normalization on NVIDIA GB300 (sm_103a).

Thin Python binding over the C ABI of ``libb200norm.so`` (``include/b200norm.h``).
It only marshals arguments: checks that tensors are contiguous CUDA tensors of
matching shapes and types, allocates outputs with torch, and passes raw device
pointers and the current CUDA stream.  Every step of every operator runs in the
library's CUDA kernels; there is no CPU or PyTorch fallback -- a missing or
unloadable library raises.

Operators (ONNX Runtime contrib operators, as the webgpu-kernels README pages
describe them):

  skip_rms        com.microsoft.SkipSimplifiedLayerNormalization
  skip_rms_stats  the same, plus the per-row mean / inv_std_var outputs
  gated_rms       com.microsoft.GatedRMSNorm
  skip_group      com.microsoft.SkipGroupNorm

and the operators that stand beside them on a residual stream, in serving and in
training (gradients are calls of their own, not autograd functions):

  skip_layer        layer normalization with the residual add fused in
  skip_layer_stats  the same, plus the per-row mean / inv_std_var outputs
  skip_layer_grad   its gradients
  linear            act(x W^T + b) + residual
  linear_grad       its gradients
  gated_linear      act(x Wg^T + bg) * (x Wu^T + bu)
  gated_linear_grad its gradients

and on query and key heads, on their way to attention:

  rotary                position rotation, or its inverse (its gradient)
  head_rms_rotary       an RMS norm of each head, then the rotation
  head_rms_rotary_grad  its gradients
  rotary_frequencies    the frequencies of a rotation, scaled for long contexts
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

__all__ = ["skip_rms", "skip_rms_stats", "gated_rms", "skip_group", "skip_layer",
           "skip_layer_stats", "skip_layer_grad", "linear", "linear_grad", "linear_status",
           "gated_linear", "gated_linear_grad",
           "ACTIVATIONS", "rotary", "head_rms_rotary", "head_rms_rotary_grad",
           "rotary_frequencies", "ROTARY_SCALINGS",
           "workspace_size",
           "workspace_init", "workspace_status", "noalloc_status", "rows_status", "library",
           "library_path", "B200NormError", "SSLN_EPS_DEFAULT"]

# float32(1e-12): SkipSimplifiedLayerNormalization README, Attributes, epsilon.
SSLN_EPS_DEFAULT = 9.999999960041972e-13

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libb200norm.so")
_lock = threading.Lock()
_lib = None

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


class B200NormError(RuntimeError):
    """A b200norm call returned a non-OK status."""

    def __init__(self, status: int, name: str, detail: str):
        super().__init__(f"{name}: {detail}" if detail else name)
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def library() -> ctypes.CDLL:
    """The loaded C library (loaded on first use; raises if it is not built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is not built; run `python -m residual_add_normalization_gb300.buildlib`"
                " (needs nvcc) -- there is no fallback implementation")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i64, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                                 ctypes.c_size_t)
        sig = {
            "b200norm_version": ([], i32),
            "b200norm_status_string": ([i32], ctypes.c_char_p),
            "b200norm_last_error": ([], ctypes.c_char_p),
            "b200norm_skip_rms": ([vp, vp, vp, vp, vp, vp, i64, i64, i32, f32, vp], i32),
            "b200norm_skip_rms_stats": ([vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, f32, vp],
                                        i32),
            "b200norm_gated_rms": ([vp, vp, vp, vp, i64, i64, i32, f32, vp], i32),
            "b200norm_skip_group_workspace_size": ([i64, i64, i64, i64, i32, i32, i32], sz),
            "b200norm_skip_group": ([vp, vp, i32, ctypes.POINTER(ctypes.c_int64), vp, vp, vp,
                                     vp, vp, i64, i64, i64, i64, i32, i32, i32, f32, i32, i32,
                                     vp, sz, vp], i32),
            "b200norm_skip_group_noalloc": ([vp, vp, i32, ctypes.POINTER(ctypes.c_int64), vp,
                                             vp, vp, vp, vp, i64, i64, i64, i64, i32, i32, i32,
                                             f32, i32, i32, vp], i32),
            "b200norm_skip_group_noalloc_status": ([vp], i32),
            "b200norm_workspace_init": ([vp, sz, vp], i32),
            "b200norm_workspace_status": ([vp, vp], i32),
            "b200norm_rows_status": ([vp], i32),
            "b200norm_skip_layer": ([vp] * 9 + [i64, i64, i32, i32, f32, vp], i32),
            "b200norm_skip_layer_grad_workspace_size": ([i64, i64], sz),
            "b200norm_skip_layer_grad": ([vp] * 10 + [i64, i64, i32, i32, vp, sz, vp], i32),
            "b200norm_linear_workspace_size": ([i64, i64, i64, i32, i32], sz),
            "b200norm_linear": ([vp] * 6 + [i64, i64, i64, i32, i32, vp, sz, vp], i32),
            "b200norm_linear_status": ([vp], i32),
            "b200norm_linear_grad_workspace_size": ([i64, i64, i64, i32, i32, i32], sz),
            "b200norm_linear_grad": ([vp] * 7 + [i64, i64, i64, i32, i32, vp, sz, vp], i32),
            "b200norm_gated_linear_workspace_size": ([i64, i64, i64, i32, i32], sz),
            "b200norm_gated_linear": ([vp] * 5 + [i64, i64, i64, i32, i32, vp, sz, vp], i32),
            "b200norm_gated_linear_grad_workspace_size": ([i64, i64, i64, i32, i32], sz),
            "b200norm_gated_linear_grad": ([vp] * 7 + [i64, i64, i64, i32, i32, vp, sz, vp], i32),
            "b200norm_rotary": ([vp] * 3 + [i64] * 3 + [i32, i32, vp], i32),
            "b200norm_head_rms_rotary": ([vp] * 3 + [i64] * 3 + [i32, i32, f32, vp], i32),
            "b200norm_head_rms_rotary_grad_workspace_size": ([i64] * 5, sz),
            "b200norm_head_rms_rotary_grad": ([vp] * 3 + [i64] * 3 + [i32, i32, f32, vp, sz, vp],
                                              i32),
            "b200norm_rotary_frequencies": ([ctypes.POINTER(ctypes.c_double), i64,
                                             ctypes.c_double, i32] + [ctypes.c_double] * 4, i32),
            "b200norm_testing_barrier_timeout": ([vp, sz, ctypes.c_uint64, vp], i32),
            "b200norm_testing_noalloc_barrier_timeout": ([ctypes.c_uint64, vp], i32),
            "b200norm_testing_force": ([i32, i32], i32),
            "b200norm_testing_force_split": ([i32, i32], i32),
            "b200norm_testing_set_pdl": ([i32], i32),
            "b200norm_testing_force_linear": ([i32] * 4, i32),
            "b200norm_testing_linear_stall": ([i32, ctypes.c_uint64], i32),
            "b200norm_testing_layer_withhold": ([i32, ctypes.c_uint64], i32),
            "b200norm_testing_linear_withhold": ([i32, ctypes.c_uint64], i32),
            "b200norm_testing_pipe_stall": ([i32, ctypes.c_uint64], i32),
            "b200norm_testing_plan_rows": ([i64, i64, i32, i32, ctypes.POINTER(ctypes.c_int64)],
                                           i32),
            "b200norm_testing_plan_gated": ([i64, i64, i32, i32, ctypes.POINTER(ctypes.c_int64)],
                                            i32),
            "b200norm_testing_plan_group": ([i64, i64, i64, i64, i32, i32, i32, i32, i32,
                                             ctypes.POINTER(ctypes.c_int64)], i32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def _check(status: int) -> None:
    if status != 0:
        lib = library()
        name = lib.b200norm_status_string(status).decode()
        detail = lib.b200norm_last_error().decode()
        raise B200NormError(status, name, detail)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _of_device(stream, index):
    """The caller's stream, of the device of that index."""
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    return stream


def _torch_stream(device, stream):
    if stream is None:
        return torch.cuda.current_stream(device)
    index = torch.device(device).index  # None: "cuda", the current device
    return stream if index is None else _of_device(stream, index)


def _stream(device, stream):
    return ctypes.c_void_p(_torch_stream(device, stream).cuda_stream)


def _cuda(name, t, device=None, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device}); there is no CPU path")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name}: only float32, float16 and bfloat16 are supported "
                        f"(got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _out(name, t, like, dtype=None):
    if t is None:
        return torch.empty(like.shape, dtype=dtype or like.dtype, device=like.device)
    _cuda(name, t, like.device, dtype or like.dtype)
    if t.numel() != like.numel():
        raise ValueError(f"{name} must have {like.numel()} elements")
    return t


# ---------------------------------------------------------------------------
# SkipSimplifiedLayerNormalization
# ---------------------------------------------------------------------------

def _skip_rms(input, skip, gamma, bias, epsilon, want_sum, output, sum_out, stats, stream):
    x = _cuda("input", input)
    dev, dt = x.device, x.dtype
    _cuda("skip", skip, dev, dt)
    _cuda("gamma", gamma, dev, dt)
    if bias is not None:
        _cuda("bias", bias, dev, dt)
    if x.dim() < 1 or skip.shape != x.shape:
        raise ValueError("skip must have input's shape")
    hidden = x.shape[-1]
    rows = x.numel() // hidden if hidden else 0
    if gamma.numel() != hidden or (bias is not None and bias.numel() != hidden):
        raise ValueError("gamma and bias must have hidden_size elements")
    y = _out("output", output, x)
    s = _out("input_skip_bias_sum", sum_out, x) if want_sum or sum_out is not None else None
    st = _stream(dev, stream)
    lib = library()
    if stats:
        stat_shape = tuple(x.shape[:-1]) + (1,)
        mean = torch.empty(stat_shape, dtype=torch.float32, device=dev)
        inv = torch.empty(stat_shape, dtype=torch.float32, device=dev)
        _check(lib.b200norm_skip_rms_stats(_ptr(x), _ptr(skip), _ptr(gamma), _ptr(bias), _ptr(y),
                                           _ptr(s), _ptr(mean), _ptr(inv), rows, hidden,
                                           _DTYPES[dt], float(epsilon), st))
        return y, s, mean, inv
    _check(lib.b200norm_skip_rms(_ptr(x), _ptr(skip), _ptr(gamma), _ptr(bias), _ptr(y), _ptr(s),
                                 rows, hidden, _DTYPES[dt], float(epsilon), st))
    return y, s


def skip_rms(input, skip, gamma, bias=None, *, epsilon=SSLN_EPS_DEFAULT, want_sum=True,
             output=None, sum_out=None, stream=None):
    """SkipSimplifiedLayerNormalization over the last axis of ``input``.

    Returns ``(output, input_skip_bias_sum)``; the second is ``None`` unless
    ``want_sum`` (default True) or ``sum_out`` is given.
    """
    return _skip_rms(input, skip, gamma, bias, epsilon, want_sum, output, sum_out, False, stream)


def skip_rms_stats(input, skip, gamma, bias=None, *, epsilon=SSLN_EPS_DEFAULT, want_sum=True,
                   output=None, sum_out=None, stream=None):
    """As :func:`skip_rms`, also returning the float32 ``mean`` (zeros) and
    ``inv_std_var`` outputs of shape ``input.shape[:-1] + (1,)``."""
    return _skip_rms(input, skip, gamma, bias, epsilon, want_sum, output, sum_out, True, stream)


# ---------------------------------------------------------------------------
# GatedRMSNorm
# ---------------------------------------------------------------------------

def gated_rms(x, gate, scale, *, epsilon=1e-5, y=None, stream=None):
    """GatedRMSNorm: RMS-normalize each contiguous span of ``C = scale.numel()``
    elements of ``x``, times ``scale`` times SiLU(``gate``)."""
    x = _cuda("X", x)
    _cuda("gate", gate, x.device, x.dtype)
    _cuda("scale", scale, x.device, x.dtype)
    if gate.shape != x.shape:
        raise ValueError("gate must have X's shape")
    if x.dim() < 1:
        raise ValueError("X must have rank >= 1")
    C = scale.numel()
    out = _out("Y", y, x)
    _check(library().b200norm_gated_rms(_ptr(x), _ptr(gate), _ptr(scale), _ptr(out), x.numel(),
                                        C, _DTYPES[x.dtype], float(epsilon),
                                        _stream(x.device, stream)))
    return out


# ---------------------------------------------------------------------------
# SkipGroupNorm
# ---------------------------------------------------------------------------

_workspaces = {}
_ws_lock = threading.Lock()


def rows_status(stream=None, device=None):
    """Synchronizes ``stream`` and raises B200NormError if a pipelined row
    kernel (short SkipSimplifiedLayerNormalization / GatedRMSNorm rows, or the
    gradient of layer normalization) on the device gave up a bounded wait
    since the last call; the record is then cleared."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        _check(library().b200norm_rows_status(_stream(dev, stream)))


def noalloc_status(stream=None, device=None):
    """Synchronizes ``stream`` and raises B200NormError if a bounded
    device-side wait of an allocation-free SkipGroupNorm call
    (``b200norm_skip_group_noalloc``) on the device gave up since the last
    call; the record is then cleared."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        _check(library().b200norm_skip_group_noalloc_status(_stream(dev, stream)))


def workspace_size(N, C, H, W, groups, dtype=torch.float16, channels_last=1) -> int:
    return int(library().b200norm_skip_group_workspace_size(N, C, H, W, groups, _DTYPES[dtype],
                                                            1 if channels_last else 0))


def workspace_init(ws, stream=None):
    _check(library().b200norm_workspace_init(_ptr(ws), ws.numel(), _stream(ws.device, stream)))


def workspace_status(ws, stream=None):
    """Synchronizes ``stream`` and raises B200NormError if a device-side wait
    recorded a timeout in ``ws``."""
    _check(library().b200norm_workspace_status(_ptr(ws), _stream(ws.device, stream)))


def _workspace_for(device, stream, nbytes):
    """A zero-filled workspace cached per (device, stream); calls on one
    stream are serialized, so they may share it.  It is allocated and zeroed
    on that stream, so the clear is ordered before the kernels that use it,
    and a smaller one it replaces goes back to the caching allocator on the
    stream its kernels ran on (its allocation stream)."""
    key = (device.index, stream.cuda_stream)
    with _ws_lock:
        ws = _workspaces.get(key)
        if ws is None or ws.numel() < nbytes:
            with torch.cuda.stream(stream):
                ws = torch.zeros(max(nbytes, 1 << 16), dtype=torch.uint8, device=device)
            _workspaces[key] = ws
        return ws


def skip_group(x, skip, gamma, beta, bias=None, *, groups, activation, epsilon=1e-5,
               channels_last=1, want_sum=False, y=None, s=None, workspace=None, stream=None):
    """SkipGroupNorm.  ``x`` is (N, H, W, C) when ``channels_last`` is non-zero
    (the default), else (N, C, H, W).  ``skip`` is x's shape, (N, C) or
    (N, 1, 1, C).  ``groups`` and ``activation`` (0 none, 1 SiLU) are required.
    Returns ``(Y, S)``; ``S`` is ``None`` unless ``want_sum`` or ``s`` is given.
    """
    x = _cuda("X", x)
    dev, dt = x.device, x.dtype
    if x.dim() != 4:
        raise ValueError("X must be rank 4")
    _cuda("skip", skip, dev, dt)
    _cuda("gamma", gamma, dev)
    _cuda("beta", beta, dev, gamma.dtype)
    if bias is not None:
        _cuda("bias", bias, dev, dt)
    cl = 1 if channels_last else 0
    if cl:
        N, H, W, C = x.shape
    else:
        N, C, H, W = x.shape
    if gamma.numel() != C or beta.numel() != C or (bias is not None and bias.numel() != C):
        raise ValueError("gamma, beta and bias must have C elements")
    out = _out("Y", y, x)
    ssum = _out("S", s, x) if want_sum or s is not None else None
    tst = _torch_stream(dev, stream)
    st = ctypes.c_void_p(tst.cuda_stream)
    nbytes = workspace_size(N, C, H, W, groups, dt, cl)
    if workspace is None:
        workspace = _workspace_for(dev, tst, nbytes)
    if skip.dim() > 4:
        raise ValueError("skip must have X's shape, (N, C) or (N, 1, 1, C)")
    dims = (ctypes.c_int64 * 4)(*([int(d) for d in skip.shape] + [0] * (4 - skip.dim())))
    _check(library().b200norm_skip_group(
        _ptr(x), _ptr(skip), skip.dim(), dims, _ptr(bias), _ptr(gamma), _ptr(beta), _ptr(out),
        _ptr(ssum), N, C, H, W, _DTYPES[dt], _DTYPES[gamma.dtype], int(groups), float(epsilon),
        int(activation), cl, _ptr(workspace), workspace.numel(), st))
    return out, ssum


# ---------------------------------------------------------------------------
# Layer normalization and the linear operator
# ---------------------------------------------------------------------------

# Activation codes of linear / linear_grad.
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}

# A call of one token is over in a few microseconds on the GPU, so these
# bindings keep the host's part short: pointers pass as plain integers, a tensor
# is checked with one expression, and only a failed check asks what was wrong.


def _first(name, t):
    """(index of its device, type) of a call's first tensor."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()
            and t.dtype in _DTYPES):
        _cuda(name, t)
    return t.get_device(), t.dtype


def _is(name, t, shape, x, index, dtype):
    """``t``, contiguous on x's device (of that index) with that type and shape
    (None: any)."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        return t
    _cuda(name, t, x.device, dtype)
    raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")


def _vector(name, t, n, x, index, dtype):
    _is(name, t, None, x, index, dtype)
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements")
    return t


def _weights(name, t, n, x, index):
    """gamma / beta: x's type or float32."""
    if not isinstance(t, torch.Tensor) or t.dtype not in (x.dtype, torch.float32):
        _cuda(name, t, x.device)
        raise TypeError(f"{name} must be {x.dtype} or torch.float32 (got {t.dtype})")
    return _vector(name, t, n, x, index, t.dtype)


def _at(t):
    return None if t is None else t.data_ptr()


def _raw_stream(index, stream):
    return (torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)


def _on(index, stream, tensors):
    """None, or the context to allocate and launch in.  With a stream of the
    caller's own, outputs and scratch are allocated on it, and the caller's
    tensors (inputs, outputs and workspace) are kept from reuse until it has
    passed this call."""
    if stream is not None:
        _of_device(stream, index)
        for t in tensors:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
        return torch.cuda.stream(stream)
    if index != torch._C._cuda_getDevice():
        return torch.cuda.device(index)
    return None


# Small scratch blocks kept per thread, device and stream: a thread's work on one
# stream is in order, so its calls may share one (the launches of two threads'
# calls on a stream may interleave).  A block that is outgrown goes back to the
# caching allocator, in that stream's order.  Streams that torch did not make get
# blocks of the caching allocator's call by call: such a stream may be destroyed, and
# its handle come back for another while its work still runs.
_SCRATCH_KEPT = 32 << 20
_scratch_of_thread = threading.local()


def _from_torch(index, stream):
    """Whether the current stream, of that handle, is one of torch's own, which live as
    long as the process: the others' ids are their handles."""
    return stream == 0 or torch._C._cuda_getCurrentStream(index)[0] != stream


def _scratch(workspace, nbytes, x, index, stream):
    """Workspace arguments: the caller's, or a kept or new block.  A call that is
    being captured into a graph gets a block of the graph's own, which lives as
    long as the graph replays."""
    if workspace is not None:
        if workspace.device != x.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {x.device}")
        return workspace, workspace.numel() * workspace.element_size()
    if not nbytes:
        return None, 0
    if (nbytes > _SCRATCH_KEPT or not _from_torch(index, stream)
            or torch.cuda.is_current_stream_capturing()):
        return torch.empty(nbytes, dtype=torch.uint8, device=x.device), nbytes
    blocks = getattr(_scratch_of_thread, "blocks", None)
    if blocks is None:
        blocks = _scratch_of_thread.blocks = {}
    block = blocks.get((index, stream))
    if block is None or block.numel() < nbytes:
        block = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=x.device)
        blocks[(index, stream)] = block
    return block, block.numel()


def _like(name, t, x, index):
    """An output of x's shape and type: the caller's, or a new one."""
    return torch.empty_like(x) if t is None else _is(name, t, x.shape, x, index, x.dtype)


def _new(name, t, shape, x, index):
    """An output of x's type and another shape."""
    if t is not None:
        return _is(name, t, shape, x, index, x.dtype)
    return torch.empty(shape, dtype=x.dtype, device=x.device)


def _last_axis(name, t):
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} needs a last axis of at least one element")
    return t.shape[-1]


def _skip_layer(x, skip, gamma, beta, bias, epsilon, want_sum, output, sum_out, stats, stream):
    index, dt = _first("input", x)
    hidden = _last_axis("input", x)
    _weights("gamma", gamma, hidden, x, index)
    if beta is not None:
        _vector("beta", beta, hidden, x, index, gamma.dtype)
    if skip is not None:
        _is("skip", skip, x.shape, x, index, dt)
    elif bias is not None or sum_out is not None:
        raise ValueError("bias and sum_out need a skip (S is the input without one)")
    if bias is not None:
        _vector("bias", bias, hidden, x, index, dt)

    def run():
        y = _like("output", output, x, index)
        s = None
        if skip is not None and (want_sum or sum_out is not None):
            s = _like("input_skip_bias_sum", sum_out, x, index)
        mean = inv = None
        if stats:
            mean = torch.empty(x.shape[:-1] + (1,), dtype=torch.float32, device=x.device)
            inv = torch.empty_like(mean)
        _check((_lib or library()).b200norm_skip_layer(
            x.data_ptr(), _at(skip), gamma.data_ptr(), _at(beta), _at(bias), y.data_ptr(), _at(s),
            _at(mean), _at(inv), x.numel() // hidden, hidden, _DTYPES[dt], _DTYPES[gamma.dtype],
            float(epsilon), _raw_stream(index, stream)))
        return y, (x if skip is None and want_sum else s), mean, inv

    context = _on(index, stream, (x, skip, gamma, beta, bias, output, sum_out))
    if context is None:
        return run()
    with context:
        return run()


def skip_layer(input, skip, gamma, beta=None, bias=None, *, epsilon=1e-5, want_sum=True,
               output=None, sum_out=None, stream=None):
    """Layer normalization of ``S = (input + skip) + bias`` over the last axis,
    times ``gamma`` plus ``beta`` (both of ``input``'s type or both float32).  No
    autograd graph is made, whatever requires gradients (as of every entry here).

    ``skip=None`` normalizes ``input`` itself.  Returns ``(output, S)``; ``S`` is
    ``None`` unless ``want_sum`` (default True) or ``sum_out`` is given, and is
    ``input`` itself without a skip.
    """
    return _skip_layer(input, skip, gamma, beta, bias, epsilon, want_sum, output, sum_out, False,
                       stream)[:2]


def skip_layer_stats(input, skip, gamma, beta=None, bias=None, *, epsilon=1e-5, want_sum=True,
                     output=None, sum_out=None, stream=None):
    """As :func:`skip_layer`, also returning the float32 ``mean`` and
    ``inv_std_var`` of shape ``input.shape[:-1] + (1,)`` that
    :func:`skip_layer_grad` takes."""
    return _skip_layer(input, skip, gamma, beta, bias, epsilon, want_sum, output, sum_out, True,
                       stream)


def skip_layer_grad(dy, s, mean, inv_std_var, gamma, *, ds=None, want_input=True,
                    want_gamma=True, want_beta=True, want_bias=False, dx=None, dgamma=None,
                    dbeta=None, dbias=None, workspace=None, stream=None):
    """Gradients of :func:`skip_layer`: ``(dx, dgamma, dbeta, dbias)``.

    ``s``, ``mean`` and ``inv_std_var`` are the forward call's; ``ds`` is the
    gradient that reaches S by other paths.  ``dx`` is the gradient of S, which
    is that of both ``input`` and ``skip``.  An output that is not wanted is
    ``None``; one that is given is wanted.
    """
    index, dt = _first("dy", dy)
    hidden = _last_axis("dy", dy)
    rows = dy.numel() // hidden
    _is("s", s, dy.shape, dy, index, dt)
    _weights("gamma", gamma, hidden, dy, index)
    _vector("mean", mean, rows, dy, index, torch.float32)
    _vector("inv_std_var", inv_std_var, rows, dy, index, torch.float32)
    if ds is not None:
        _is("ds", ds, dy.shape, dy, index, dt)

    def run():
        lib = _lib or library()
        outs = (
            _like("dx", dx, dy, index) if want_input or dx is not None else None,
            _like("dgamma", dgamma, gamma, index) if want_gamma or dgamma is not None else None,
            _like("dbeta", dbeta, gamma, index) if want_beta or dbeta is not None else None,
            _new("dbias", dbias, gamma.shape, dy, index) if want_bias or dbias is not None
            else None)
        need = lib.b200norm_skip_layer_grad_workspace_size(rows, hidden) if rows else 0
        raw = _raw_stream(index, stream)
        ws, n = _scratch(workspace, need, dy, index, raw)
        _check(lib.b200norm_skip_layer_grad(
            dy.data_ptr(), s.data_ptr(), mean.data_ptr(), inv_std_var.data_ptr(),
            gamma.data_ptr(), _at(ds), *map(_at, outs), rows, hidden, _DTYPES[dt],
            _DTYPES[gamma.dtype], _at(ws), n, raw))
        return outs

    context = _on(index, stream, (dy, s, mean, inv_std_var, gamma, ds, dx, dgamma, dbeta, dbias,
                                  workspace))
    if context is None:
        return run()
    with context:
        return run()


def _weight(weight, x, index, dtype):
    _is("weight", weight, None, x, index, dtype)
    if weight.dim() != 2 or weight.numel() == 0:
        raise ValueError("weight must be (out_features, in_features), neither zero")
    return weight.shape


def linear(x, weight, bias=None, residual=None, *, activation=0, want_z=False, y=None, z=None,
           workspace=None, stream=None):
    """``act(x @ weight.T + bias) + residual`` over the last axis of ``x``;
    ``weight`` is (out_features, in_features), ``activation`` a code of
    ``ACTIVATIONS``.  No autograd graph is made.

    Returns ``(y, z)``; ``z``, the value before the activation that
    :func:`linear_grad` takes, is ``None`` unless ``want_z`` or ``z`` is given.
    """
    index, dt = _first("x", x)
    activation = int(activation)
    n_out, n_in = _weight(weight, x, index, dt)
    if _last_axis("x", x) != n_in:
        raise ValueError(f"x's last axis must have weight's in_features ({n_in})")
    rows = x.numel() // n_in
    shape = x.shape[:-1] + (n_out,)
    if bias is not None:
        _vector("bias", bias, n_out, x, index, dt)
    if residual is not None:
        _is("residual", residual, shape, x, index, dt)

    def run():
        lib = _lib or library()
        yv = _new("y", y, shape, x, index)
        zv = _like("z", z, yv, index) if want_z or z is not None else None
        px, pw, code = x.data_ptr(), weight.data_ptr(), _DTYPES[dt]
        need = lib.b200norm_linear_workspace_size(rows, n_in, n_out, code, (px | pw) % 16 == 0)
        raw = _raw_stream(index, stream)
        ws, n = _scratch(workspace, need, x, index, raw)
        _check(lib.b200norm_linear(px, pw, _at(bias), _at(residual), yv.data_ptr(), _at(zv), rows,
                                   n_in, n_out, code, activation, _at(ws), n, raw))
        return yv, zv

    context = _on(index, stream, (x, weight, bias, residual, y, z, workspace))
    if context is None:
        return run()
    with context:
        return run()


def linear_grad(dy, x, weight, z=None, *, activation=0, want_input=True, want_weight=True,
                want_bias=True, dx=None, dw=None, db=None, workspace=None, stream=None):
    """Gradients of :func:`linear`: ``(dx, dw, db)`` (that of ``residual`` is
    ``dy``).  ``z`` is the forward call's, needed with an activation.  An output
    that is not wanted is ``None``; one that is given is wanted.
    """
    index, dt = _first("dy", dy)
    activation = int(activation)
    n_out, n_in = _weight(weight, dy, index, dt)
    if _last_axis("dy", dy) != n_out:
        raise ValueError(f"dy's last axis must have weight's out_features ({n_out})")
    rows = dy.numel() // n_out
    in_shape = dy.shape[:-1] + (n_in,)
    _is("x", x, in_shape, dy, index, dt)
    if activation:
        if z is None:
            raise ValueError("z is needed with an activation")
        _is("z", z, dy.shape, dy, index, dt)
    else:
        z = None

    def run():
        lib = _lib or library()
        dxv = _like("dx", dx, x, index) if want_input or dx is not None else None
        dwv = _like("dw", dw, weight, index) if want_weight or dw is not None else None
        dbv = _new("db", db, (n_out,), dy, index) if want_bias or db is not None else None
        pd, px, pw, code = dy.data_ptr(), x.data_ptr(), weight.data_ptr(), _DTYPES[dt]
        aligned = (pd | (px if dwv is not None else 0) | (pw if dxv is not None else 0)) % 16 == 0
        need = lib.b200norm_linear_grad_workspace_size(rows, n_in, n_out, code, activation,
                                                       aligned)
        raw = _raw_stream(index, stream)
        ws, n = _scratch(workspace, need, dy, index, raw)
        _check(lib.b200norm_linear_grad(pd, px, pw, _at(z), _at(dxv), _at(dwv), _at(dbv), rows,
                                        n_in, n_out, code, activation, _at(ws), n, raw))
        return dxv, dwv, dbv

    context = _on(index, stream, (dy, x, weight, z, dx, dw, db, workspace))
    if context is None:
        return run()
    with context:
        return run()


def _gated_weight(weight, x, index, dtype):
    n, n_in = _weight(weight, x, index, dtype)
    if n % 2:
        raise ValueError("weight must have as many rows for the gate as for what it gates")
    return n // 2, n_in


def gated_linear(x, weight, bias=None, *, activation=1, want_z=False, h=None, z=None,
                 workspace=None, stream=None):
    """``act(x @ gate.T + b_gate) * (x @ up.T + b_up)`` over the last axis of ``x``;
    ``weight`` is (2 out_features, in_features), the rows of ``gate`` before those of
    ``up``, and ``bias`` in the same order.  ``activation`` is a code of
    ``ACTIVATIONS`` (SiLU by default).  No autograd graph is made.

    Returns ``(h, z)``; ``z`` (..., 2 out_features), both products as
    :func:`gated_linear_grad` takes them, is ``None`` unless ``want_z`` or ``z`` is
    given.
    """
    index, dt = _first("x", x)
    activation = int(activation)
    n_out, n_in = _gated_weight(weight, x, index, dt)
    if _last_axis("x", x) != n_in:
        raise ValueError(f"x's last axis must have weight's in_features ({n_in})")
    rows = x.numel() // n_in
    lead = x.shape[:-1]
    if bias is not None:
        _vector("bias", bias, 2 * n_out, x, index, dt)

    def run():
        lib = _lib or library()
        hv = _new("h", h, lead + (n_out,), x, index)
        zv = _new("z", z, lead + (2 * n_out,), x, index) if want_z or z is not None else None
        px, pw, code = x.data_ptr(), weight.data_ptr(), _DTYPES[dt]
        need = lib.b200norm_gated_linear_workspace_size(rows, n_in, n_out, code,
                                                        (px | pw) % 16 == 0)
        raw = _raw_stream(index, stream)
        ws, n = _scratch(workspace, need, x, index, raw)
        _check(lib.b200norm_gated_linear(px, pw, _at(bias), hv.data_ptr(), _at(zv), rows, n_in,
                                         n_out, code, activation, _at(ws), n, raw))
        return hv, zv

    context = _on(index, stream, (x, weight, bias, h, z, workspace))
    if context is None:
        return run()
    with context:
        return run()


def gated_linear_grad(dh, x, weight, z, *, activation=1, want_input=True, want_weight=True,
                      want_bias=True, dx=None, dw=None, db=None, workspace=None, stream=None):
    """Gradients of :func:`gated_linear`: ``(dx, dw, db)``, the latter two in the order of
    ``weight``'s rows.  ``z`` is the forward call's.  An output that is not wanted is
    ``None``; one that is given is wanted.
    """
    index, dt = _first("dh", dh)
    activation = int(activation)
    n_out, n_in = _gated_weight(weight, dh, index, dt)
    if _last_axis("dh", dh) != n_out:
        raise ValueError(f"dh's last axis must have half of weight's rows ({n_out})")
    rows = dh.numel() // n_out
    _is("x", x, dh.shape[:-1] + (n_in,), dh, index, dt)
    _is("z", z, dh.shape[:-1] + (2 * n_out,), dh, index, dt)

    def run():
        lib = _lib or library()
        dxv = _like("dx", dx, x, index) if want_input or dx is not None else None
        dwv = _like("dw", dw, weight, index) if want_weight or dw is not None else None
        dbv = _new("db", db, (2 * n_out,), dh, index) if want_bias or db is not None else None
        px, pw, code = x.data_ptr(), weight.data_ptr(), _DTYPES[dt]
        aligned = ((px if dwv is not None else 0) | (pw if dxv is not None else 0)) % 16 == 0
        need = lib.b200norm_gated_linear_grad_workspace_size(rows, n_in, n_out, code, aligned)
        raw = _raw_stream(index, stream)
        ws, n = _scratch(workspace, need, dh, index, raw)
        _check(lib.b200norm_gated_linear_grad(dh.data_ptr(), px, pw, z.data_ptr(), _at(dxv),
                                              _at(dwv), _at(dbv), rows, n_in, n_out, code,
                                              activation, _at(ws), n, raw))
        return dxv, dwv, dbv

    context = _on(index, stream, (dh, x, weight, z, dx, dw, db, workspace))
    if context is None:
        return run()
    with context:
        return run()


def linear_status(stream=None, device=None):
    """Synchronizes ``stream`` and raises B200NormError if a bounded wait of a
    kernel of ``linear``, ``gated_linear`` or their gradients on the device gave up
    since the last call; the record is then cleared."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        _check(library().b200norm_linear_status(_stream(dev, stream)))


# ---------------------------------------------------------------------------
# Query and key heads
# ---------------------------------------------------------------------------

# Codes of rotary_frequencies.
ROTARY_SCALINGS = {"none": 0, "linear": 1, "base": 2, "turns": 3}

# The C structs b200norm_rotation, b200norm_heads and b200norm_heads_grad.
_ROTATION = struct.Struct("@PiqqPqif")
_HEADS = struct.Struct("@PPPq6q")
_HEADS_GRAD = struct.Struct("@PPPPPq9q")
_NO_STRIDES = (0, 0, 0)


def rotary_frequencies(rotary_size, base=10000.0, *, scaling=0, factor=1.0, original_length=0.0,
                       low=1.0, high=32.0, device="cuda"):
    """Frequencies ``base ** (-2 i / rotary_size)`` of a rotation's pairs, in
    radians per position: float64 on ``device``, as :func:`rotary` takes them.

    ``scaling``, a code of ``ROTARY_SCALINGS``, is for contexts ``factor`` times
    longer than the ``original_length`` a model was trained on: "linear" divides
    all by ``factor``; "base" raises the base so that the lowest is divided by it
    and the highest kept; "turns" keeps those that turn ``high`` times or more over
    the original length, divides those that turn ``low`` times or less, and mixes
    the others in proportion.  (A ``scale`` of ``0.1 * log(factor) + 1`` in the
    rotation goes with it where a model wants that.)
    """
    n = int(rotary_size)
    out = (ctypes.c_double * max(1, n // 2))()
    _check((_lib or library()).b200norm_rotary_frequencies(
        out, n, float(base), int(scaling), float(factor), float(original_length), float(low),
        float(high)))
    return torch.tensor(list(out), dtype=torch.float64).to(device)


def _heads(name, t, lead, size, index, dtype):
    """(heads, their steps): of ``t``, heads of that leading shape and size, with any steps
    between them."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index:
        shape, st = t.shape, t.stride()
        if len(lead) == 2:
            if (len(shape) == 4 and shape[3] == size and shape[0] == lead[0]
                    and shape[1] == lead[1] and (st[3] == 1 or size == 1)):
                return shape[2], st[0], st[1], st[2]
        elif (len(shape) == 3 and shape[2] == size and shape[0] == lead[0]
              and (st[2] == 1 or size == 1)):
            return shape[1], 0, st[0], st[1]
        if shape[:-2] == lead and shape[-1] == size:
            raise ValueError(f"{name}'s elements must be next to one another in a head")
        raise ValueError(f"{name} must have shape {tuple(lead)} + (heads, {size}) "
                         f"(got {tuple(shape)})")
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in _DTYPES:
        if t.dtype is not dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    _cuda(name, t)
    raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _heads_like(name, t, lead, size, heads, index, dtype):
    """The steps of ``t``, with that many heads."""
    n, *steps = _heads(name, t, lead, size, index, dtype)
    if n != heads:
        raise ValueError(f"{name} must have {heads} heads (got {n})")
    return steps


def _new_heads(lead, heads, size, x, dtype):
    """New heads, dense, and their steps."""
    t = torch.empty((*lead, heads, size), dtype=dtype, device=x.device)
    row = heads * size
    return t, (lead[1] * row if len(lead) == 2 else 0, row, size)


def _rotation(positions, inv_freq, lead, index, interleaved, scale):
    """The C rotation."""
    if inv_freq is None:
        if positions is not None:
            raise ValueError("positions need inv_freq")
        return _ROTATION.pack(0, 8, 0, 0, 0, 0, 1 if interleaved else 0, scale)
    if not (isinstance(inv_freq, torch.Tensor) and inv_freq.dtype is torch.float64):
        raise TypeError("inv_freq must be a float64 torch.Tensor")
    if inv_freq.get_device() != index or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be contiguous, of one axis, on cuda:{index}")
    wide = isinstance(positions, torch.Tensor) and positions.dtype is torch.int64
    if not wide and not (isinstance(positions, torch.Tensor) and positions.dtype is torch.int32):
        raise TypeError("positions must be an int64 or int32 torch.Tensor")
    if positions.get_device() != index:
        raise ValueError(f"positions is on {positions.device}, expected cuda:{index}")
    shape, st = positions.shape, positions.stride()
    if shape == lead:
        b, s = st if len(st) == 2 else (0, st[0])
    elif len(lead) == 2 and shape == lead[1:]:
        b, s = 0, st[0]
    else:
        raise ValueError(f"positions must have shape {tuple(lead)}"
                         + (f" or {tuple(lead[1:])}" if len(lead) == 2 else "")
                         + f" (got {tuple(shape)})")
    return _ROTATION.pack(positions.data_ptr(), 8 if wide else 4, b, s, inv_freq.data_ptr(),
                          2 * inv_freq.numel(), 1 if interleaved else 0, scale)


def _first_heads(q, k):
    """(queries, or keys without them; their leading shape and size, device index, type)."""
    x, name = (q, "q") if q is not None else (k, "k")
    if x is None:
        raise ValueError("queries or keys are needed")
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype in _DTYPES):
        _cuda(name, x)
    shape = x.shape
    if len(shape) not in (3, 4) or shape[-1] < 1:
        raise ValueError(f"{name} must have shape (..., heads, head_size) with one or two leading "
                         f"axes (got {tuple(shape)})")
    return x, shape[:-2], shape[-1], x.get_device(), x.dtype


def _gammas(q, gamma_q, k, gamma_k, size, x, index):
    """The type of both gammas (x's without any)."""
    if gamma_q is not None and gamma_k is not None and q is not None and k is not None:
        _weights("gamma_q", gamma_q, size, x, index)
        _weights("gamma_k", gamma_k, size, x, index)
        if gamma_q.dtype is not gamma_k.dtype:
            raise TypeError("gamma_q and gamma_k must be of one type")
        return gamma_q.dtype
    m = None
    for name, heads, gamma in (("gamma_q", q, gamma_q), ("gamma_k", k, gamma_k)):
        if gamma is None:
            continue
        if heads is None:
            raise ValueError(f"{name} needs its heads")
        _weights(name, gamma, size, x, index)
        if m is not None and gamma.dtype is not m:
            raise TypeError("gamma_q and gamma_k must be of one type")
        m = gamma.dtype
    return m or x.dtype


def _rotated(norm, q, k, gamma_q, gamma_k, positions, inv_freq, epsilon, interleaved, inverse,
             scale, q_out, k_out, stream):
    x, lead, size, index, dt = _first_heads(q, k)
    q_at = k_at = qo_at = ko_at = None
    if q is not None:
        q_at = _heads("q", q, lead, size, index, dt)
    if k is not None:
        k_at = _heads("k", k, lead, size, index, dt)
    if q_out is not None:
        if q is None:
            raise ValueError("q_out needs q")
        qo_at = _heads_like("q_out", q_out, lead, size, q_at[0], index, dt)
    if k_out is not None:
        if k is None:
            raise ValueError("k_out needs k")
        ko_at = _heads_like("k_out", k_out, lead, size, k_at[0], index, dt)
    m = _gammas(q, gamma_q, k, gamma_k, size, x, index) if norm else dt
    rotation = _rotation(positions, inv_freq, lead, index, interleaved, scale)

    def run():
        a = b = None
        qo, ko, qs, ks = q_out, k_out, qo_at, ko_at
        if q is not None:
            if qo is None:
                qo, qs = _new_heads(lead, q_at[0], size, x, dt)
            a = _HEADS.pack(q.data_ptr(), qo.data_ptr(),
                            0 if gamma_q is None else gamma_q.data_ptr(), *q_at, *qs)
        if k is not None:
            if ko is None:
                ko, ks = _new_heads(lead, k_at[0], size, x, dt)
            b = _HEADS.pack(k.data_ptr(), ko.data_ptr(),
                            0 if gamma_k is None else gamma_k.data_ptr(), *k_at, *ks)
        batch, seq = lead if len(lead) == 2 else (1, lead[0])
        if norm:
            _check((_lib or library()).b200norm_head_rms_rotary(
                a, b, rotation, batch, seq, size, _DTYPES[dt], _DTYPES[m], float(epsilon),
                _raw_stream(index, stream)))
        else:
            _check((_lib or library()).b200norm_rotary(
                a, b, rotation, batch, seq, size, _DTYPES[dt], 1 if inverse else 0,
                _raw_stream(index, stream)))
        return qo, ko

    context = _on(index, stream, (q, k, gamma_q, gamma_k, positions, inv_freq, q_out, k_out))
    if context is None:
        return run()
    with context:
        return run()


def rotary(q, k, positions, inv_freq, *, interleaved=False, scale=1.0, inverse=False, q_out=None,
           k_out=None, stream=None):
    """Rotate the heads of ``q`` and ``k`` by their tokens' positions, or back
    (``inverse``: the gradient of the rotation).  Returns ``(q, k)``, rotated.

    ``q`` and ``k`` are (tokens, heads, head_size) or (batch, seq, heads,
    head_size), of one type; either may be ``None``.  Only a head's elements need
    be next to one another: views of a product's rows, or of permuted tensors, are
    taken as they are.  ``positions``, int64 or int32 of any sign, has the tokens'
    shape, or (seq,).  ``inv_freq`` holds a frequency (radians per position,
    float64) for each pair: elements (i, i + n) of the first 2 n = 2
    ``inv_freq.numel()``, or (2 i, 2 i + 1) when ``interleaved``; the others stay
    as they are.  ``scale`` multiplies the rotated elements.  ``q_out`` may be
    ``q`` itself, and ``k_out`` ``k``.
    """
    return _rotated(False, q, k, None, None, positions, inv_freq, 0.0, interleaved, inverse, scale,
                    q_out, k_out, stream)


def head_rms_rotary(q, k, gamma_q, gamma_k, positions, inv_freq, *, epsilon=1e-6,
                    interleaved=False, scale=1.0, q_out=None, k_out=None, stream=None):
    """RMS-normalize each head of ``q`` and ``k``, ``x / sqrt(mean(x^2) + epsilon) *
    gamma``, then rotate it as :func:`rotary` does.  Returns ``(q, k)``.

    ``gamma_q`` and ``gamma_k`` have head_size elements of the heads' type or
    float32; ``None`` is ones.  ``positions=None, inv_freq=None`` leaves out the
    rotation.
    """
    return _rotated(True, q, k, gamma_q, gamma_k, positions, inv_freq, epsilon, interleaved, False,
                    scale, q_out, k_out, stream)


def head_rms_rotary_grad(dq, dk, q, k, gamma_q, gamma_k, positions, inv_freq, *, epsilon=1e-6,
                         interleaved=False, scale=1.0, want_input=True, want_gamma=True,
                         dq_out=None, dk_out=None, dgamma_q=None, dgamma_k=None, workspace=None,
                         stream=None):
    """Gradients of :func:`head_rms_rotary`: ``(dq, dk, dgamma_q, dgamma_k)``.

    ``dq`` and ``dk`` are the gradients of its results, ``q`` and ``k`` its inputs.
    ``dq_out`` and ``dk_out`` receive those of the inputs (views of one tensor of
    rows, for the gradient of the product they came from).  An output that is not
    wanted is ``None``; one that is given is wanted; a gamma of ``None`` has no
    gradient.  Without tokens or heads a gamma's gradient is zeros.
    """
    x, lead, size, index, dt = _first_heads(q, k)
    sets = []
    for name, t, d, gamma, o, dg in (("q", q, dq, gamma_q, dq_out, dgamma_q),
                                     ("k", k, dk, gamma_k, dk_out, dgamma_k)):
        if t is None:
            if not (d is None and o is None and dg is None):
                raise ValueError(f"d{name}, d{name}_out and dgamma_{name} need {name}")
            sets.append(None)
            continue
        if dg is not None and gamma is None:
            raise ValueError(f"dgamma_{name} needs gamma_{name}")
        t_at = _heads(name, t, lead, size, index, dt)
        d_at = _heads_like("d" + name, d, lead, size, t_at[0], index, dt)
        o_at = _NO_STRIDES if o is None else _heads_like(f"d{name}_out", o, lead, size, t_at[0],
                                                         index, dt)
        sets.append((name, t, d, gamma, o, dg, t_at, d_at, o_at))
    m = _gammas(q, gamma_q, k, gamma_k, size, x, index)
    rotation = _rotation(positions, inv_freq, lead, index, interleaved, scale)

    def run():
        lib = _lib or library()
        dxs, dgs, args, heads = [None, None], [None, None], [None, None], [0, 0]
        empty = [None, None]  # no heads, whose sum the call for the others does not store
        for i, one in enumerate(sets):
            if one is None:
                continue
            name, t, d, gamma, o, dg, t_at, d_at, o_at = one
            if o is None and want_input:
                o, o_at = _new_heads(lead, t_at[0], size, x, dt)
            if gamma is not None and (dg is not None or want_gamma):
                dg = _like("dgamma_" + name, dg, gamma, index)
            dxs[i], dgs[i], heads[i] = o, dg, t_at[0]
            if t_at[0] == 0 and dg is not None:
                empty[i] = _HEADS_GRAD.pack(0, 0, 0, 0, dg.data_ptr(), 1, *_NO_STRIDES,
                                            *_NO_STRIDES, *_NO_STRIDES)
            args[i] = _HEADS_GRAD.pack(
                d.data_ptr(), t.data_ptr(), 0 if gamma is None else gamma.data_ptr(),
                0 if o is None else o.data_ptr(), 0 if dg is None else dg.data_ptr(), t_at[0],
                *d_at, *t_at[1:], *o_at)
        batch, seq = lead if len(lead) == 2 else (1, lead[0])
        need = lib.b200norm_head_rms_rotary_grad_workspace_size(batch, seq, *heads, size)
        raw = _raw_stream(index, stream)
        ws, n = _scratch(workspace, need, x, index, raw)
        _check(lib.b200norm_head_rms_rotary_grad(*args, rotation, batch, seq, size, _DTYPES[dt],
                                                 _DTYPES[m], float(epsilon), _at(ws), n,
                                                 raw))
        if empty != [None, None]:  # of no tokens: zeros
            _check(lib.b200norm_head_rms_rotary_grad(*empty, rotation, 0, 0, size, _DTYPES[dt],
                                                     _DTYPES[m], float(epsilon), None, 0, raw))
        return dxs[0], dxs[1], dgs[0], dgs[1]

    context = _on(index, stream, (dq, dk, q, k, gamma_q, gamma_k, positions, inv_freq, dq_out,
                                  dk_out, dgamma_q, dgamma_k, workspace))
    if context is None:
        return run()
    with context:
        return run()
