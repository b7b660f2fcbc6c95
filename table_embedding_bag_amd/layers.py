"""Layers on looked-up rows: dropout, the gated linear recurrence over jagged sequences, and a
linear layer for each of several ragged row groups, each with its gradient.

The functions check their arguments, allocate outputs and workspaces with torch and call the
HIP kernels of ``libtbe.so`` (``include/tbe.h``) on the current stream of the tensors' GPU.
Rows may be strided (a slice of a wider buffer); the elements of a row are adjacent.  Bad
arguments raise ValueError, statuses of the library TBEError.

torch's autograd does not see these calls: a tensor that requires gradients is taken like any
other, results are not part of a graph, and each layer's backward function is called explicitly.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import (BF16, F16, F32, GATE_DECAY, GATE_SIGMOID, I32, I64, _check, _ScanInput, load)

_DTYPE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_INDEX = {torch.int32: I32, torch.int64: I64}
_U64 = (1 << 64) - 1
_MAX_POLLS = 0   # tbe_scan_input.max_polls: the library's default
_GATE = {"sigmoid": GATE_SIGMOID, "decay": GATE_DECAY}


def _fail(what):
    raise ValueError(what)


def _rows(t, name, dtype=None, shape=None):
    """The row stride of a 2-D tensor of rows, its type, shape and layout checked."""
    stride = t.stride()
    if len(stride) != 2:
        _fail(f"{name} must have 2 dimensions, got {len(stride)}")
    if dtype is None:
        if t.dtype not in _DTYPE:
            _fail(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    elif t.dtype != dtype:
        _fail(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        _fail(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if stride[1] != 1 and t.shape[1] > 1 and t.numel():
        _fail(f"the elements of a row of {name} must be adjacent")
    return stride[0]


def _out(t, name, dtype, shape):
    """The row stride of an output given by the caller: its rows must not overlap."""
    stride = _rows(t, name, dtype, shape)
    if t.shape[0] > 1 and stride < t.shape[1] and t.numel():
        _fail(f"the rows of {name} overlap")
    return stride


def _dense(t, name, dtype, shape):
    if t.dtype != dtype or t.shape != shape:
        _fail(f"{name} must be {dtype} of the shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        _fail(f"{name} must be contiguous")


def _offsets(t):
    """The number of ranges of CSR offsets."""
    if t.dtype not in _INDEX:
        _fail(f"offsets must be int32 or int64, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] < 1:
        _fail("offsets must have one dimension and at least one entry")
    if not t.is_contiguous():
        _fail("offsets must be contiguous")
    return t.shape[0] - 1


def _on_one_gpu(*tensors):
    """The tensors' GPU; None stands for an argument that was not given."""
    device = tensors[0].device
    for t in tensors:
        if t is not None:
            if not t.is_cuda:
                _fail("tensor must live on the GPU")
            if t.device != device:
                _fail("tensors must live on one GPU")
    return device


# One call's worth of microseconds counts for the smallest calls: the raw stream without a Stream
# object around it, where torch has that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(device, name, *args):
    """The library's function on the current stream of the device."""
    index = device.index
    if index == torch.cuda.current_device():
        status = getattr(load(), name)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = getattr(load(), name)(*args, _raw_stream(index))
    if status:
        _check(status, name)


def _p(t):
    return None if t is None else t.data_ptr()


def _like(t):
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _workspace(nbytes, like):
    return like.new_empty(nbytes, dtype=torch.uint8) if nbytes else None


# --- dropout -----------------------------------------------------------------------------------

def dropout(x, p, seed, offset, residual=None, out=None):
    """x / (1 - p) where an element is kept, else 0; plus residual, where given.

    Element n (in row-major order of x's shape) is kept where word n % 4 of the 7-round
    Philox4x32 block with counter ``offset + n // 4`` and key ``seed`` is at least
    floor(p * 2**32): the same (p, seed, offset) gives the same mask, which is never stored.
    A call uses ceil(x.numel() / 4) counters; the next call under this seed should start that
    much later.  x is a matrix of (strided) rows or a contiguous tensor of any shape; out may be
    x or residual itself.
    """
    if not 0.0 <= p <= 1.0:
        _fail(f"p must lie in [0, 1], got {p}")
    if not 0 <= seed <= _U64:
        _fail(f"seed must lie in [0, 2**64), got {seed}")
    if not 0 <= offset <= _U64:
        _fail(f"offset must lie in [0, 2**64), got {offset}")
    shape = x.shape
    if residual is not None and residual.shape != shape:
        _fail(f"residual must have the shape {tuple(shape)}, got {tuple(residual.shape)}")
    if out is not None and out.shape != shape:
        _fail(f"out must have the shape {tuple(shape)}, got {tuple(out.shape)}")
    x2, r2, out2 = x, residual, out
    if len(shape) != 2:
        for t in (x, residual, out):
            if t is not None and not t.is_contiguous():
                _fail("a tensor that is no matrix must be contiguous")
        x2 = x.view(1, -1)
        r2 = None if residual is None else residual.view(1, -1)
        out2 = None if out is None else out.view(1, -1)
    xs = _rows(x2, "x")
    rs = 0 if r2 is None else _rows(r2, "residual", x.dtype)
    if out is not None:
        ys = _out(out2, "out", x.dtype, x2.shape)
        device = _on_one_gpu(x, residual, out)
    else:
        device = _on_one_gpu(x, residual)
        out = _like(x)
        ys = x2.shape[1]
    _call(device, "tbe_dropout", x.data_ptr(), xs, _p(residual), rs, out.data_ptr(), ys, *x2.shape,
          _DTYPE[x.dtype], p, seed, offset)
    return out


def dropout_backward(grad, p, seed, offset, out=None):
    """The gradient with respect to x of ``dropout(x, p, seed, offset)``: the same map on the
    output's gradient.  (A residual's gradient is the output's itself.)"""
    return dropout(grad, p, seed, offset, out=out)


# --- gated linear recurrence -------------------------------------------------------------------

def _gate(kind):
    if kind not in _GATE:
        _fail(f"gate_kind must be 'sigmoid' or 'decay', got {kind!r}")
    return _GATE[kind]


def scan_step(x, gate, state=None, gate_kind="sigmoid", out_state=None):
    """One new token of each sequence: state' = a * state + b * x.

    x, gate [S, D]; state fp32 [S, D] (None: zeros).  Returns (h, state'), h being state' in x's
    type.  out_state may be state itself, which is then updated in place.
    """
    kind = _gate(gate_kind)
    xs = _rows(x, "x")
    gs = _rows(gate, "gate", x.dtype, x.shape)
    ss = 0 if state is None else _rows(state, "state", torch.float32, x.shape)
    if x.shape[1] < 1:
        _fail("rows must have at least one element")
    if out_state is not None:
        _dense(out_state, "out_state", torch.float32, x.shape)
    device = _on_one_gpu(x, gate, state, out_state)
    h = _like(x)
    if out_state is None:
        out_state = x.new_empty(x.shape, dtype=torch.float32) if state is None else _like(state)
    _call(device, "tbe_scan_step", x.data_ptr(), xs, gate.data_ptr(), gs, _p(state), ss, h.data_ptr(),
          out_state.data_ptr(), *x.shape, _DTYPE[x.dtype], kind)
    return h, out_state


def _scan_input(x, gate, offsets, initial, gate_kind):
    kind = _gate(gate_kind)
    xs = _rows(x, "x")
    gs = _rows(gate, "gate", x.dtype, x.shape)
    S = _offsets(offsets)
    N, D = x.shape
    if D < 1:
        _fail("rows must have at least one element")
    if S == 0 and N > 0:
        _fail("offsets hold no sequence for the tokens")
    ins = 0 if initial is None else _rows(initial, "initial", torch.float32, (S, D))
    return S, _ScanInput(N, S, D, _DTYPE[x.dtype], kind, _INDEX[offsets.dtype], _MAX_POLLS,
                         x.data_ptr(), xs, gate.data_ptr(), gs, offsets.data_ptr(), _p(initial), ins)


@functools.lru_cache(maxsize=256)
def _scan_sizes(N, S, D, dtype):
    carry, ws = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load().tbe_scan_sizes(N, S, D, _DTYPE[dtype], ctypes.byref(carry), ctypes.byref(ws)),
           "tbe_scan_sizes")
    return carry.value, ws.value


def scan_forward(x, gate, offsets, initial=None, gate_kind="sigmoid", need_carry=True):
    """The recurrence h_t = a_t h_{t-1} + b_t x_t along each jagged sequence, per channel.

    x, gate [N, D]; offsets [S + 1] (int32 or int64, 0 first, N last): sequence s holds the
    tokens offsets[s] .. offsets[s+1]; initial: fp32 [S, D] states before the first tokens
    (None: zeros).  gate_kind "sigmoid": a = sigmoid(gate), b = 1 - a; "decay": a = gate, b = 1.
    Returns (h [N, D] in x's type, final fp32 [S, D], carry): carry is what scan_backward needs
    (None without need_carry).  An empty sequence's final state is its initial one.

    States pass along a sequence through products of up to 1024 gates in fp32.  Where gates above
    1 take such a product past fp32's range, a state of 0 stays 0, another may come out infinite
    or NaN where one token after another would not; the same holds for the gradients.
    """
    S, inp = _scan_input(x, gate, offsets, initial, gate_kind)
    device = _on_one_gpu(x, gate, offsets, initial)
    N, D = x.shape
    nc, nw = _scan_sizes(N, S, D, x.dtype)
    h = x.new_empty((N, D))
    final = x.new_empty((S, D), dtype=torch.float32)
    carry = x.new_empty(nc // 4, dtype=torch.float32) if need_carry else None
    ws = _workspace(nw, x)
    _call(device, "tbe_scan_forward", ctypes.byref(inp), h.data_ptr(), final.data_ptr(), _p(carry), _p(ws),
          nw)
    return h, final, carry


def scan_backward(x, gate, offsets, carry, grad_h=None, grad_final=None, initial=None,
                  gate_kind="sigmoid", out=None):
    """Gradients of scan_forward(x, gate, offsets, initial, gate_kind), whose carry this is.

    grad_h [N, D] (x's type) and grad_final (fp32 [S, D]) are the gradients of h and final
    (None: zeros).  Returns (dx, dgate, dinitial); out=(dx, dgate) takes two matrices of rows to
    write, the halves of one projection's gradient, say.
    """
    S, inp = _scan_input(x, gate, offsets, initial, gate_kind)
    N, D = x.shape
    hs = 0 if grad_h is None else _rows(grad_h, "grad_h", x.dtype, x.shape)
    fs = 0 if grad_final is None else _rows(grad_final, "grad_final", torch.float32, (S, D))
    nc, nw = _scan_sizes(N, S, D, x.dtype)
    if carry is None or carry.dtype != torch.float32 or carry.numel() * 4 != nc or \
            not carry.is_contiguous():
        _fail("carry is not that of a forward call of these sizes")
    if out is not None:
        for t, name in zip(out, ("dx", "dgate")):
            _out(t, name, x.dtype, x.shape)
    device = _on_one_gpu(x, gate, offsets, initial, carry, grad_h, grad_final, *(out or ()))
    dx, dgate = out if out is not None else (x.new_empty((N, D)), x.new_empty((N, D)))
    dinitial = x.new_empty((S, D), dtype=torch.float32)
    ws = _workspace(nw, x)
    _call(device, "tbe_scan_backward", ctypes.byref(inp), carry.data_ptr(), _p(grad_h), hs, _p(grad_final),
          fs, dx.data_ptr(), dx.stride(0), dgate.data_ptr(), dgate.stride(0), dinitial.data_ptr(), _p(ws), nw)
    return dx, dgate, dinitial


# --- grouped linear layer ----------------------------------------------------------------------

@functools.lru_cache(maxsize=256)
def _grouped_sizes(N, G, K, M, dtype):
    fw, bw = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load().tbe_grouped_linear_sizes(N, G, K, M, _DTYPE[dtype], ctypes.byref(fw), ctypes.byref(bw)),
           "tbe_grouped_linear_sizes")
    return fw.value, bw.value


def _grouped(x, weight, offsets):
    xs = _rows(x, "x")
    G = _offsets(offsets)
    N, K = x.shape
    if weight.dim() != 3 or weight.dtype != x.dtype or weight.shape[0] != G or \
            weight.shape[2] != K or weight.shape[1] < 1 or K < 1:
        _fail(f"weight must be {x.dtype} of the shape ({G}, out_features, {K}), got {weight.dtype} "
              f"{tuple(weight.shape)}")
    if not weight.is_contiguous():
        _fail("weight must be contiguous")
    if G == 0 and N > 0:
        _fail("offsets hold no group for the rows")
    M = weight.shape[1]
    return (xs, N, G, K, M, *_grouped_sizes(N, G, K, M, x.dtype))


def grouped_linear(x, weight, offsets, bias=None, out=None):
    """y_n = weight[g] @ x_n + bias[g] for the rows offsets[g] .. offsets[g+1] of each group g.

    x [N, K]; weight [G, M, K]; offsets [G + 1] (int32 or int64, 0 first, N last; they stay on
    the GPU, groups may be empty); bias [G, M].  Returns y [N, M] in x's type.
    """
    xs, N, G, K, M, nw, _ = _grouped(x, weight, offsets)
    if bias is not None:
        _dense(bias, "bias", x.dtype, (G, M))
    if out is not None:
        _out(out, "out", x.dtype, (N, M))
    device = _on_one_gpu(x, weight, offsets, bias, out)
    ys = M if out is None else out.stride(0)
    if out is None:
        out = x.new_empty((N, M))
    ws = _workspace(nw, x)
    _call(device, "tbe_grouped_linear", x.data_ptr(), xs, weight.data_ptr(), _p(bias), offsets.data_ptr(),
          _INDEX[offsets.dtype], out.data_ptr(), ys, N, G, K, M, _DTYPE[x.dtype], _p(ws), nw)
    return out


def grouped_linear_backward(x, weight, offsets, grad, bias=False, need_dx=True, need_dweight=True):
    """Gradients (dx, dweight, dbias) of grouped_linear from that of its output, grad [N, M].

    dbias is computed where ``bias`` is true; what is not asked for is None.  Empty groups get
    gradients of zero.
    """
    xs, N, G, K, M, _, nw = _grouped(x, weight, offsets)
    gs = _rows(grad, "grad", x.dtype, (N, M))
    device = _on_one_gpu(x, weight, offsets, grad)
    dx = x.new_empty((N, K)) if need_dx else None
    dw = x.new_empty((G, M, K)) if need_dweight else None
    db = x.new_empty((G, M)) if bias else None
    if not need_dweight:   # the workspace is for the weights' chunks of rows alone
        nw = 0
    ws = _workspace(nw, x)
    _call(device, "tbe_grouped_linear_backward", x.data_ptr(), xs, weight.data_ptr(), offsets.data_ptr(),
          _INDEX[offsets.dtype], grad.data_ptr(), gs, _p(dx), K, _p(dw), _p(db), N, G, K, M, _DTYPE[x.dtype],
          _p(ws), nw)
    return dx, dw, db
