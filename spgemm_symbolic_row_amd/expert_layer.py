"""The sparse expert layer: routing, dispatch, the experts' products with their
gradients, and clipping by the global gradient norm.

A router's output is a sparse matrix R (tokens x experts): row t holds the
experts picked for token t, columns rising, with their weights.  It is kept in
k slots a row (`col`, `val`; column -1 in an empty slot, and those last).

    r = sg.route(logits, k)
    y, kept = sg.experts(x, w_in, w_out, r.col, r.val, keep=True)
    dx, dw_in, dw_out, dval = sg.experts_backward(dy, kept)
    dlogits = sg.route_backward(logits, r, dval)
    norm = sg.clip_grad_norm([dw_in, dw_out, dlogits], max_norm=1.0)

Argument marshalling only: every step runs in the HIP library on the current
stream of the tensors' device, asynchronously.  Nothing is recorded for torch's
backward pass, the backward calls are the only way to the gradients: while torch
records, tensors that require one are refused (torch.no_grad() or detach()).
"""
from __future__ import annotations

import ctypes
from array import array
from contextlib import nullcontext
from dataclasses import dataclass
from functools import lru_cache

import torch

import spgemm_symbolic_row_amd as _package

from ._expert_abi import ExpertsDesc, RouteOptions, c_i64

_TYPES = {torch.float32: 0, torch.bfloat16: 2, torch.float16: 3}


def _lib():
    return _package._lib or _package.lib()


def _check(status):
    if status:
        _package._check(status)


_HERE = nullcontext()


def _on(x):
    """Makes x's device current, so that the call runs on its stream there."""
    i = x.get_device()
    if i < 0:
        raise TypeError("tensors must be device tensors")
    return _HERE if i == torch.cuda.current_device() else torch.cuda.device(i)


# The current stream's handle by device index, without a Stream object around
# it (2 us of a call's 10) where torch has that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(x):
    if _raw_stream is not None:
        return _raw_stream(x.get_device())
    return torch.cuda.current_stream(x.device).cuda_stream


_requires_grad = torch.Tensor.requires_grad.__get__


def _unrecorded(*tensors):
    """A result of tensors that require a gradient would have no graph."""
    if torch.is_grad_enabled() and True in map(_requires_grad, tensors):
        raise TypeError("a tensor requires a gradient, and nothing is recorded here: use the "
                        "backward calls, under torch.no_grad() or with detached tensors")


def _rows(x, what):
    """Row stride of a 2-d tensor whose rows are contiguous."""
    if x.dim() != 2:
        raise ValueError(f"{what} must have two dimensions")
    T, n = x.shape
    if n > 1 and x.stride(1) != 1:
        raise TypeError(f"{what} must have contiguous rows")
    ld = x.stride(0) if T > 1 else n  # the stride of a single row says nothing
    if ld < n:
        raise TypeError(f"{what} must not have overlapping rows")
    return ld


def _dense(x, shape, dtype, device, what):
    if x.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    if x.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {x.dtype}")
    if x.device != device:
        raise TypeError(f"{what} must be on {device}")
    if not x.is_contiguous():
        raise TypeError(f"{what} must be contiguous")


@lru_cache(maxsize=256)
def _route_options(scores, groups, top_groups, renormalise, scale):
    if scores not in ("softmax", "sigmoid"):
        raise ValueError("scores must be 'softmax' or 'sigmoid'")
    if not scale > 0.0:
        raise ValueError("scale must be positive")
    if groups < 1 or top_groups < 0:
        raise ValueError("groups must be positive and top_groups not negative")
    return RouteOptions(int(scores == "sigmoid"), groups, top_groups, int(not renormalise), scale)


@dataclass
class Routing:
    """A routing matrix, tokens x experts: k slots a row, and how it was made."""
    col: "torch.Tensor"      # T x k int32, rising; -1 in empty slots, which come last
    val: "torch.Tensor"      # T x k float32
    n_experts: int
    options: RouteOptions
    bias: "torch.Tensor | None" = None

    def csr(self):
        """R as a CsrDevice, for matmul and transpose (blocks once)."""
        from . import CsrDevice
        there = self.col >= 0
        row_ptr = torch.zeros(self.col.shape[0] + 1, dtype=torch.int32, device=self.col.device)
        row_ptr[1:] = torch.cumsum(there.sum(1), 0)
        return CsrDevice(row_ptr, self.col[there], self.val[there], self.col.shape[0],
                         self.n_experts)


def route(logits, k, scores="softmax", bias=None, groups=1, top_groups=0, renormalise=True,
          scale=1.0, active=None):
    """Row t of the routing matrix from row t of the logits (T x E; float32,
    bfloat16 or float16, rows contiguous): the k experts with the largest keys
    and their weights.  spgemm_route has the definition; `bias` (E, float32)
    enters the keys only, `active` (T, bool) marks the rows that are routed."""
    ld = _rows(logits, "logits")
    T, E = logits.shape
    dt = _TYPES.get(logits.dtype)
    if dt is None:
        raise TypeError("logits must be float32, bfloat16 or float16")
    dev = logits.device
    if bias is not None:
        _dense(bias, (E,), torch.float32, dev, "bias")
    if active is not None:
        _dense(active, (T,), torch.bool, dev, "active")
    _unrecorded(logits)
    o = _route_options(scores, groups, top_groups, bool(renormalise), float(scale))
    with _on(logits):
        col = torch.empty(T, max(k, 0), dtype=torch.int32, device=dev)
        val = torch.empty(T, max(k, 0), dtype=torch.float32, device=dev)
        _check(_lib().spgemm_route(T, E, k, logits.data_ptr(), ld, dt,
                                   None if bias is None else bias.data_ptr(),
                                   None if active is None else active.data_ptr(), o,
                                   col.data_ptr(), val.data_ptr(), _stream(logits)))
    return Routing(col, val, E, o, bias)


def route_backward(logits, routing, grad_val):
    """The gradient of the logits of `route`, in their type, for the gradient
    of the values (T x k, float32)."""
    ld = _rows(logits, "logits")
    T, E = logits.shape
    dt = _TYPES.get(logits.dtype)
    if dt is None:
        raise TypeError("logits must be float32, bfloat16 or float16")
    if E != routing.n_experts or T != routing.col.shape[0]:
        raise ValueError("logits are not the ones of this routing")
    dev = logits.device
    _dense(grad_val, routing.col.shape, torch.float32, dev, "grad_val")
    _unrecorded(grad_val)
    b = routing.bias
    with _on(logits):
        out = torch.empty(T, E, dtype=logits.dtype, device=dev)
        _check(_lib().spgemm_route_backward(T, E, routing.col.shape[1], logits.data_ptr(), ld, dt,
                                            None if b is None else b.data_ptr(), routing.options,
                                            routing.col.data_ptr(), grad_val.data_ptr(),
                                            out.data_ptr(), _stream(logits)))
    return out


def dispatch(col, n_experts):
    """The transpose of a routing matrix: (row_ptr, entry), the entries
    t * k + i of every expert in rising order (int32; the first
    row_ptr[n_experts] of the T * k places of `entry` are filled)."""
    if col.dim() != 2:
        raise ValueError("col must have two dimensions")
    T, k = col.shape
    dev = col.device
    _dense(col, (T, k), torch.int32, dev, "col")
    L = _lib()
    with _on(col):
        row_ptr = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
        entry = torch.empty(T * k, dtype=torch.int32, device=dev)
        need = L.spgemm_dispatch_workspace(T, k, n_experts)
        work = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        _check(L.spgemm_dispatch(T, k, n_experts, col.data_ptr(), row_ptr.data_ptr(),
                                 entry.data_ptr(), work.data_ptr(), need, _stream(col)))
    return row_ptr, entry


@lru_cache(maxsize=1024)
def _experts_desc(T, E, D, F, x_ld, grad_ld, k, dt, unaligned):
    d = ExpertsDesc(T, E, D, F, x_ld, grad_ld, k, dt, unaligned, 0)
    sizes = [c_i64(), c_i64(), c_i64()]
    _check(_lib().spgemm_experts_sizes(d, *map(ctypes.byref, sizes)))
    return d, sizes[0].value, sizes[1].value, sizes[2].value


class _Kept:
    """What a forward pass keeps for its backward pass: its inputs (borrowed,
    and not to be changed before), the library's block, and the stream that
    the block was taken from."""
    __slots__ = ("x", "w_in", "w_out", "val", "block", "stream")

    def __init__(self, *a):
        self.x, self.w_in, self.w_out, self.val, self.block, self.stream = a


def _off16(*tensors):
    bits = 0
    for t in tensors:
        bits |= t.data_ptr()
    return int(bits % 16 != 0)


def experts(x, w_in, w_out, col, val, keep=False):
    """y_t = sum over row t of the routing matrix (col, val: T x k) of
    val * W_out[e] (silu(W_gate[e] x_t) * (W_up[e] x_t)).

    x: T x D (rows contiguous), w_in: E x 2F x D, an expert's gate rows before
    its up rows, w_out: E x D x F; all bfloat16 or all float16.  With keep
    also returns what experts_backward takes."""
    x_ld = _rows(x, "x")
    T, D = x.shape
    if w_in.dim() != 3 or w_out.dim() != 3 or col.dim() != 2:
        raise ValueError("w_in and w_out must have three dimensions, col two")
    E, F = w_out.shape[0], w_out.shape[2]
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("x must be bfloat16 or float16")
    dev, k = x.device, col.shape[1]
    _dense(w_in, (E, 2 * F, D), x.dtype, dev, "w_in")
    _dense(w_out, (E, D, F), x.dtype, dev, "w_out")
    _dense(col, (T, k), torch.int32, dev, "col")
    _dense(val, (T, k), torch.float32, dev, "val")
    _unrecorded(x, w_in, w_out, val)
    d, kept_bytes, work_bytes, _ = _experts_desc(T, E, D, F, x_ld, D, k, _TYPES[x.dtype],
                                                 _off16(x, w_in, w_out))
    with _on(x):
        y = torch.empty(T, D, dtype=x.dtype, device=dev)
        block = torch.empty(kept_bytes, dtype=torch.uint8, device=dev) if keep else None
        work = torch.empty(max(work_bytes, 1), dtype=torch.uint8, device=dev)
        stream = _stream(x)
        _check(_lib().spgemm_experts_forward(d, x.data_ptr(), w_in.data_ptr(), w_out.data_ptr(),
                                             col.data_ptr(), val.data_ptr(), y.data_ptr(),
                                             block.data_ptr() if keep else None, work.data_ptr(),
                                             work_bytes, stream))
    return (y, _Kept(x, w_in, w_out, val, block, stream)) if keep else y


def experts_backward(grad_y, kept):
    """Gradients (grad_x, grad_w_in, grad_w_out, grad_val) of `experts` for the
    gradient of y (T x D, rows contiguous), from what its pass kept."""
    x, w_in, w_out, val = kept.x, kept.w_in, kept.w_out, kept.val
    if grad_y.shape != x.shape:
        raise ValueError(f"grad_y must have shape {tuple(x.shape)}, got {tuple(grad_y.shape)}")
    if grad_y.dtype != x.dtype or grad_y.device != x.device:
        raise TypeError(f"grad_y must be {x.dtype} on {x.device}")
    _unrecorded(grad_y)
    x_ld, g_ld = _rows(x, "x"), _rows(grad_y, "grad_y")
    T, D = x.shape
    E, F, k, dev = w_out.shape[0], w_out.shape[2], val.shape[1], x.device
    d, _, _, work_bytes = _experts_desc(T, E, D, F, x_ld, g_ld, k, _TYPES[x.dtype],
                                        _off16(x, w_in, w_out, grad_y))
    with _on(x):
        gx = torch.empty(T, D, dtype=x.dtype, device=dev)
        gw_in, gw_out = torch.empty_like(w_in), torch.empty_like(w_out)
        gval = torch.empty_like(val)
        stream = _stream(x)
        if stream != kept.stream:
            # What only `kept` may still hold is not given away before this stream is done with it.
            for t in (x, w_in, w_out, kept.block):
                t.record_stream(torch.cuda.current_stream(dev))
        work = torch.empty(max(work_bytes, 1), dtype=torch.uint8, device=dev)
        _check(_lib().spgemm_experts_backward(
            d, x.data_ptr(), w_in.data_ptr(), w_out.data_ptr(), grad_y.data_ptr(),
            kept.block.data_ptr(), gx.data_ptr(), gw_in.data_ptr(),
            gw_out.data_ptr(), gval.data_ptr(), work.data_ptr(), work_bytes, stream))
    return gx, gw_in, gw_out, gval


def clip_grad_norm(grads, max_norm, out=None):
    """The 2-norm over all the tensors (a float32 scalar on the device), and
    the tensors scaled by min(1, max_norm / (norm + 1e-6)): in place, or into
    the tensors of `out`, of as many elements each.  Contiguous float32, bfloat16 or float16 tensors of
    one device, mixed at will."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError("out must have as many tensors as grads")
    if not grads:
        raise ValueError("no gradients")
    dev, n = grads[0].device, len(grads)
    T = torch.Tensor
    if len(set(map(T.get_device, grads)) | set(map(T.get_device, outs))) != 1:
        raise TypeError("tensors must be on one device")
    sizes = array("q", map(T.numel, grads))
    if outs is not grads and sizes != array("q", map(T.numel, outs)):
        raise ValueError("out must have as many elements as grads, each")
    if not (all(map(T.is_contiguous, grads)) and all(map(T.is_contiguous, outs))):
        raise TypeError("tensors must be contiguous")
    _unrecorded(*(grads if outs is grads else grads + outs))
    try:
        types = array("i", [_TYPES[g.dtype] for g in grads])
        out_types = types if outs is grads else array("i", [_TYPES[o.dtype] for o in outs])
    except KeyError:
        raise TypeError("tensors must be float32, bfloat16 or float16") from None
    pointers = array("Q", map(T.data_ptr, grads))
    out_pointers = pointers if outs is grads else array("Q", map(T.data_ptr, outs))
    tables = [t.buffer_info()[0] for t in (pointers, out_pointers, sizes, types, out_types)]
    L = _lib()
    with _on(grads[0]):
        need = L.spgemm_clip_grad_norm_workspace(n)
        work = torch.empty(need, dtype=torch.uint8, device=dev)
        norm = torch.empty((), dtype=torch.float32, device=dev)
        _check(L.spgemm_clip_grad_norm(n, *tables, float(max_norm), norm.data_ptr(),
                                       work.data_ptr(), need, _stream(norm)))
    # Torch does not see the writes: tensors that it saved for a backward pass have changed.
    torch.autograd.graph.increment_version(outs)
    return norm
