"""Layer norm in front of an expert layer, with its gradient.

    h, kept = sg.layer_norm(x, weight, bias, keep=True)     # or keep="e4m3"
    dx, dweight, dbias = sg.layer_norm_backward(dh, kept)

As in the expert layer, every step runs in the HIP library on the current
stream of the tensors' device, and nothing is recorded for torch's backward pass.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from ._expert_abi import LayerNormDesc, c_i64
from .expert_layer import _TYPES, _check, _lib, _on, _rows, _stream, _unrecorded

_FORMS = {False: 0, True: 1, "e4m3": 2}


@lru_cache(maxsize=1024)
def _desc(T, D, x_ld, grad_ld, dt, weight_dt, eps, form):
    d = LayerNormDesc(T, D, x_ld, grad_ld, dt, weight_dt, eps, form)
    sizes = [c_i64(), c_i64()]
    _check(_lib().spgemm_layer_norm_sizes(d, *map(ctypes.byref, sizes)))
    return d, sizes[0].value, sizes[1].value


class _KeptRows:
    """What a forward pass keeps: x (borrowed, and not to be changed before the
    backward pass; None where the library's block holds it in 8 bits), the weight, the
    block, and the stream that the block was taken from."""
    __slots__ = ("x", "weight", "biased", "rows", "dtype", "eps", "form", "block", "stream")

    def __init__(self, *a):
        (self.x, self.weight, self.biased, self.rows, self.dtype, self.eps, self.form, self.block,
         self.stream) = a


def layer_norm(x, weight, bias=None, eps=1e-5, keep=False):
    """(x - mean) / sqrt(variance + eps) * weight + bias of every row of x.

    x: T x D (rows contiguous; float32, bfloat16 or float16; D up to 16384),
    weight and bias: D elements, float32 or x's type, both alike.  With keep=True also returns
    what layer_norm_backward takes, and x and weight must not change before; with
    keep="e4m3" that holds x in 8 bits (a power-of-two scale for each 128 columns of
    a row), and x itself need not stay: the gradients are then those at the values
    that the 8 bits stand for, with the mean and the variance of x.  They are up to
    1/16 of |x| off, so take keep=True for rows whose mean is many deviations."""
    x_ld = _rows(x, "x")
    T, D = x.shape
    dt = _TYPES.get(x.dtype)
    if dt is None:
        raise TypeError("x must be float32, bfloat16 or float16")
    form = _FORMS.get(keep) if isinstance(keep, (bool, str)) else None
    if form is None:
        raise ValueError("keep must be False, True or 'e4m3'")
    dev = x.device
    for w, what in ((weight, "weight"), (bias, "bias")):
        if w is None and what == "bias":
            continue
        if w.shape != (D,):
            raise ValueError(f"{what} must have shape ({D},), got {tuple(w.shape)}")
        if w.dtype is not weight.dtype or w.dtype not in (torch.float32, x.dtype):
            raise TypeError("weight and bias must both be float32 or both of x's type")
        if w.device != dev:
            raise TypeError(f"{what} must be on {dev}")
        if not w.is_contiguous():
            raise TypeError(f"{what} must be contiguous")
    if bias is None:
        _unrecorded(x, weight)
    else:
        _unrecorded(x, weight, bias)
    eps = float(eps)
    d, kept_bytes, _ = _desc(T, D, x_ld, D, dt, _TYPES[weight.dtype], eps, form)
    with _on(x):
        y = torch.empty(T, D, dtype=x.dtype, device=dev)
        block = torch.empty(kept_bytes, dtype=torch.uint8, device=dev) if form else None
        stream = _stream(x)
        _check(_lib().spgemm_layer_norm_forward(
            d, x.data_ptr(), weight.data_ptr(), None if bias is None else bias.data_ptr(),
            y.data_ptr(), block.data_ptr() if form else None, stream))
    if not form:
        return y
    return y, _KeptRows(x if form == 1 else None, weight, bias is not None, (T, D), x.dtype, eps,
                        form, block, stream)


def layer_norm_backward(grad_y, kept):
    """Gradients (grad_x, grad_weight, grad_bias) of `layer_norm` for the gradient
    of y (T x D, rows contiguous, in x's type), from what its pass kept; the last is
    None where there was no bias, the weights' are in their type."""
    x, weight, (T, D) = kept.x, kept.weight, kept.rows
    if grad_y.shape != kept.rows:
        raise ValueError(f"grad_y must have shape {kept.rows}, got {tuple(grad_y.shape)}")
    dev = weight.device
    if grad_y.dtype != kept.dtype or grad_y.device != dev:
        raise TypeError(f"grad_y must be {kept.dtype} on {dev}")
    _unrecorded(grad_y)
    d, _, work_bytes = _desc(T, D, D if x is None else _rows(x, "x"), _rows(grad_y, "grad_y"),
                             _TYPES[kept.dtype], _TYPES[weight.dtype], kept.eps, kept.form)
    with _on(weight):
        gx = torch.empty(T, D, dtype=kept.dtype, device=dev)
        gw = torch.empty_like(weight)
        gb = torch.empty_like(weight) if kept.biased else None
        stream = _stream(weight)
        if stream != kept.stream:
            # What only `kept` may still hold is not given away before this stream is done with it.
            for t in (x, weight, kept.block):
                if t is not None:
                    t.record_stream(torch.cuda.current_stream(dev))
        work = torch.empty(work_bytes, dtype=torch.uint8, device=dev)
        _check(_lib().spgemm_layer_norm_backward(
            d, None if x is None else x.data_ptr(), weight.data_ptr(), grad_y.data_ptr(),
            kept.block.data_ptr(), gx.data_ptr(), gw.data_ptr(), None if gb is None else gb.data_ptr(),
            work.data_ptr(), work_bytes, stream))
    return gx, gw, gb
