"""Expert products in 8-bit floating point, activation checkpoints in 8 bits, and a whole layer for a few tokens.

Numbers in 8 bits are e4m3 with one 32-bit scale for each block of 128 columns of a row (``Rows8``) or of 128 x 128 of a
matrix (``Weights8``).  The scales that ``quantise_rows`` and ``quantise_weights`` make are powers of two, so that each
number is rounded once and the same on any path.  Scales made elsewhere may be any numbers for ``dequantise``, the
gradients and ``expert_layer``; ``expert_product8`` wants powers of two and tells of others through ``grouped_status``
(``quantise_rows(dequantise(q, torch.float32))`` and its like for matrices make them).

The calls follow the rules of the other grouped calls (streams, checks, no part in autograd): see grouped.py.
"""
from __future__ import annotations

import struct
from dataclasses import dataclass
from typing import Any

from .grouped import (Routing, _call, _dense, _entry_point, _pack_rule, _same_device, _SCORES, _GROUP_SCORES, _want,
                      _weights)

_pack_rows8 = struct.Struct("@PPqqqq").pack        # spgemm_rows8
_pack_weights8 = struct.Struct("@PPqqqqq").pack    # spgemm_weights8
BLOCK = 128


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def _values_ok(t, dims: int, name: str):
    import torch
    if t.dtype is not torch.float8_e4m3fn:
        raise TypeError("%s: float8_e4m3fn wanted, got %s" % (name, t.dtype))
    shape, step = t.shape, t.stride()
    if not t.is_cuda or len(shape) != dims or (shape[-1] > 1 and step[-1] != 1):
        raise ValueError("%s: a CUDA tensor of %d dimensions with contiguous rows is wanted" % (name, dims))
    if t.data_ptr() % 16 or any(shape[i] > 1 and step[i] % 16 for i in range(dims - 1)):
        raise ValueError("%s: rows and matrices start on 16 bytes (pad their strides)" % name)
    if shape[-2] > 1 and step[-2] < shape[-1]:
        raise ValueError("%s: rows overlap" % name)


class Rows8:
    """Rows in 8 bits: values (rows, cols) float8_e4m3fn, scales (rows, ceil(cols / 128)) float32, the scales of a block of
    columns one behind the other (the transpose of a contiguous tensor).  ``dtype``: what ``dequantise`` hands back and
    products of these rows give, unless told otherwise."""
    __slots__ = ("dtype", "shape", "_values", "_scales", "_store", "_at", "_bytes")

    def __init__(self, values, scales, dtype=None):
        import torch
        _values_ok(values, 2, "values")
        rows, cols = values.shape
        if scales.dtype is not torch.float32 or scales.device != values.device or tuple(scales.shape) != (rows, _blocks(cols)):
            raise ValueError("scales: (rows, ceil(cols / 128)) float32 beside the values is wanted")
        if (rows > 1 and scales.stride(0) != 1) or (scales.shape[1] > 1 and scales.stride(1) < rows):
            raise ValueError("scales: those of a block of columns one behind the other are wanted (scales.t().contiguous().t())")
        self.dtype, self.shape, self._values, self._scales, self._store, self._bytes = dtype, values.shape, values, scales, None, None

    @classmethod
    def _made(cls, store, at: int, rows: int, cols: int, dtype) -> "Rows8":
        """In bytes `at` and up of a tensor that this module allocated: the values, then the scales.  The tensors that a caller
        sees are made when they are asked for."""
        r = cls.__new__(cls)
        step, ptr = (cols + 15) // 16 * 16, store.data_ptr() + at
        r.dtype, r.shape, r._values, r._scales, r._store, r._at = dtype, (rows, cols), None, None, store, at
        r._bytes = _pack_rows8(ptr, ptr + rows * step, rows, cols, step, rows)
        return r

    @property
    def values(self):
        if self._values is None:
            import torch
            (rows, cols), at = self.shape, self._at
            step = (cols + 15) // 16 * 16
            self._values = self._store[at:at + rows * step].view(torch.float8_e4m3fn).view(rows, step)[:, :cols]
            self.shape = self._values.shape
        return self._values

    @property
    def scales(self):
        if self._scales is None:
            import torch
            (rows, cols), at = self.shape, self._at
            at += rows * ((cols + 15) // 16 * 16)
            blocks = _blocks(cols)
            self._scales = self._store[at:at + 4 * rows * blocks].view(torch.float32).view(blocks, rows).t()
        return self._scales

    @property
    def device(self):
        return (self._store if self._store is not None else self._values).device

    @property
    def requires_grad(self) -> bool:
        return any(t is not None and t.requires_grad for t in (self._values, self._scales))

    @property
    def _tensors(self):
        return tuple(t for t in (self._store, self._values, self._scales) if t is not None)

    def _with_scales(self, scales) -> "Rows8":
        r = Rows8.__new__(Rows8)
        r.dtype, r.shape, r._values, r._scales, r._store, r._bytes = self.dtype, self.shape, self.values, scales, None, None
        return r

    def __copy__(self) -> "Rows8":
        r = Rows8.__new__(Rows8)
        for name in Rows8.__slots__:
            if hasattr(self, name):
                setattr(r, name, getattr(self, name))
        return r

    def __reduce__(self):
        """Copies and saved ones are made of the tensors: the packed addresses are this one's.  As bytes, because the values
        and the scales may lie in one storage, which cannot be saved as two types."""
        import torch
        if self.requires_grad:
            raise RuntimeError("Rows8: of an input that wants a gradient, there is no copy (make it of detach()ed inputs)")
        if self._store is not None:
            return Rows8._made, (self._store, self._at, *map(int, self.shape), self.dtype)
        scales = self._scales.t().clone(memory_format=torch.contiguous_format)
        return _rows8_again, (self._values.view(torch.uint8), scales.view(torch.uint8), self.dtype)

    def _packed(self) -> bytes:
        if self._bytes is not None:
            return self._bytes
        v, s = self._values, self._scales
        rows, cols = v.shape
        stride = v.stride(0) if rows > 1 else (cols + 15) // 16 * 16
        return _pack_rows8(v.data_ptr(), s.data_ptr(), rows, cols, stride, s.stride(1) if s.shape[1] > 1 else rows)


def _rows8_again(values, scales, dtype) -> Rows8:
    """A Rows8 from its bytes."""
    import torch
    r = Rows8.__new__(Rows8)
    r.dtype, r.shape, r._store, r._bytes = dtype, values.shape, None, None
    r._values, r._scales = values.view(torch.float8_e4m3fn), scales.view(torch.float32).t()
    return r


@dataclass(frozen=True)
class Weights8:
    """One matrix per group in 8 bits: values (groups, rows, cols) float8_e4m3fn, scales (groups, ceil(rows / 128),
    ceil(cols / 128)) float32, contiguous.  ``dtype``: what ``dequantise`` hands back."""
    values: Any
    scales: Any
    dtype: Any = None

    def __post_init__(self):
        import torch
        _values_ok(self.values, 3, "values")
        s, (groups, rows, cols) = self.scales, self.values.shape
        if s.dtype is not torch.float32 or s.device != self.values.device or not s.is_contiguous() or \
                tuple(s.shape) != (groups, _blocks(rows), _blocks(cols)):
            raise ValueError("scales: (groups, ceil(rows / 128), ceil(cols / 128)) contiguous float32 beside the values is wanted")

    @classmethod
    def _made(cls, values, scales, dtype) -> "Weights8":
        w = cls.__new__(cls)
        w.__dict__.update(values=values, scales=scales, dtype=dtype)
        return w

    def _with_scales(self, scales) -> "Weights8":
        return Weights8._made(self.values, scales, self.dtype)

    @property
    def shape(self):
        return self.values.shape

    @property
    def device(self):
        return self.values.device

    @property
    def requires_grad(self) -> bool:
        return self.values.requires_grad or self.scales.requires_grad

    @property
    def _tensors(self):
        return (self.values, self.scales)

    def _packed(self) -> bytes:
        v = self.values
        groups, rows, cols = v.shape
        row = v.stride(1) if rows > 1 else (cols + 15) // 16 * 16
        return _pack_weights8(v.data_ptr(), self.scales.data_ptr(), groups, rows, cols, v.stride(0) if groups > 1 else rows * row,
                              row)


def _of(t, cls, name: str):
    if t.__class__ is not cls:
        raise TypeError("%s: %s wanted, got %s" % (name, cls.__name__, type(t).__name__))
    return t._packed()


def _16_bits(dtype, name: str):
    import torch
    if dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise TypeError("%s: float32, bfloat16 or float16 wanted, got %s" % (name, dtype))
    return dtype


def _empty_rows(rows: int, cols: int, dtype, device, count: int = 1) -> list:
    """`count` matrices of rows in 8 bits, in one allocation."""
    import torch
    each = (rows * ((cols + 15) // 16 * 16) + 4 * rows * _blocks(cols) + 15) // 16 * 16
    store = torch.empty(count * each, dtype=torch.uint8, device=device)
    return [Rows8._made(store, i * each, rows, cols, dtype) for i in range(count)]


@_entry_point
def quantise_rows(x, *, stream=None) -> Rows8:
    """x (rows, cols) in 8 bits (see spgemm_quantise_rows)."""
    d = _dense(x, "x")
    q, = _empty_rows(x.shape[0], x.shape[1], x.dtype, x.device)
    _call("spgemm_quantise_rows", x.device, d, q._packed())
    return q


@_entry_point
def quantise_weights(w, *, stream=None) -> Weights8:
    """w (groups, rows, cols) in 8 bits (see spgemm_quantise_weights)."""
    import torch
    d = _weights(w, "w")
    groups, rows, cols = w.shape
    step = (cols + 15) // 16 * 16
    values = torch.empty((groups, rows, step), dtype=torch.float8_e4m3fn, device=w.device)
    scales = torch.empty((groups, _blocks(rows), _blocks(cols)), dtype=torch.float32, device=w.device)
    q = Weights8._made(values[..., :cols], scales, w.dtype)
    _call("spgemm_quantise_weights", w.device, d, q._packed())
    return q


@_entry_point
def dequantise(q, dtype=None, *, stream=None):
    """What ``Rows8`` or ``Weights8`` stand for, in ``dtype`` (their own by default, float32 where they have none)."""
    import torch
    dtype = _16_bits(dtype or getattr(q, "dtype", None) or torch.float32, "dtype")
    if q.__class__ is Weights8:
        out = torch.empty(q.shape, dtype=dtype, device=q.device)
        _call("spgemm_dequantise_weights", q.device, q._packed(), _weights(out, "out"))
    else:
        d = _of(q, Rows8, "q")
        out = torch.empty(q.shape, dtype=dtype, device=q.device)
        _call("spgemm_dequantise_rows", q.device, d, _dense(out, "out"))
    return out


@_entry_point
def expert_product8(x, w, routing: Routing, *, grouped: bool = False, out_dtype=None, stream=None):
    """``expert_product`` in 8 bits: x ``Rows8``, or a tensor that is brought to 8 bits on the way; w ``Weights8``.

    The rows of the result have ``out_dtype``, else x's type.  See spgemm_quantised_product."""
    import torch
    _same_device("expert_product8", x, w, routing)
    g, dw = routing._grouping, _of(w, Weights8, "w")
    own = x.__class__ is Rows8
    dtype = _16_bits(out_dtype or x.dtype or torch.bfloat16, "out_dtype")
    y = torch.empty((routing.ids.numel(), w.shape[1]), dtype=dtype, device=x.device)
    _call("spgemm_quantised_product", x.device, g, None if own else _dense(x, "x"), x._packed() if own else None, int(grouped), dw,
          _dense(y, "y"))
    return y


@_entry_point
def expert_product8_backward(dy, x, w, routing: Routing, *, need_dx: bool = True, need_dw: bool = True, stream=None):
    """(dx, dw) of ``expert_product8`` with one row of x (``Rows8``, as the forward pass kept it) per token, in dy's type:
    the gradients of the product of what the 8 bits stand for (see spgemm_quantised_product_backward)."""
    import torch
    _same_device("expert_product8_backward", dy, x, w, routing)
    g, d8, w8 = routing._grouping, _of(x, Rows8, "x"), _of(w, Weights8, "w")
    dx = torch.empty(x.shape, dtype=dy.dtype, device=dy.device) if need_dx else None
    dw = torch.empty(w.shape, dtype=dy.dtype, device=dy.device) if need_dw else None
    _call("spgemm_quantised_product_backward", dy.device, g, _dense(dy, "dy"), d8, w8, _dense(dx, "dx") if need_dx else None,
          _weights(dw, "dw") if need_dw else None)
    return dx, dw


@_entry_point
def gated8(pre, *, out_dtype=None, stream=None):
    """(h, gate8, up8) of pre (rows, 2 * hidden) = gate | up: h = silu(gate) * up in ``out_dtype`` (pre's by default), and
    both halves as ``Rows8``, which is all that ``gated8_backward`` needs (see spgemm_quantised_gated)."""
    import torch
    d = _dense(pre, "pre")
    rows, both = pre.shape
    if both % 2:
        raise ValueError("pre: an even number of columns is wanted (gate, then up)")
    h = torch.empty((rows, both // 2), dtype=_16_bits(out_dtype or pre.dtype, "out_dtype"), device=pre.device)
    gate8, up8 = _empty_rows(rows, both // 2, h.dtype, pre.device, 2)
    _call("spgemm_quantised_gated", pre.device, d, _dense(h, "h"), gate8._packed(), up8._packed())
    return h, gate8, up8


@_entry_point
def gated8_backward(dh, gate8, up8, *, need_h: bool = True, stream=None):
    """(dpre, h) of ``gated8`` from what it kept, in dh's type; h, formed again, is the rows that the gradient of the next
    product's matrices wants (None without ``need_h``).  See spgemm_quantised_gated_backward."""
    import torch
    _same_device("gated8_backward", dh, gate8, up8)
    d, g, u = _dense(dh, "dh"), _of(gate8, Rows8, "gate8"), _of(up8, Rows8, "up8")
    dpre = torch.empty((dh.shape[0], 2 * dh.shape[1]), dtype=dh.dtype, device=dh.device)
    h = torch.empty(dh.shape, dtype=dh.dtype, device=dh.device) if need_h else None
    _call("spgemm_quantised_gated_backward", dh.device, d, g, u, _dense(dpre, "dpre"), _dense(h, "h") if need_h else None)
    return dpre, h


@_entry_point
def expert_layer(x, w_router, w_up, w_down, top_k: int, *, bias=None, score: str = "softmax", groups: int = 1,
                 groups_kept: int = 1, group_score: str = "max", renormalise: bool = True, scale: float = 1.0, stream=None):
    """A whole layer, (out, ids, weights): logits = x w_router^T, the choice of ``route``, the gated experts of ``experts``.

    x (tokens, d); w_router (experts, d) in x's type (a router in other bits: ``route`` of its logits, then ``experts``);
    w_up (experts, 2 * hidden, d) and w_down (experts, n, hidden) in x's type or as ``Weights8`` (x stays in 16 bits); ids
    and weights (tokens, top_k) as in ``Routing``.

    Made for decoding, up to 32 tokens (64 with ``Weights8``) in 16 bits with rows of full 16-byte pieces.  There the hidden
    row is held in two numbers of x's type, and scales multiply in 32 bits.  Anything else is the calls one after the other:
    the hidden row in one number, as in ``experts`` (in bf16 the result is 2.4e-3 off instead of 1.7e-3), and ``Weights8``
    of all experts, chosen or not, widened in every call to x's type (scratch of twice their size; scales that are no powers of two
    rounded with the weights): slower than the same matrices in 16 bits.  Keep those, or the calls in 8 bits
    (``expert_product8``, ``gated8``), for prompts.  See spgemm_expert_layer."""
    import torch
    _same_device("expert_layer", x, w_router, w_up, w_down, bias)
    d, r = _dense(x, "x"), _dense(w_router, "w_router")
    if score not in _SCORES or group_score not in _GROUP_SCORES:
        raise ValueError("score: softmax or sigmoid; group_score: max or top2")
    rule = _pack_rule(top_k, _SCORES[score], groups, groups_kept, _GROUP_SCORES[group_score], bool(renormalise), scale, 0)
    if bias is not None:
        _want(bias, "bias", torch.float32)
        if bias.numel() != w_router.shape[0]:
            raise ValueError("bias: one value per expert is wanted")
    eight = w_up.__class__ is Weights8
    if eight != (w_down.__class__ is Weights8):
        raise TypeError("w_up and w_down: both tensors or both Weights8")
    up, down = (w_up._packed(), w_down._packed()) if eight else (_weights(w_up, "w_up"), _weights(w_down, "w_down"))
    t, k, dev = x.shape[0], min(max(int(top_k), 1), 32), x.device  # other values are refused below
    out = torch.empty((t, w_down.shape[1]), dtype=x.dtype, device=dev)
    ids = torch.empty((t, k), dtype=torch.int32, device=dev)
    weights = torch.empty((t, k), dtype=torch.float32, device=dev)
    _call("spgemm_expert_layer", dev, d, r, rule, bias.data_ptr() if bias is not None else None, None if eight else up,
          None if eight else down, up if eight else None, down if eight else None, _dense(out, "out"), ids.data_ptr(),
          weights.data_ptr())
    return out, ids, weights
