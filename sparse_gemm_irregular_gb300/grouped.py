"""Routing, expert products and per-request adapters: rows of a dense matrix multiplied by the
matrix of the group that a sparse choice sends them to.

The calls marshal PyTorch device tensors into the C entry points of include/spgemm.h
(``spgemm_route`` and those after it) and allocate the outputs; they enqueue on the given or the
current stream and do not synchronise.  ``Routing`` is the choice together with its transpose.

A call with ``stream=`` is the call with that stream current: its outputs belong to that stream, its inputs'
memory is not handed out again before the stream has passed it.  What the inputs still wait for on other
streams, and who reads the outputs on others, is the caller's to order, as everywhere in PyTorch.

The calls take no part in autograd: gradients are formed by the calls whose names end in ``_backward``.  An output
of inputs that want a gradient raises when one is asked of it.
"""
from __future__ import annotations

import functools
import struct
from dataclasses import dataclass
from typing import Any

from . import binding
from .binding import _check, load

# The structures of include/spgemm.h as bytes (a call borrows them): packed in one step, these calls are
# short enough for the difference to ctypes' field-by-field structures to count.
_pack_dense = struct.Struct("@Pqqqii").pack        # spgemm_dense
_pack_weights = struct.Struct("@Pqqqqqii").pack    # spgemm_weights
_pack_grouping = struct.Struct("@qiiPPP").pack     # spgemm_grouping
_pack_rule = struct.Struct("@6ifi").pack           # spgemm_route_rule

_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}


@dataclass(frozen=True)
class Routing:
    """The choice of every token and its transpose, in device memory.

    ids (tokens, top_k) int32: chosen groups, ascending, -1 for none; weights (tokens, top_k)
    float32; offsets (groups + 1) int32: positions of each group; order (slots) int32: the slot
    (token * top_k + j) at each position, -1 behind the last group; position (tokens, top_k)
    int32: the position of each slot, -1 for none.  ``rule`` holds the options of ``route``."""
    ids: Any
    weights: Any
    offsets: Any
    order: Any
    position: Any
    rule: Any = None

    def __post_init__(self):
        import torch
        i32, n = torch.int32, self.ids.numel()
        for name in ("ids", "offsets", "order", "position", "weights"):
            t = getattr(self, name)
            if t.dtype is not (torch.float32 if name == "weights" else i32) or not t.is_cuda or not t.is_contiguous():
                raise ValueError("%s: a contiguous CUDA tensor of %s is wanted"
                                 % (name, "float32" if name == "weights" else "int32"))
            if t.numel() != n and name != "offsets":
                raise ValueError("routing: ids, weights, order and position want tokens * top_k entries each")
        _same_device("routing", self.ids, self.weights, self.offsets, self.order, self.position)
        if self.ids.dim() != 2 or self.offsets.dim() != 1:
            raise ValueError("ids: (tokens, top_k) and offsets: (groups + 1) are wanted")

    @classmethod
    def _made(cls, ids, weights, offsets, order, position, rule=None) -> "Routing":
        """From arrays that this module allocated: nothing to check."""
        r = cls.__new__(cls)
        r.__dict__.update(ids=ids, weights=weights, offsets=offsets, order=order, position=position, rule=rule)
        return r

    @property
    def _grouping(self) -> bytes:
        tokens, k = self.ids.shape
        return _pack_grouping(tokens * k, k, self.offsets.shape[0] - 1, self.offsets.data_ptr(), self.order.data_ptr(),
                              self.position.data_ptr())

    @property
    def device(self):
        return self.ids.device

    @property
    def tokens(self) -> int:
        return self.ids.shape[0]

    @property
    def top_k(self) -> int:
        return self.ids.shape[1]

    @property
    def groups(self) -> int:
        return self.offsets.numel() - 1

    def to_csr(self):
        """The choice as a DeviceCSR (tokens x groups, the weights in float64) for the library's
        sparse products.  Copies the number of entries to the host."""
        import torch
        from . import DeviceCSR
        there = self.position >= 0  # an id out of range has none
        row_ptr = torch.zeros(self.tokens + 1, dtype=torch.int64, device=self.ids.device)
        row_ptr[1:] = there.sum(1).cumsum(0)
        return DeviceCSR(self.tokens, self.groups, row_ptr, self.ids[there].contiguous(),
                         self.weights[there].double().contiguous())

    def transposed_csr(self):
        """The transposed choice as a DeviceCSR (groups x tokens)."""
        import torch  # noqa: F401
        from . import DeviceCSR
        n = int(self.offsets[-1])
        slot = self.order[:n].long()
        return DeviceCSR(self.groups, self.tokens, self.offsets.long(), (slot // self.top_k).int(),
                         self.weights.reshape(-1)[slot].double())


_codes: dict = {}  # torch dtype -> SPGEMM_DTYPE_*, filled on first use (the package imports without torch)


def _refuse(t, name: str, dims: int):
    import torch
    if not _codes:
        _codes.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    if t.dtype not in _codes:
        raise TypeError("%s: float32, bfloat16 or float16 wanted, got %s" % (name, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s: a CUDA tensor is wanted" % name)
    if t.dim() != dims or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError("%s: %d dimensions with contiguous rows are wanted" % (name, dims))


def _want(t, name: str, dtype):
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s: a contiguous CUDA tensor of %s is wanted" % (name, dtype))


def _one_row(rows: int, cols: int, step: int, name: str) -> int:
    """The stride of a matrix whose own is shorter than a row: any will do for a single row, others are refused
    (expanded tensors and sliding windows: the library's matrices have their rows one behind the other)."""
    if rows > 1:
        raise ValueError("%s: rows overlap (stride %d, %d columns); contiguous() makes a copy that does not" % (name, step, cols))
    return cols


def _dense(t, name: str) -> bytes:
    shape, step, code = t.shape, t.stride(), _codes.get(t.dtype)
    if code is None or not t.is_cuda or len(shape) != 2 or (step[1] != 1 and shape[1] > 1):
        _refuse(t, name, 2)
        code = _codes[t.dtype]
    rows, cols = shape
    return _pack_dense(t.data_ptr(), rows, cols, step[0] if step[0] >= cols else _one_row(rows, cols, step[0], name), code, 0)


def _weights(t, name: str) -> bytes:
    shape, step, code = t.shape, t.stride(), _codes.get(t.dtype)
    if code is None or not t.is_cuda or len(shape) != 3 or (step[2] != 1 and shape[2] > 1):
        _refuse(t, name, 3)
        code = _codes[t.dtype]
    groups, rows, cols = shape
    return _pack_weights(t.data_ptr(), groups, rows, cols, step[0],
                         step[1] if step[1] >= cols else _one_row(rows, cols, step[1], name), code, 0)


_entry: dict = {}  # entry points by name


def _same_device(name: str, first, *others):
    """Refuses tensors (and routings, None left out) of different devices: a kernel follows their addresses on one."""
    dev = first.device
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError("%s: tensors on %s and on %s" % (name, dev, t.device))


def _used(args, kw) -> list:
    """The tensors of a call, those of its routing among them."""
    found = []
    for a in (*args, *kw.values()):
        if isinstance(a, Routing):
            found += (a.ids, a.weights, a.offsets, a.order, a.position)
        elif hasattr(a, "requires_grad"):
            found.append(a)
    return found


def _wants_gradient(args, kw) -> bool:
    for a in args if not kw else (*args, *kw.values()):
        if getattr(a.weights if a.__class__ is Routing else a, "requires_grad", False):
            return True
    return False


_stop = None  # made on first use (the package imports without torch)


def _without_graph(name: str, out, used):
    """`out`, with a node in the graph that says that there is no way back through `name`."""
    import torch
    global _stop
    if _stop is None:
        class Stop(torch.autograd.Function):
            @staticmethod
            def forward(ctx, name, t, *used):
                ctx.call = name
                return t.view_as(t)

            @staticmethod
            def backward(ctx, *_):
                raise RuntimeError("%s takes no part in autograd: form its gradient with the call of that name that ends in "
                                   "_backward, or detach() its inputs" % ctx.call)
        _stop = Stop

    def stop(t):
        return _stop.apply(name, t, *used) if t is not None and t.is_floating_point() else t

    if isinstance(out, Routing):
        return Routing._made(out.ids, stop(out.weights), out.offsets, out.order, out.position, out.rule)
    return tuple(map(stop, out)) if isinstance(out, tuple) else stop(out)


def _entry_point(fn):
    """Gives a call its ``stream`` argument (everything that it allocates, fills and launches belongs there), and an
    end to the graph that tells of itself where an input wants a gradient."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        import torch
        if stream is None:
            out = fn(*args, **kw)
        else:
            used = _used(args, kw)
            for t in used:
                if t.device != stream.device:
                    raise ValueError("stream: on %s, a tensor on %s" % (stream.device, t.device))
            with torch.cuda.stream(stream):
                out = fn(*args, **kw)
            for t in used:
                t.record_stream(stream)
        if torch.is_grad_enabled() and _wants_gradient(args, kw):
            return _without_graph(fn.__name__, out, _used(args, kw))
        return out
    return call


def _call(name: str, device, *args):
    """Call an entry point with `device` current and its current stream as last argument."""
    import torch
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(load(), name)
    index = device.index
    raw = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc:
        _check(rc, name)


@_entry_point
def route(logits, top_k: int, *, bias=None, score: str = "softmax", groups: int = 1, groups_kept: int = 1,
          group_score: str = "max", renormalise: bool = True, scale: float = 1.0, stream=None) -> Routing:
    """Choose ``top_k`` experts per token from router logits (tokens, experts).

    score: "softmax" or "sigmoid"; bias (experts) float32 takes part in the choice only; the
    experts form ``groups`` equal runs of which the ``groups_kept`` best ("max": by their best
    expert, "top2": by the sum of their two best) take part.  See spgemm_route."""
    import torch
    _same_device("route", logits, bias)
    d = _dense(logits, "logits")
    if score not in _SCORES or group_score not in _GROUP_SCORES:
        raise ValueError("score: softmax or sigmoid; group_score: max or top2")
    rule = _pack_rule(top_k, _SCORES[score], groups, groups_kept, _GROUP_SCORES[group_score], bool(renormalise), scale,
                      0)
    if bias is not None:
        _want(bias, "bias", torch.float32)
        if bias.numel() != logits.shape[1]:
            raise ValueError("bias: one value per expert is wanted")
    t, dev, k = logits.shape[0], logits.device, min(max(int(top_k), 1), 32)  # other values are refused below
    n = t * k
    weights = torch.empty((t, k), dtype=torch.float32, device=dev)
    whole = torch.empty(3 * n + logits.shape[1] + 1, dtype=torch.int32, device=dev)  # one allocation for four arrays
    ids, position = whole.as_strided((t, k), (k, 1)), whole.as_strided((t, k), (k, 1), n)
    order, offsets = whole.as_strided((n,), (1,), 2 * n), whole.as_strided((logits.shape[1] + 1,), (1,), 3 * n)
    _call("spgemm_route", dev, d, rule, bias.data_ptr() if bias is not None else None,
          ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(), order.data_ptr(), position.data_ptr())
    return Routing._made(ids, weights, offsets, order, position, rule)


@_entry_point
def route_backward(logits, routing: Routing, grad_weights, *, stream=None):
    """Gradient of the logits for a gradient of ``routing.weights`` (see spgemm_route_backward)."""
    import torch
    _same_device("route_backward", logits, routing, grad_weights)
    if routing.rule is None:
        raise ValueError("route_backward: the routing does not come from route()")
    d = _dense(logits, "logits")
    _want(grad_weights, "grad_weights", torch.float32)
    if grad_weights.shape != routing.ids.shape or logits.shape[0] != routing.tokens:
        raise ValueError("grad_weights: (tokens, top_k) is wanted")
    out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    _call("spgemm_route_backward", logits.device, d, routing.rule, routing.ids.data_ptr(),
          grad_weights.data_ptr(), _dense(out, "grad_logits"))
    return out


@_entry_point
def group_rows(ids, groups: int, *, weights=None, stream=None) -> Routing:
    """The Routing of given ids (tokens, top_k) or (tokens,) int32, -1 for none; weights default to
    ones (see spgemm_group_rows)."""
    import torch
    _same_device("group_rows", ids, weights)
    _want(ids, "ids", torch.int32)
    if ids.dim() not in (1, 2):
        raise ValueError("ids: (tokens, top_k) or (tokens) are wanted")
    ids = ids if ids.dim() == 2 else ids[:, None]
    dev = ids.device
    offsets = torch.empty(groups + 1, dtype=torch.int32, device=dev)
    order = torch.empty(ids.numel(), dtype=torch.int32, device=dev)
    position = torch.empty_like(ids)
    _call("spgemm_group_rows", dev, ids.data_ptr(), ids.numel(), groups, offsets.data_ptr(),
          order.data_ptr(), position.data_ptr())
    if weights is None:
        weights = torch.ones(ids.shape, dtype=torch.float32, device=dev)
    _want(weights, "weights", torch.float32)
    if weights.numel() != ids.numel():
        raise ValueError("weights: one per id is wanted")
    return Routing._made(ids, weights, offsets, order, position)


@_entry_point
def expert_product(x, w, routing: Routing, *, grouped: bool = False, out_dtype=None, stream=None):
    """Rows times the matrix of their group: (slots, w.shape[1]) in group order.

    x (tokens, d), or (slots, d) in group order with ``grouped``; w (groups, n, d).  See
    spgemm_grouped_product."""
    import torch
    _same_device("expert_product", x, w, routing)
    g = routing._grouping
    dx, dw = _dense(x, "x"), _weights(w, "w")
    y = torch.empty((routing.ids.numel(), w.shape[1]), dtype=out_dtype or x.dtype, device=x.device)
    _call("spgemm_grouped_product", x.device, g, dx, int(grouped), dw, _dense(y, "y"))
    return y


@_entry_point
def expert_product_backward(dy, x, w, routing: Routing, *, need_dx: bool = True, need_dw: bool = True, stream=None):
    """(dx, dw) of ``expert_product`` with one row of x per token (see spgemm_grouped_product_backward)."""
    import torch
    _same_device("expert_product_backward", x, dy, w, routing)
    g = routing._grouping
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need_dx else None
    dw = torch.empty(w.shape, dtype=w.dtype, device=x.device) if need_dw else None
    _call("spgemm_grouped_product_backward", x.device, g, _dense(dy, "dy"), _dense(x, "x"),
          _weights(w, "w"), _dense(dx, "dx") if need_dx else None,
          _weights(dw, "dw") if need_dw else None)
    return dx, dw


@_entry_point
def combine(y, routing: Routing, *, out_dtype=None, stream=None):
    """Weighted sum of a token's rows: (tokens, y.shape[1]) (see spgemm_combine)."""
    import torch
    _same_device("combine", y, routing)
    g = routing._grouping
    out = torch.empty((routing.tokens, y.shape[1]), dtype=out_dtype or y.dtype, device=y.device)
    _call("spgemm_combine", y.device, g, routing.weights.data_ptr(), _dense(y, "y"),
          _dense(out, "out"))
    return out


@_entry_point
def combine_backward(dout, y, routing: Routing, *, stream=None):
    """(dy, dweights) of ``combine``; dy has dout's type, y may have another (see spgemm_combine_backward)."""
    import torch
    _same_device("combine_backward", y, dout, routing)
    g = routing._grouping
    dy = torch.empty(y.shape, dtype=dout.dtype, device=y.device)
    dweights = torch.empty(routing.ids.shape, dtype=torch.float32, device=y.device)
    _call("spgemm_combine_backward", y.device, g, routing.weights.data_ptr(),
          _dense(dout, "dout"), _dense(y, "y"), _dense(dy, "dy"), dweights.data_ptr())
    return dy, dweights


@_entry_point
def experts(x, w_up, w_down, routing: Routing, *, stream=None):
    """A gated expert layer, (tokens, d) -> (tokens, w_down.shape[1]): w_up (groups, 2 * hidden, d)
    holds the gate's rows, then up's; w_down (groups, n, hidden).  See spgemm_experts."""
    import torch
    _same_device("experts", x, w_up, w_down, routing)
    g = routing._grouping
    out = torch.empty((x.shape[0], w_down.shape[1]), dtype=x.dtype, device=x.device)
    _call("spgemm_experts", x.device, g, routing.weights.data_ptr(), _dense(x, "x"),
          _weights(w_up, "w_up"), _weights(w_down, "w_down"), _dense(out, "out"))
    return out


@_entry_point
def adapted_product(x, w, a, b, ids, scale=None, *, stream=None):
    """x w^T + scale[i] (x a[i]^T) b[i]^T with i = ids[token] (int32; -1: the projection alone).

    x (tokens, d), w (n, d), a (adapters, rank, d), b (adapters, n, rank), scale (adapters)
    float32.  See spgemm_adapted_product."""
    import torch
    _same_device("adapted_product", x, w, a, b, ids, scale)
    _want(ids, "ids", torch.int32)
    if ids.numel() != x.shape[0]:
        raise ValueError("ids: one per row of x is wanted")
    if scale is not None:
        _want(scale, "scale", torch.float32)
        if scale.numel() != a.shape[0]:
            raise ValueError("scale: one value per adapter is wanted")
    y = torch.empty((x.shape[0], w.shape[0]), dtype=x.dtype, device=x.device)
    _call("spgemm_adapted_product", x.device, _dense(x, "x"), _dense(w, "w"),
          _weights(a, "a"), _weights(b, "b"), ids.data_ptr(),
          scale.data_ptr() if scale is not None else None, _dense(y, "y"))
    return y


def grouped_status(stream=None):
    """Synchronise and raise SpgemmError if a device-side check of the calls above failed on the stream's device.

    Without a stream: the current one.  A call whose wait expired hands back meaningless values and says so only here:
    ask before results are handed on (after a training step, at the end of a request)."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.device(s.device):
        binding.spgemm_grouped_status(s.cuda_stream)
