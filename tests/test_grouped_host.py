"""The grouped-product entry points without a GPU: layouts of their structures, and calls that are
refused before any device work."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import sparse_gemm_irregular_gb300 as sg
from _grouped_ref import route, route_grad, scores, transpose
from sparse_gemm_irregular_gb300 import binding as b

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include")


def test_struct_layouts_match_the_header(tmp_path):
    if not shutil.which("gcc"):
        pytest.skip("no host C compiler")
    structs = [b.spgemm_dense, b.spgemm_weights, b.spgemm_grouping, b.spgemm_route_rule]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "spgemm.h"', "int main(void) {"]
    for cls in structs:
        lines.append('printf("%%zu\\n", sizeof(%s));' % cls.__name__)
        lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (cls.__name__, f) for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call(["gcc", "-std=c99", "-I", HEADER, str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)], text=True).split()]
    want = []
    for cls in structs:
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def test_packed_structures_have_the_layouts():
    from sparse_gemm_irregular_gb300 import grouped as G
    d = b.spgemm_dense.from_buffer_copy(G._pack_dense(16, 2, 3, 4, 1, 0))
    assert (d.data, d.rows, d.cols, d.stride, d.dtype) == (16, 2, 3, 4, 1)
    w = b.spgemm_weights.from_buffer_copy(G._pack_weights(16, 2, 3, 4, 5, 6, 2, 0))
    assert (w.data, w.groups, w.rows, w.cols, w.group_stride, w.row_stride, w.dtype) == (16, 2, 3, 4, 5, 6, 2)
    g = b.spgemm_grouping.from_buffer_copy(G._pack_grouping(6, 2, 3, 16, 32, 48))
    assert (g.slots, g.top_k, g.groups, g.offsets, g.order, g.position) == (6, 2, 3, 16, 32, 48)
    r = b.spgemm_route_rule.from_buffer_copy(G._pack_rule(1, 0, 3, 2, 1, True, 2.5, 0))
    assert (r.top_k, r.score, r.groups, r.groups_kept, r.group_score, r.renormalise, r.scale) == (1, 0, 3, 2, 1, 1, 2.5)
    for pack, cls in ((G._pack_dense, b.spgemm_dense), (G._pack_weights, b.spgemm_weights),
                      (G._pack_grouping, b.spgemm_grouping), (G._pack_rule, b.spgemm_route_rule)):
        assert pack.__self__.size == ctypes.sizeof(cls)


def dense(rows, cols, stride=None, dtype=1, data=16):
    return b.spgemm_dense(data, rows, cols, cols if stride is None else stride, dtype, 0)


def weights(groups, rows, cols, dtype=1):
    return b.spgemm_weights(16, groups, rows, cols, rows * cols, cols, dtype, 0)


def grouping(slots, top_k, groups):
    return b.spgemm_grouping(slots, top_k, groups, 16, 16, 16)


def rule(**kw):
    d = dict(top_k=2, score=0, groups=1, groups_kept=1, group_score=0, renormalise=1, scale=1.0, reserved=0) | kw
    return b.spgemm_route_rule(*[d[f] for f, _ in b.spgemm_route_rule._fields_])


R = ctypes.byref


@pytest.mark.parametrize("kw", [dict(top_k=0), dict(top_k=9), dict(score=2), dict(score=-1), dict(groups=3), dict(groups=0),
                                dict(groups=2, groups_kept=3), dict(groups_kept=0), dict(group_score=5),
                                dict(scale=float("nan")), dict(scale=float("inf"))])
def test_route_refuses_rules(kw):
    lib = sg.load()
    assert lib.spgemm_route(R(dense(4, 8)), R(rule(**kw)), None, 16, 16, 16, 16, 16, None) == -1
    assert lib.spgemm_route_backward(R(dense(4, 8)), R(rule(**kw)), 16, 16, R(dense(4, 8)), None) == -1


def test_route_refuses_matrices():
    lib = sg.load()
    ok = rule()
    for l in (dense(4, 0), dense(4, 1025), dense(-1, 8), dense(4, 8, stride=7), dense(4, 8, dtype=3), dense(4, 8, data=0)):
        assert lib.spgemm_route(R(l), R(ok), None, 16, 16, 16, 16, 16, None) == -1
    assert lib.spgemm_route(None, R(ok), None, 16, 16, 16, 16, 16, None) == -1
    assert lib.spgemm_route(R(dense(4, 8)), None, None, 16, 16, 16, 16, 16, None) == -1
    assert lib.spgemm_route(R(dense(4, 8)), R(ok), None, None, 16, 16, 16, 16, None) == -1
    assert lib.spgemm_route(R(dense(4, 8)), R(ok), None, 16, 16, None, 16, 16, None) == -1
    assert lib.spgemm_route(R(dense(1 << 31, 8)), R(ok), None, 16, 16, 16, 16, 16, None) == -5
    assert lib.spgemm_route_backward(R(dense(4, 8)), R(ok), 16, 16, R(dense(4, 7)), None) == -1
    assert lib.spgemm_route_backward(R(dense(4, 8)), R(ok), 16, 16, R(dense(4, 8, dtype=0)), None) == -1
    assert "gradient" in sg.spgemm_last_error()


def test_group_rows_refuses():
    lib = sg.load()
    assert lib.spgemm_group_rows(16, -1, 4, 16, 16, 16, None) == -1
    assert lib.spgemm_group_rows(16, 4, 0, 16, 16, 16, None) == -1
    assert lib.spgemm_group_rows(16, 4, 1025, 16, 16, 16, None) == -1
    assert lib.spgemm_group_rows(None, 4, 4, 16, 16, 16, None) == -1
    assert lib.spgemm_group_rows(16, 1 << 31, 4, 16, 16, 16, None) == -5


def test_debug_refuses_negative_polls():
    lib = sg.load()
    assert lib.spgemm_grouped_debug(0, -1) == -1
    assert lib.spgemm_grouped_debug(0, 0) == 0


def test_force_refuses_what_no_kernel_has():
    lib = sg.load()
    for args in ((8, 0, 0), (48, 0, 0), (512, 0, 0), (-16, 0, 0), (256, 2, 0), (256, -1, 0), (64, 0, 9), (64, 0, -1)):
        assert lib.spgemm_grouped_force(*args) == -1, args
    assert lib.spgemm_grouped_force(64, 0, 4) == 0 and lib.spgemm_grouped_force(0, 0, 0) == 0


def test_products_refuse():
    lib = sg.load()
    g, x, w, y = grouping(8, 2, 3), dense(4, 16), weights(3, 24, 16), dense(8, 24)
    call = lambda g=g, x=x, flag=0, w=w, y=y: lib.spgemm_grouped_product(R(g), R(x), flag, R(w), R(y), None)  # noqa: E731
    for kw in (dict(g=grouping(8, 2, 4)), dict(g=grouping(8, 0, 3)), dict(g=grouping(8, 33, 3)), dict(g=grouping(9, 2, 3)),
               dict(x=dense(4, 15)), dict(x=dense(5, 16)), dict(x=dense(4, 16, dtype=2)), dict(w=weights(3, 24, 17)),
               dict(w=weights(2, 24, 16)), dict(y=dense(8, 23)), dict(y=dense(7, 24)), dict(y=dense(8, 24, dtype=2)),
               dict(flag=1), dict(x=dense(4, 16, data=0))):
        assert call(**kw) == -1, kw
    back = lambda g=g, dy=y, x=x, w=w, dx=x, dw=w: lib.spgemm_grouped_product_backward(  # noqa: E731
        R(g), R(dy), R(x), R(w), R(dx), R(dw), None)
    for kw in (dict(dy=dense(8, 25)), dict(dy=dense(7, 24)), dict(dx=dense(4, 15)), dict(dx=dense(4, 16, dtype=0)),
               dict(dw=weights(3, 24, 8)), dict(x=dense(3, 16)), dict(w=weights(3, 24, 16, dtype=2))):
        assert back(**kw) == -1, kw


def test_gradients_of_groups_may_not_share_storage():
    lib = sg.load()
    g, x, w, dy = grouping(8, 2, 3), dense(4, 16), weights(3, 24, 16), dense(8, 24)
    for stride in (0, 16, 24 * 16 - 1):
        dw = weights(3, 24, 16)
        dw.group_stride = stride
        assert lib.spgemm_grouped_product_backward(R(g), R(dy), R(x), R(w), None, R(dw), None) == -1
        assert "overlap" in sg.spgemm_last_error()


def test_layers_refuse():
    lib = sg.load()
    g, x, up, down, out = grouping(8, 2, 3), dense(4, 16), weights(3, 48, 16), weights(3, 40, 24), dense(4, 40)
    call = lambda g=g, wt=16, x=x, up=up, down=down, out=out: lib.spgemm_experts(  # noqa: E731
        R(g), wt, R(x), R(up), R(down), R(out), None)
    for kw in (dict(wt=None), dict(up=weights(3, 47, 16)), dict(down=weights(3, 40, 23)), dict(out=dense(4, 41)),
               dict(out=dense(5, 40)), dict(x=dense(4, 16, dtype=0)), dict(g=grouping(8, 2, 2))):
        assert call(**kw) == -1, kw
    w, a, bb, y = dense(24, 16), weights(5, 4, 16), weights(5, 24, 4), dense(4, 24)
    call = lambda x=x, w=w, a=a, bb=bb, ids=16, y=y: lib.spgemm_adapted_product(  # noqa: E731
        R(x), R(w), R(a), R(bb), ids, None, R(y), None)
    for kw in (dict(ids=None), dict(w=dense(24, 15)), dict(a=weights(4, 4, 16)), dict(a=weights(5, 3, 16)),
               dict(bb=weights(5, 23, 4)), dict(y=dense(4, 23)), dict(y=dense(3, 24)), dict(a=weights(5, 4, 16, dtype=2)),
               dict(a=weights(1025, 4, 16), bb=weights(1025, 24, 4))):
        assert call(**kw) == -1, kw
    c = lambda g=g, y=dense(8, 40), o=out: lib.spgemm_combine(R(g), 16, R(y), R(o), None)  # noqa: E731
    for kw in (dict(y=dense(7, 40)), dict(y=dense(8, 39)), dict(o=dense(3, 40)), dict(g=grouping(8, 3, 3))):
        assert c(**kw) == -1, kw
    assert lib.spgemm_combine_backward(R(g), 16, R(out), R(dense(8, 40)), R(dense(8, 39)), 16, None) == -1
    assert lib.spgemm_combine_backward(R(g), 16, R(out), R(dense(8, 40)), R(dense(8, 40)), None, None) == -1


class Stand:
    """What the packing looks at, of a tensor on a GPU."""
    def __init__(self, shape, step):
        import torch
        self.shape, self.step, self.dtype, self.is_cuda = shape, step, torch.bfloat16, True

    def stride(self, i=None):
        return self.step if i is None else self.step[i]

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 64


@pytest.mark.parametrize("shape,step", [((16, 8), (0, 1)), ((16, 8), (7, 1)), ((2, 8), (1, 1)), ((5, 1), (0, 1)), ((5, 1), (0, 0))])
def test_rows_that_overlap_are_refused(shape, step):
    """A stride shorter than a row is not replaced by a longer one: that would read past the storage."""
    from sparse_gemm_irregular_gb300 import grouped as G
    with pytest.raises(ValueError, match="overlap"):
        G._dense(Stand(shape, step), "x")
    with pytest.raises(ValueError, match="overlap"):
        G._weights(Stand((3,) + shape, (64,) + step), "w")


def test_strides_arrive_as_they_are():
    from sparse_gemm_irregular_gb300 import grouped as G
    for shape, step, want in (((16, 8), (8, 1), 8), ((16, 8), (24, 1), 24), ((1, 8), (0, 1), 8), ((1, 8), (3, 1), 8), ((0, 8), (8, 1), 8),
                              ((5, 1), (1, 7), 1), ((5, 1), (9, 0), 9), ((5, 0), (1, 1), 1)):
        assert b.spgemm_dense.from_buffer_copy(G._dense(Stand(shape, step), "x")).stride == want
        w = b.spgemm_weights.from_buffer_copy(G._weights(Stand((3,) + shape, (0,) + step), "w"))  # one matrix for all groups
        assert (w.row_stride, w.group_stride) == (want, 0)


def test_sparse_matrices_of_a_routing_hold_no_id_out_of_range():
    """An id outside its range counts as none in the grouping: as a column it would lead the product astray."""
    import torch
    ids = np.array([[0, 5], [2, -1], [-7, 1]], np.int32)
    off, order, pos = transpose(np.where((ids < 3) & (ids >= 0), ids, -1), 3)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32)  # noqa: E731
    r = sg.Routing._made(i32(ids), torch.arange(6.0).view(3, 2), i32(off), i32(order), i32(pos))
    m = r.to_csr()
    assert (m.rows, m.cols, m.nnz) == (3, 3, 3)
    assert m.row_ptr.tolist() == [0, 1, 2, 3] and m.col.tolist() == [0, 2, 1] and m.val.tolist() == [0, 2, 5]
    t = r.transposed_csr()
    assert t.row_ptr.tolist() == [0, 1, 2, 3] and t.col.tolist() == [0, 2, 1] and t.val.tolist() == [0, 5, 2]


def test_tensors_of_different_devices_are_refused():
    """Every tensor of every call, before anything is allocated or launched."""
    import types
    here, there = (types.SimpleNamespace(device="cuda:%d" % i) for i in range(2))
    routing = lambda on: sg.Routing._made(on, on, on, on, on, rule=b"")  # noqa: E731
    calls = {
        sg.route: ([here, 2], dict(bias=here)), sg.route_backward: ([here, routing(here), here], {}),
        sg.group_rows: ([here, 2], dict(weights=here)), sg.expert_product: ([here, here, routing(here)], {}),
        sg.expert_product_backward: ([here, here, here, routing(here)], {}), sg.combine: ([here, routing(here)], {}),
        sg.combine_backward: ([here, here, routing(here)], {}), sg.experts: ([here, here, here, routing(here)], {}),
        sg.adapted_product: ([here, here, here, here, here, here], {})}
    for fn, (args, kw) in calls.items():
        for i in range(len(args)):
            if isinstance(args[i], int):
                continue
            bad = list(args)
            bad[i] = routing(there) if isinstance(args[i], sg.Routing) else there
            if len(args) - sum(isinstance(a, int) for a in args) + len(kw) > 1:
                with pytest.raises(ValueError, match="cuda:0.*cuda:1|cuda:1.*cuda:0"):
                    fn(*bad, **kw)
        for name in kw:
            with pytest.raises(ValueError, match="cuda:1"):
                fn(*args, **{name: there})


@pytest.mark.parametrize("shape", [(), (2, 3, 4)])
def test_ids_of_other_dimensions_are_refused(shape):
    import types

    import torch
    ids = types.SimpleNamespace(dtype=torch.int32, is_cuda=True, device="cuda:0", is_contiguous=lambda: True, dim=lambda: len(shape))
    with pytest.raises(ValueError, match="ids"):
        sg.group_rows(ids, 4)


def test_status_is_read_on_the_device_of_its_stream(monkeypatch):
    """Each device has a status word: the call looks at the stream's, not at the current one's."""
    import contextlib
    import types

    import torch
    at, seen = ["cuda:0"], []

    @contextlib.contextmanager
    def device(d):
        at.append(d)
        yield
        at.pop()

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(device="cuda:0", cuda_stream=7))
    monkeypatch.setattr(b, "spgemm_grouped_status", lambda s=0: seen.append((at[-1], s)))
    sg.grouped_status(types.SimpleNamespace(device="cuda:1", cuda_stream=9))
    sg.grouped_status()
    assert seen == [("cuda:1", 9), ("cuda:0", 7)]


# ---- the reference of the GPU tests, pinned by closed forms -------------------------------------
def test_reference_route_closed_forms():
    ids, w, _ = route(np.array([[0.0, np.log(2.0), np.log(4.0), -np.inf]]), 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[1 / 3, 2 / 3]])
    ids, w, _ = route(np.zeros((1, 6)), 3, renormalise=False)
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(w, 1 / 6)
    ids, _, _ = route(np.array([[5.0, 0.0, 3.0, 3.0]]), 2, groups=2, groups_kept=1, group_score="top2", score="sigmoid",
                      bias=np.zeros(4))
    assert ids.tolist() == [[2, 3]]
    ids, w, _ = route(np.full((1, 4), -np.inf), 2)
    assert ids.tolist() == [[-1, -1]] and w.tolist() == [[0, 0]]


def test_reference_gradient_against_differences():
    rng = np.random.default_rng(0)
    l, g = rng.standard_normal((4, 7)), rng.standard_normal((4, 3))
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, _, _ = route(l, 3, score=score, renormalise=renorm)
            d = route_grad(l, ids, g, score, renorm, 1.5)
            for e in range(7):
                v = []
                for sign in (1, -1):
                    x = l.copy()
                    x[:, e] += sign * 1e-6
                    w = np.take_along_axis(scores(x, score)[1], ids, 1)
                    v.append((1.5 * (w / w.sum(1, keepdims=True) if renorm else w) * g).sum(1))
                assert np.allclose(d[:, e], (v[0] - v[1]) / 2e-6, atol=1e-7)


def test_reference_transpose():
    off, order, pos = transpose(np.array([[1, 2], [-1, -1], [0, 2]]), 3)
    assert off.tolist() == [0, 1, 2, 4] and order.tolist() == [4, 0, 1, 5, -1, -1]
    assert pos.tolist() == [[1, 2], [-1, -1], [0, 3]]
