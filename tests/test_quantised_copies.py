"""Copies of matrices in 8 bits, by copy and by pickle: what a call is handed are the addresses of the copy's own memory."""
import copy
import io
import pickle

import pytest
import torch

from sparse_gemm_irregular_gb300 import binding as b
from sparse_gemm_irregular_gb300 import quantised as Q


def saved(q):
    f = io.BytesIO()
    torch.save(q, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


COPIES = [copy.deepcopy, lambda q: pickle.loads(pickle.dumps(q)), saved]


def filled(rows, cols, count=1):
    made = Q._empty_rows(rows, cols, torch.bfloat16, "cpu", count)
    for q in made:
        q.values.view(torch.uint8).copy_(torch.arange(rows * cols).view(rows, cols) % 100)
        q.scales.copy_(torch.arange(rows * Q._blocks(cols)).view(rows, -1))
    return made


def check(q, was):
    s = b.spgemm_rows8.from_buffer_copy(q._packed())
    assert q.dtype is was.dtype and tuple(q.shape) == tuple(was.shape)
    assert s.values == q.values.data_ptr() and s.scales == q.scales.data_ptr()
    rows, cols = q.shape
    assert (s.rows, s.cols, s.scale_stride) == (rows, cols, rows)
    assert s.stride >= cols and s.stride % 16 == 0 and (rows == 1 or s.stride == q.values.stride(0))
    assert torch.equal(q.values.view(torch.uint8), was.values.view(torch.uint8)) and torch.equal(q.scales, was.scales)


@pytest.mark.parametrize("fresh", [True, False])
@pytest.mark.parametrize("copied", range(len(COPIES)))
@pytest.mark.parametrize("rows,cols", [(3, 200), (1, 16), (5, 128), (2, 300)])
def test_rows_that_a_call_made(rows, cols, copied, fresh):
    q, = filled(rows, cols)
    if fresh:  # the tensors were never asked for
        q = Q.Rows8._made(q._store, 0, rows, cols, q.dtype)
    c = COPIES[copied](q)
    at = b.spgemm_rows8.from_buffer_copy(c._packed()).values
    assert at != b.spgemm_rows8.from_buffer_copy(q._packed()).values
    check(c, q)
    c.values.view(torch.uint8).fill_(7)
    assert not (q.values.view(torch.uint8) == 7).all()
    check(copy.copy(q), q)  # shares the memory of what it was made from, and holds on to it
    assert b.spgemm_rows8.from_buffer_copy(copy.copy(q)._packed()).values == q.values.data_ptr()


@pytest.mark.parametrize("copied", range(len(COPIES)))
def test_one_of_two_that_share_an_allocation(copied):
    gate, up = filled(4, 200, 2)
    for q in (gate, up):
        check(COPIES[copied](q), q)


@pytest.mark.parametrize("copied", range(len(COPIES)))
def test_rows_of_given_tensors(copied):
    made, = filled(4, 200)
    given = made._with_scales(made.scales)  # as Rows8(values, scales) holds them
    check(COPIES[copied](given), given)


@pytest.mark.parametrize("copied", range(len(COPIES)))
@pytest.mark.parametrize("scales", [torch.ones(1, 2), torch.ones(1, 6)[:, ::3], torch.ones(2, 9).t()[3:4]])
def test_a_single_row_with_scales_of_any_stride(copied, scales):
    made, = filled(1, 200)
    given = made._with_scales(scales)
    check(COPIES[copied](given), given)


def test_no_copy_of_what_wants_a_gradient():
    made, = filled(4, 200)
    wants = made._with_scales(made.scales.clone().t().contiguous().t().requires_grad_())
    assert wants.requires_grad and copy.copy(wants).requires_grad
    with pytest.raises(RuntimeError, match="gradient"):
        copy.deepcopy(wants)


@pytest.mark.parametrize("copied", [0, 2])  # (plain pickle knows no tensor of 8-bit floats)
def test_matrices(copied):
    values = torch.arange(2 * 5 * 32).view(2, 5, 32).to(torch.uint8).view(torch.float8_e4m3fn)[..., :20]
    w = Q.Weights8._made(values, torch.ones(2, 1, 1), torch.bfloat16)
    c = COPIES[copied](w)
    s = b.spgemm_weights8.from_buffer_copy(c._packed())
    assert s.values == c.values.data_ptr() != w.values.data_ptr() and s.scales == c.scales.data_ptr()
    assert c.dtype is w.dtype and torch.equal(c.values.view(torch.uint8), w.values.view(torch.uint8))
    assert s.row_stride % 16 == 0
