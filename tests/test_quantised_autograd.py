"""Which matrices in 8 bits want a gradient, on the CPU: the calls go by it (an output of such an input tells of itself when a
gradient is asked of it)."""
import copy

import pytest
import torch

from sparse_gemm_irregular_gb300 import grouped as G
from sparse_gemm_irregular_gb300 import quantised as Q


def rows(given):
    q, = Q._empty_rows(4, 200, torch.bfloat16, "cpu")
    q.values.view(torch.uint8).fill_(56)
    q.scales.fill_(1.0)
    return q._with_scales(q.scales.clone().t().contiguous().t()) if given else q


def matrices():
    return Q.Weights8._made(torch.zeros(2, 5, 16, dtype=torch.float8_e4m3fn), torch.ones(2, 1, 1), torch.bfloat16)


@pytest.mark.parametrize("make", [lambda: rows(False), lambda: rows(True), matrices])
@pytest.mark.parametrize("part", ["values", "scales"])
def test_either_part_that_wants_a_gradient_is_seen(make, part):
    q = make()
    assert not q.requires_grad and not G._wants_gradient((q,), {}) and not G._wants_gradient((), {"x": q})
    t = getattr(q, part)
    t.requires_grad_()
    assert q.requires_grad and G._wants_gradient((q,), {}) and G._wants_gradient((), {"x": q})
    assert any(u is t for u in G._used((q,), {}))
    out = G._without_graph("a_call", torch.ones(3), G._used((q,), {}))
    with pytest.raises(RuntimeError, match="a_call takes no part in autograd"):
        out.sum().backward()
    made = G._without_graph("a_call", rows(False), G._used((q,), {}))
    assert made.requires_grad
    with pytest.raises(RuntimeError, match="a_call takes no part in autograd"):
        made.scales.sum().backward()


@pytest.mark.parametrize("part", ["values", "scales"])
def test_no_copy_of_rows_that_were_made_to_want_one(part):
    q = rows(False)
    getattr(q, part).requires_grad_()
    with pytest.raises(RuntimeError, match="gradient"):
        copy.deepcopy(q)
