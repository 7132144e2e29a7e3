"""The example layer: adapters, routing, experts and their gradients together, against the same layer
written out in 64 bits."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer(gpu_lib):
    path = os.path.join(os.path.dirname(os.path.dirname(__file__)), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens", [1, 7, 300])
def test_serve_against_64_bits(layer, gpu_lib, tokens):
    import torch
    m, x, ids = layer.make(tokens, dim=128, hidden=64, experts=8)
    out, r = layer.serve(m, x, ids)
    d = {k: v.double() for k, v in m.items()}
    h = x.double() @ d["w_in"].t()
    for t in range(tokens):
        if ids[t] >= 0:
            h[t] += d["b"][ids[t]] @ (d["a"][ids[t]] @ x[t].double())
    h16 = gpu_lib.adapted_product(x, m["w_in"], m["a"], m["b"], ids, m["scale"]).double()
    # one rounding of h (2^-8 of it) and one of the adapter's middle, of entries of order one
    assert (h16 - h).abs().max() <= 2.0 ** -8 * (h.abs().max() + 8)
    chosen, weights = r.ids.cpu().numpy(), r.weights.double()
    assert np.all(chosen[-1] == -1) and torch.all(out[-1] == h16[-1].to(out.dtype))
    want = h16.clone()
    for t in range(tokens):
        for j, e in enumerate(chosen[t]):
            if e >= 0:
                pre = d["w_up"][e] @ h16[t]
                mid = torch.nn.functional.silu(pre[:64]) * pre[64:]
                want[t] += weights[t, j] * (d["w_down"][e] @ mid)
    # three roundings to 16 bits of values of order one (the hidden row, the layer's answer, the sum)
    assert (out.double() - want).abs().max() <= 3 * 2.0 ** -8 * (want.abs().max() + 1)


def test_training_lowers_the_error_and_repeats(layer):
    m, x, _ = layer.make(500, dim=256, hidden=64, experts=8)
    target = (x.float() @ m["w_in"].float().t()).bfloat16()
    n, x2, _ = layer.make(500, dim=256, hidden=64, experts=8)
    first = [layer.train_step(m, x, target) for _ in range(6)]
    again = [layer.train_step(n, x2, target) for _ in range(6)]
    assert first[-1] < first[0] and all(b <= a for a, b in zip(first, first[1:]))
    assert first == again


def test_main_runs(layer):
    out, errors, pairs = layer.main(257)
    assert out.shape == (257, 1024) and errors[-1] < errors[0]
    assert np.array_equal(pairs.numpy(), pairs.numpy().T)
