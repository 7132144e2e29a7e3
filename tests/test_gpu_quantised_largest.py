"""Rows in 8 bits and their products where every token has 32 experts."""
import numpy as np
import pytest

from _grouped_ref import SUM
from _quantised_ref import held
from test_gpu_quantised import f64, normal, product_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_at_the_largest_choice(gpu_lib, dtype):
    """32 experts a token: every lane of a warp holds a position; rows go to all of them, those of no expert to none."""
    import torch
    tokens, experts, top_k, d, n = 70, 40, 32, 300, 200
    rng = np.random.default_rng(3)
    ids = np.stack([np.sort(rng.choice(experts, top_k, replace=False)) for _ in range(tokens)]).astype(np.int32)
    ids[5, 20:] = -1
    ids[-1] = -1
    r = gpu_lib.group_rows(torch.tensor(ids).cuda(), experts)
    x = normal((tokens, d), dtype, seed=1)
    w8 = gpu_lib.quantise_weights(normal((experts, n, d), "bf16", seed=2, std=d ** -0.5))
    want, mag = product_ref(held(f64(x)), f64(gpu_lib.dequantise(w8, torch.float32)), ids)
    x8 = gpu_lib.quantise_rows(x)
    y = gpu_lib.expert_product8(x8, w8, r, out_dtype=torch.float32)
    assert np.all(np.abs(f64(y) - want) <= (d + 4) * SUM * mag)
    assert torch.equal(gpu_lib.expert_product8(x, w8, r, out_dtype=torch.float32), y)  # brought to 8 bits on the way
    # the gradients: one 32-bit row per position, summed per token; x laid out for every position
    dy = normal((ids.size, n), dtype, seed=3)
    dx, dw = gpu_lib.expert_product8_backward(dy, x8, w8, r)
    one = gpu_lib.group_rows(torch.tensor(ids.reshape(-1)).cuda(), experts)  # a row per slot instead: the same products
    slots = gpu_lib.quantise_rows(x.repeat_interleave(top_k, 0))
    each, dw_one = gpu_lib.expert_product8_backward(dy, slots, w8, one)
    assert torch.equal(one.order, r.order) and torch.equal(dw, dw_one)
    u = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    total, parts = f64(each).reshape(tokens, top_k, d).sum(1), np.abs(f64(each)).reshape(tokens, top_k, d).sum(1)
    # each row once to the type there (u of it; f16's smallest step where it is below the normal range), the sum once here
    tiny = top_k * 2.0 ** -25 if dtype == "f16" else 0.0
    bound = u * parts / (1 - u) + tiny + top_k * 2.0 ** -24 * parts
    assert np.all(np.abs(f64(dx) - total) <= bound + u * (np.abs(total) + bound) + tiny)
    gpu_lib.grouped_status()
