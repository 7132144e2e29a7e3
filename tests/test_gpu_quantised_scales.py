"""Layers, gradients and widening of matrices in 8 bits whose scales differ from block to block, powers of two or any numbers; the
serving calls at sizes that the few-token kernels take."""
import numpy as np
import pytest

from _grouped_ref import SUM, rounding, transpose
from _quantised_ref import BLOCK, spread
from test_gpu_quantised import f64, grouping, layer_ref, normal, torch_type
from test_gpu_quantised_shapes import Layer, calls_of

pytestmark = pytest.mark.gpu


def scales(shape, seed, kind, about):
    """Between about / 8 and about * 8, powers of two or any numbers, either sign for these."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "powers":
        return torch.exp2(torch.randint(-3, 4, shape, device="cuda", generator=g).double()).float() * about
    r = torch.exp2(6 * torch.rand(shape, device="cuda", generator=g) - 3) * about
    return torch.where(torch.rand(shape, device="cuda", generator=g) < 0.3, -r, r)


def matrices(gpu_lib, groups, rows, cols, seed, kind, std):
    """Weights8 with scales of their own in padded rows and groups, and the numbers that they stand for in 64 bits."""
    import torch
    q = gpu_lib.quantise_weights(normal((groups, rows, cols), "bf16", seed=seed, std=std))
    room = torch.full((groups, rows + 2, -(-cols // 16) * 16 + 16), 99, dtype=torch.uint8, device="cuda")
    room[:, :rows, :cols] = q.values.view(torch.uint8)
    s = scales(q.scales.shape, seed + 1, kind, float(q.scales.median()))
    w = gpu_lib.Weights8(room.view(torch.float8_e4m3fn)[:, :rows, :cols], s, torch.bfloat16)
    return w, np.stack([f64(q.values[g].float()) * spread(f64(s[g]), BLOCK, rows, cols) for g in range(groups)])


def to_type(v, dtype):
    """Rounded to the type, f16 without its infinity, as widening does."""
    import torch
    v = torch.tensor(v).float()  # one rounding to 32 bits where a scale is no power of two
    if dtype == "f16":
        v = v.clamp(-65504, 65504)
    return f64(v.to(torch_type(dtype)))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["powers", "any"])
@pytest.mark.parametrize("groups,rows,cols", [(3, 300, 400), (2, 129, 257), (5, 128, 16)])
def test_matrices_are_widened_block_by_block(gpu_lib, dtype, kind, groups, rows, cols):
    w, want = matrices(gpu_lib, groups, rows, cols, 5, kind, 0.05)
    got = gpu_lib.dequantise(w, torch_type(dtype))
    assert np.array_equal(f64(got), to_type(want, dtype))


@pytest.mark.parametrize("tokens", [1, 6, 31, 64, 65])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["powers", "any"])
@pytest.mark.parametrize("d,hidden,n", [(304, 272, 400), (528, 144, 160)])
def test_layer(gpu_lib, d, hidden, n, kind, dtype, tokens):
    """Every block of both matrices with a scale that its neighbours do not have."""
    experts, top_k = 7, 3
    x, router = normal((tokens, d), dtype, seed=d), normal((experts, d), dtype, seed=1, std=d ** -0.5)
    up, u64 = matrices(gpu_lib, experts, 2 * hidden, d, 2, kind, d ** -0.5)
    down, d64 = matrices(gpu_lib, experts, n, hidden, 4, kind, hidden ** -0.5)
    few = tokens <= 64 and dtype != "f32"
    if not few:  # the matrices are widened to x's type first
        u64, d64 = to_type(u64, dtype), to_type(d64, dtype)
    want, ids, weights, err, gap = layer_ref(f64(x), f64(router), u64, d64, dtype, top_k, None, parts=2 if few else 1)
    assert gap > 1e-6
    out, gi, gw = gpu_lib.expert_layer(x, router, up, down, top_k)
    gpu_lib.grouped_status()
    assert np.array_equal(gi.cpu().numpy(), ids) and np.all(np.abs(f64(gw) - weights) <= 1e-5 * np.abs(weights))
    assert np.all(np.abs(f64(out) - want) <= err)
    # the bound is far from what a wrong block's scale would change (a factor of two or more of one of two to five blocks)
    assert np.median(err / np.abs(want)) < 0.2


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["powers", "any"])
@pytest.mark.parametrize("tokens,top_k,groups,d,n", [(40, 3, 6, 300, 272), (300, 2, 3, 520, 200)])
def test_gradients(gpu_lib, tokens, top_k, groups, d, n, kind, dtype):
    """Of the product of what the 8 bits stand for, held in dy's type on the way."""
    import torch
    r, ids = grouping(gpu_lib, tokens, top_k, groups, seed=tokens)
    q = gpu_lib.quantise_rows(normal((tokens, d), "bf16", seed=d))
    sx = scales((-(-d // BLOCK), tokens + 5), 8, kind, float(q.scales.median()))[:, :tokens].t()
    x8 = gpu_lib.Rows8(q.values, sx, torch.bfloat16)
    x = to_type(f64(q.values.float()) * spread(f64(sx), 1, tokens, d), dtype)
    w8, w = matrices(gpu_lib, groups, n, d, 3, kind, d ** -0.5)
    w = to_type(w, dtype)
    dy = normal((ids.size, n), dtype, seed=8)
    offsets, order, _ = transpose(ids, groups)
    g = f64(dy)
    g[int(offsets[-1]):] = 0
    dx, dw = gpu_lib.expert_product8_backward(dy, x8, w8, r)
    gpu_lib.grouped_status()
    wx, mx = np.zeros((tokens, d)), np.zeros((tokens, d))
    for grp in range(groups):
        p = slice(offsets[grp], offsets[grp + 1])
        tok = order[p] // top_k
        np.add.at(wx, tok, g[p] @ w[grp])
        np.add.at(mx, tok, np.abs(g[p]) @ np.abs(w[grp]))
        want, mag = g[p].T @ x[tok], np.abs(g[p]).T @ np.abs(x[tok])
        err = (len(tok) + 1) * SUM * mag
        assert np.all(np.abs(f64(dw[grp]) - want) <= err + rounding(dtype, want) + rounding(dtype, err))
    err = (n + top_k) * SUM * mx
    assert np.all(np.abs(f64(dx) - wx) <= err + rounding(dtype, wx) + rounding(dtype, err))


@pytest.mark.parametrize("tokens", [1, 20, 64])
def test_serving_form_in_its_own_kernels(gpu_lib, tokens):
    """The whole-layer call against the same layer out of separate calls, hidden rows of full 16 bytes in 8 bits."""
    import torch
    m, x = Layer(gpu_lib, hidden=144), normal((tokens, 256), "bf16", seed=7)
    out, ids, weights = m.serve(x)
    up, down = gpu_lib.dequantise(m.up8), gpu_lib.dequantise(m.down8)
    r = gpu_lib.route(x.float() @ m.router.float().t(), 2)
    assert torch.equal(r.ids, ids) and torch.allclose(r.weights, weights, rtol=1e-5, atol=0)
    want = gpu_lib.experts(x, up, down, r)
    # the separate calls round the hidden row (2^-8 of a term), both the result (2^-8 each); the sum of magnitudes is rounded too
    mag = gpu_lib.experts(x.abs(), up.abs(), down.abs(), r).float()
    assert torch.all((out.float() - want.float()).abs() <= 4 * 2.0 ** -8 * mag)


def test_calls_repeat_on_several_streams_at_once(gpu_lib):
    """Training and serving calls bit for bit, the layer of 8 bits in its few-token kernels."""
    import torch
    m = Layer(gpu_lib, hidden=144)
    x, dout = normal((60, 256), "bf16", seed=1), normal((60, 256), "bf16", seed=2)

    def calls():
        return [*calls_of(gpu_lib, m, x, dout), *m.serve(x), *m.serve(x[:1])]
    want = [t.clone() for t in calls()]
    sides, got = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(8):
        for s in sides:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(calls())
    torch.cuda.synchronize()
    for mine in got:
        assert all(torch.equal(p, q) for p, q in zip(mine, want))
    gpu_lib.grouped_status()
