"""Routing, expert products and adapters on the GPU against the formulas in 64 bits (numpy), at the
sizes, masks, strides and types where they can go wrong.  Whole numbers have to be equal;
floating results stay inside bounds derived from the arithmetic: half a spacing of the output type
per rounding plus the rounding of the 32-bit sums over the absolute products."""
import numpy as np
import pytest

from _grouped_ref import SUM, TINY, U, product, rounding, route, route_grad, scores, transpose

pytestmark = pytest.mark.gpu

INF = float("inf")


def _t(dtype):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[dtype]


def _gen(seed):
    import torch
    return torch.Generator().manual_seed(seed)


def _normal(seed, *shape, dtype="bf16", std=1.0):
    import torch
    return (torch.randn(*shape, generator=_gen(seed)) * std).to(_t(dtype))


def _np(t):
    return t.detach().double().cpu().numpy()


def _random_ids(seed, tokens, groups, top_k, empty=()):
    """Ascending distinct ids per token, some slots and some tokens without a choice."""
    rng = np.random.default_rng(seed)
    allowed = [g for g in range(groups) if g not in empty]
    ids = np.full((tokens, top_k), -1, np.int32)
    for t in range(tokens):
        n = top_k if rng.random() < 0.8 else rng.integers(0, top_k + 1)
        n = min(n, len(allowed))
        p = 1.0 / (1.0 + np.arange(len(allowed)))
        ids[t, :n] = np.sort(rng.choice(allowed, n, replace=False, p=p / p.sum()))
    return ids


def _routing(gpu_lib, ids, groups, weights=None):
    import torch
    w = None if weights is None else torch.tensor(weights, dtype=torch.float32).cuda()
    return gpu_lib.group_rows(torch.tensor(ids).cuda(), groups, weights=w)


def _check_transpose(r, ids, groups):
    offsets, order, position = transpose(ids, groups)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.order.cpu().numpy(), order)
    assert np.array_equal(r.position.cpu().numpy(), position)


# ---- routing ---------------------------------------------------------------------------------
def _grid_logits(seed, tokens, experts, dtype):
    """Logits on a coarse grid (so that values are equal or well apart), with masked experts, a
    fully masked row, a row of the type's lowest value, NaN and +inf."""
    import torch
    l = (torch.randint(-12, 13, (tokens, experts), generator=_gen(seed)) * 0.25).to(_t(dtype))
    l[torch.rand(tokens, experts, generator=_gen(seed + 1)) < 0.1] = -INF
    if tokens > 4:
        l[1] = -INF
        l[2] = torch.finfo(_t(dtype)).min
        l[3, 0] = float("nan")
        l[4, experts - 1] = INF
        l[tokens - 1, 1:] = -INF
    return l


ROUTES = [
    (1, 1, 1, dict()),
    (1, 64, 6, dict()),
    (7, 33, 5, dict(score="softmax", renormalise=False)),
    (64, 8, 2, dict(score="sigmoid", scale=2.5)),
    (65, 128, 8, dict(score="softmax", groups=8, groups_kept=3)),
    (130, 96, 8, dict(score="sigmoid", groups=4, groups_kept=2)),
    (67, 12, 12, dict(score="softmax")),
    (66, 257, 32, dict(score="sigmoid", renormalise=False)),
    (40, 1000, 8, dict(score="softmax", groups=10, groups_kept=1)),
    (1500, 64, 6, dict(score="softmax")),
    # rows enough for few lanes per token
    (16413, 64, 6, dict(score="softmax", renormalise=False)),
    (9001, 120, 5, dict(score="sigmoid", groups=3, groups_kept=2)),
    (4199, 250, 8, dict(score="softmax", groups=5, groups_kept=3)),
    (2111, 512, 9, dict(score="softmax", groups=16, groups_kept=4)),
]


@pytest.mark.parametrize("tokens,experts,top_k,opt", ROUTES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_route_and_gradient(gpu_lib, tokens, experts, top_k, opt, dtype):
    import torch
    l = _grid_logits(tokens * experts, tokens, experts, dtype)
    ids, weights, _ = route(l.double().numpy(), top_k, **opt)
    r = gpu_lib.route(l.cuda(), top_k, **opt)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    # exp and the division are a few spacings off, the sum over `experts` terms one each
    tol = (8 + experts) * 2.0 ** -23
    assert np.allclose(_np(r.weights), weights, rtol=tol, atol=1e-37)
    _check_transpose(r, ids, experts)
    g = torch.randn(tokens, top_k, generator=_gen(5))
    d = gpu_lib.route_backward(l.cuda(), r, g.cuda())
    o = dict(score="softmax", renormalise=True, scale=1.0) | {k: v for k, v in opt.items() if k in ("score", "renormalise", "scale")}
    want = route_grad(l.double().numpy(), ids, g.numpy(), **o)
    _, s = scores(l.double().numpy(), o["score"])
    # size of the terms that are subtracted from each other: |g| (and |g| / sum) times s
    total = np.array([max(s[t, ids[t][ids[t] >= 0]].sum(), 1e-30) for t in range(tokens)])[:, None]
    size = o["scale"] * np.abs(g.numpy()).max() * top_k * (1 / total if o["renormalise"] else 1.0) * s * 2
    assert np.all(np.abs(_np(d) - want) <= rounding(dtype, want) + 4 * tol * size)
    gpu_lib.grouped_status()


@pytest.mark.parametrize("tokens,experts,top_k,opt", [
    (50, 64, 6, dict(score="sigmoid", groups=8, groups_kept=4, group_score="top2")),
    (33, 32, 4, dict(score="sigmoid")),
    (21, 40, 3, dict(score="softmax", groups=20, groups_kept=7, group_score="top2")),
    (20, 24, 4, dict(score="softmax", groups=3, groups_kept=2, group_score="max")),
])
def test_route_with_bias(gpu_lib, tokens, experts, top_k, opt):
    import torch
    for seed in range(6):
        l = _grid_logits(seed + 70, tokens, experts, "f32")
        bias = torch.randint(-60, 61, (experts,), generator=_gen(seed)) * 1e-3
        ids, weights, gap = route(l.double().numpy(), top_k, bias=bias.double().numpy(), **opt)
        if gap > 2e-6:  # compared values are equal or further apart than 32 bits can confuse
            break
    else:
        pytest.fail("no seed keeps the compared values apart")
    r = gpu_lib.route(l.cuda(), top_k, bias=bias.cuda(), **opt)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.allclose(_np(r.weights), weights, rtol=(8 + experts) * 2.0 ** -23, atol=1e-37)
    _check_transpose(r, ids, experts)


def test_route_top2_without_bias_and_strided_logits(gpu_lib):
    import torch
    big = _normal(3, 90, 200, dtype="f32")
    l = big[:, 17:17 + 64]
    ids, _, gap = route(l.double().numpy(), 4, groups=8, groups_kept=3, group_score="top2")
    assert gap > 1e-7
    r = gpu_lib.route(big.cuda()[:, 17:17 + 64], 4, groups=8, groups_kept=3, group_score="top2")
    assert np.array_equal(r.ids.cpu().numpy(), ids)


def test_route_gradient_against_differences(gpu_lib):
    import torch
    l = _normal(11, 9, 16, dtype="f32")
    g = _normal(12, 9, 3, dtype="f32")
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            r = gpu_lib.route(l.cuda(), 3, score=score, renormalise=renorm)
            d = _np(gpu_lib.route_backward(l.cuda(), r, g.cuda()))
            ids = r.ids.cpu().numpy()
            h = 1e-5
            for e in range(16):
                vals = []
                for sign in (1, -1):
                    x = l.double().numpy().copy()
                    x[:, e] += sign * h
                    _, s = scores(x, score)
                    w = np.take_along_axis(s, ids, 1)
                    vals.append(((w / w.sum(1, keepdims=True) if renorm else w) * g.double().numpy()).sum(1))
                # differences: h^2 / 6 of a third derivative below 10; the kernel: 32 bits of values below 10
                assert np.allclose(d[:, e], (vals[0] - vals[1]) / (2 * h), atol=2e-5, rtol=0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_a_single_renormalised_choice_has_no_gradient(gpu_lib, score, dtype):
    """Its weight is 1 whatever the logits: the gradient is 0, not a rounding error."""
    import torch
    l = _normal(4, 777, 53, dtype=dtype).cuda()
    r = gpu_lib.route(l, 1, score=score, scale=2.5)
    assert torch.all(r.weights == 2.5)
    assert torch.all(gpu_lib.route_backward(l, r, torch.randn(777, 1, device="cuda")) == 0)


def test_gradient_where_the_chosen_scores_are_tiny(gpu_lib):
    """Renormalised weights do not care how small the scores are, and neither do their gradients: the gradient of the
    scores themselves, a weight's divided by their sum, is past the 32-bit range here."""
    import torch
    # sigmoid: every logit near -88, scores near 1e-38
    l = (torch.rand(64, 16, generator=_gen(1)) * 2 - 88).float()
    g = _normal(2, 64, 3, dtype="f32")
    opt = dict(score="sigmoid", scale=50.0)
    r = gpu_lib.route(l.cuda(), 3, **opt)
    d = _np(gpu_lib.route_backward(l.cuda(), r, g.cuda()))
    want = route_grad(l.double().numpy(), r.ids.cpu().numpy(), g.numpy(), "sigmoid", True, 50.0)
    # terms of at most 50 |g|, a few roundings each; the scores, below 2^-126, keep 21 bits
    assert np.abs(d - want).max() <= 50 * np.abs(g.numpy()).max() * 4 * 2.0 ** -20
    # softmax: a bias prefers experts 86 below the best
    l = torch.rand(64, 16, generator=_gen(3)).float() - 86
    l[:, 0] = 0.0
    bias = torch.full((16,), 2.0)
    bias[0] = 0.0
    opt = dict(score="softmax", scale=100.0)
    r = gpu_lib.route(l.cuda(), 3, bias=bias.cuda(), **opt)
    ids = r.ids.cpu().numpy()
    assert (ids > 0).all()
    d = _np(gpu_lib.route_backward(l.cuda(), r, g.cuda()))
    want = route_grad(l.double().numpy(), ids, g.numpy(), "softmax", True, 100.0)
    # exp of -86 in 32 bits is 8 spacings off at most
    assert np.abs(d - want).max() <= 100 * np.abs(g.numpy()).max() * 4 * 2.0 ** -20


def test_route_empty_batch(gpu_lib):
    import torch
    r = gpu_lib.route(torch.empty(0, 16, device="cuda"), 2)
    assert r.ids.shape == (0, 2) and torch.all(r.offsets == 0)
    x = torch.empty(0, 32, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(16, 24, 32, device="cuda", dtype=torch.bfloat16)
    assert gpu_lib.expert_product(x, w, r).shape == (0, 24)
    dx, dw = gpu_lib.expert_product_backward(torch.empty(0, 24, device="cuda", dtype=torch.bfloat16), x, w, r)
    assert dx.shape == (0, 32) and torch.all(dw == 0)
    assert gpu_lib.experts(x, torch.ones(16, 48, 32, device="cuda", dtype=torch.bfloat16),
                           torch.ones(16, 32, 24, device="cuda", dtype=torch.bfloat16), r).shape == (0, 32)
    assert gpu_lib.adapted_product(x, w[0], w[:, :8], w[:, :, :8], torch.empty(0, dtype=torch.int32, device="cuda")).shape == (0, 24)


# ---- the transpose of given ids ----------------------------------------------------------------
@pytest.mark.parametrize("tokens,groups,top_k", [(1, 1, 1), (5, 3, 2), (2049, 7, 1), (3000, 300, 4), (4097, 1024, 1), (31, 40, 32)])
def test_group_rows(gpu_lib, tokens, groups, top_k):
    rng = np.random.default_rng(tokens)
    ids = rng.integers(-1, groups, (tokens, top_k)).astype(np.int32)  # repeats inside a token are allowed here
    _check_transpose(_routing(gpu_lib, ids, groups), ids, groups)


def test_group_rows_out_of_range_ids_are_reported(gpu_lib):
    ids = np.array([[0, 5, 2, -7, 1]], np.int32).T.copy()
    r = _routing(gpu_lib, ids, 3)
    _check_transpose(r, np.where((ids < 3) & (ids >= 0), ids, -1), 3)
    with pytest.raises(gpu_lib.SpgemmError) as e:
        gpu_lib.grouped_status()
    assert e.value.code == -6
    gpu_lib.grouped_status()  # reading clears it


def test_status_of_a_side_stream(gpu_lib):
    """An error set on one stream is told once, on whichever stream of the device asks next."""
    import torch
    side = torch.cuda.Stream()
    ids = torch.tensor([[0], [9]], dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    gpu_lib.group_rows(ids, 3, stream=side)
    with pytest.raises(gpu_lib.SpgemmError):
        gpu_lib.grouped_status(side)
    gpu_lib.grouped_status()
    gpu_lib.group_rows(ids, 3)
    torch.cuda.synchronize()
    with pytest.raises(gpu_lib.SpgemmError, match="range"):
        gpu_lib.grouped_status(side)
    gpu_lib.grouped_status(side)


# ---- products --------------------------------------------------------------------------------
# tokens, groups, top_k, d, n: one token; a group longer than a tile; empty groups; sizes that end
# inside every tile; rows that do not start on 16 bytes (odd d, odd n)
PRODUCTS = [
    (1, 1, 1, 8, 8), (1, 4, 2, 64, 128), (3, 5, 2, 72, 40), (17, 8, 4, 136, 264), (33, 64, 6, 256, 96),
    (300, 3, 2, 128, 72), (700, 5, 3, 328, 392), (1000, 2, 1, 1000, 136), (90, 7, 2, 61, 33), (260, 4, 4, 64, 640),
]


@pytest.mark.parametrize("tokens,groups,top_k,d,n", PRODUCTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_expert_product_and_gradients(gpu_lib, tokens, groups, top_k, d, n, dtype):
    import torch
    ids = _random_ids(tokens + d, tokens, groups, min(top_k, groups), empty=(1,) if groups > 2 else ())
    k = ids.shape[1]
    r = _routing(gpu_lib, ids, groups)
    offsets, order, position = transpose(ids, groups)
    x, w = _normal(1, tokens, d, dtype=dtype), _normal(2, groups, n, d, dtype=dtype)
    y = gpu_lib.expert_product(x.cuda(), w.cuda(), r)
    xd, wd = _np(x), _np(w)
    want, mag = product(xd, wd, ids, offsets, order)
    assert np.all(np.abs(_np(y) - want) <= rounding(dtype, want) + SUM * d * mag)
    assert torch.all(y[offsets[-1]:] == 0)
    full = gpu_lib.expert_product(x.cuda(), w.cuda(), r, out_dtype=torch.float32)
    assert np.all(np.abs(_np(full) - want) <= SUM * d * mag)
    # rows already in group order
    rows = torch.zeros(ids.size, d, dtype=x.dtype)
    rows[:offsets[-1]] = x[torch.tensor(order[:offsets[-1]] // k, dtype=torch.long)]
    again = gpu_lib.expert_product(rows.cuda(), w.cuda(), r, grouped=True)
    assert np.all(np.abs(_np(again) - want) <= rounding(dtype, want) + SUM * d * mag)
    # gradients
    dy = _normal(3, ids.size, n, dtype=dtype)
    dy[offsets[-1]:] = float("nan")  # rows without a slot take no part
    dx, dw = gpu_lib.expert_product_backward(dy.cuda(), x.cuda(), w.cuda(), r)
    dyd = _np(dy)
    wx, mx = np.zeros((tokens, d)), np.zeros((tokens, d))
    ww, mw, most = np.zeros((groups, n, d)), np.zeros((groups, n, d)), 1
    for g in range(groups):
        p = slice(offsets[g], offsets[g + 1])
        tok = order[p] // k
        np.add.at(wx, tok, dyd[p] @ wd[g])
        np.add.at(mx, tok, np.abs(dyd[p]) @ np.abs(wd[g]))
        ww[g], mw[g] = dyd[p].T @ xd[tok], np.abs(dyd[p]).T @ np.abs(xd[tok])
        most = max(most, len(tok))
    assert np.all(np.abs(_np(dx) - wx) <= rounding(dtype, wx) + SUM * (n + k) * mx)
    assert np.all(np.abs(_np(dw) - ww) <= rounding(dtype, ww) + SUM * most * mw)
    only = gpu_lib.expert_product_backward(dy.cuda(), x.cuda(), w.cuda(), r, need_dx=False)
    assert only[0] is None and torch.equal(only[1], dw)
    gpu_lib.grouped_status()


def _ordered_sums(x, w, ids, offsets, order):
    """y in 32 bits, added in the order of the columns by fused multiply-adds (the products of 16-bit values are
    exact in 64 bits, their sum with a 32-bit value is rounded to 64 bits 2^29 times finer than to 32)."""
    y = np.zeros((ids.size, w.shape[1]), np.float32)
    for g in range(w.shape[0]):
        p = slice(offsets[g], offsets[g + 1])
        rows = x[order[p] // ids.shape[1]]
        for k in range(x.shape[1]):
            y[p] = (y[p].astype(np.float64) + rows[:, k:k + 1] * w[g, None, :, k]).astype(np.float32)
    return y


# a few rows per group (rows gathered), many (laid out first), tiles of 256 rows shared by two blocks
@pytest.mark.parametrize("tokens,groups,top_k,d,n", [
    (1, 4, 2, 64, 128), (33, 64, 6, 256, 96), (300, 3, 2, 328, 72), (700, 5, 3, 500, 392), (2500, 2, 1, 264, 1200)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_16_bit_rows_are_the_ordered_sums_rounded_on_both_paths(gpu_lib, tokens, groups, top_k, d, n, dtype):
    """The matrix instructions add in another order, but not one element may be rounded another way for it: the
    gradient of the weights is formed from these rows in 32 bits."""
    import torch
    ids = _random_ids(tokens + d, tokens, groups, top_k)
    r = _routing(gpu_lib, ids, groups)
    offsets, order, _ = transpose(ids, groups)
    x, w = _normal(1, tokens, d, dtype=dtype), _normal(2, groups, n, d, dtype=dtype, std=d ** -0.5)
    want = torch.from_numpy(_ordered_sums(_np(x), _np(w), ids, offsets, order)).to(_t(dtype))
    y = gpu_lib.expert_product(x.cuda(), w.cuda(), r)
    assert torch.equal(y.cpu(), want)
    off = torch.nn.functional.pad(x, (1, 0)).cuda()[:, 1:]  # rows that do not start on 16 bytes
    assert torch.equal(gpu_lib.expert_product(off, w.cuda(), r), y)
    rows = torch.zeros(ids.size, d, dtype=x.dtype)
    rows[:offsets[-1]] = x[torch.tensor(order[:offsets[-1]] // ids.shape[1], dtype=torch.long)]
    assert torch.equal(gpu_lib.expert_product(rows.cuda(), w.cuda(), r, grouped=True), y)
    gpu_lib.grouped_status()


@pytest.mark.parametrize("n", [1, 3, 33, 36, 161])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_16_bit_rows_with_few_columns_beside(gpu_lib, n, dtype):
    """The last columns may have none beside them to tell how large a sum's parts were."""
    import torch
    r = _routing(gpu_lib, np.zeros((20000, 1), np.int32), 1)
    x, w = _normal(1, 20000, 1024, dtype=dtype).cuda(), _normal(2, 1, n, 1024, dtype=dtype, std=1 / 32).cuda()
    want = gpu_lib.expert_product(x.float(), w.float(), r).to(x.dtype)  # the CUDA cores add in order
    assert torch.equal(gpu_lib.expert_product(x, w, r), want)


def test_weights_with_any_group_stride(gpu_lib):
    """Groups need not lie a whole number of rows apart."""
    import torch
    r = _routing(gpu_lib, _random_ids(8, 700, 3, 2), 3)
    x, dy = _normal(1, 700, 64).cuda(), _normal(3, 1400, 40).cuda()
    flat = _normal(2, 3 * (40 * 72 + 8)).cuda()
    w = flat.as_strided((3, 40, 64), (40 * 72 + 8, 72, 1))
    assert torch.equal(gpu_lib.expert_product(x, w, r), gpu_lib.expert_product(x, w.contiguous(), r))
    assert torch.equal(gpu_lib.expert_product_backward(dy, x, w, r)[0], gpu_lib.expert_product_backward(dy, x, w.contiguous(), r)[0])
    overlap = flat.as_strided((3, 40, 64), (8, 72, 1))  # read only: groups may share storage
    assert torch.equal(gpu_lib.expert_product(x, overlap, r), gpu_lib.expert_product(x, overlap.contiguous(), r))


@pytest.mark.parametrize("tokens,groups,top_k,d,n,dtype", [
    (4096, 8, 4, 2048, 1024, "bf16"), (509, 16, 2, 1024, 776, "f16"), (900, 30, 3, 4000, 520, "bf16"), (2000, 6, 2, 1576, 792, "f16")])
def test_gradient_of_the_weights_in_the_chain(gpu_lib, tokens, groups, top_k, d, n, dtype):
    """dweights of product and weighted sum: as from 32-bit rows added in order and rounded once, to the rounding of
    the 32-bit scalar product, and not to that of the rows' 16 bits."""
    import torch
    ids = _random_ids(tokens, tokens, groups, top_k)
    r = _routing(gpu_lib, ids, groups)
    x, w = _normal(1, tokens, d, dtype=dtype).cuda(), _normal(2, groups, n, d, dtype=dtype, std=d ** -0.5).cuda()
    dout = _normal(3, tokens, n, dtype=dtype).cuda()
    _, dweights = gpu_lib.combine_backward(dout, gpu_lib.expert_product(x, w, r), r)
    rows = gpu_lib.expert_product(x.float(), w.float(), r).to(x.dtype).double()  # the CUDA cores add in order
    at = r.position.long()
    picked = torch.where(at[..., None] >= 0, rows[at.clamp(min=0)], 0.0)
    want = (picked * dout.double()[:, None]).sum(2)
    mag = (picked * dout.double()[:, None]).abs().sum(2)
    assert ((dweights.double() - want).abs() <= SUM * n * mag).all()
    assert float((dweights.double() - want).norm() / want.norm()) <= 2e-6


def test_product_gradients_against_differences(gpu_lib):
    import torch
    ids = _random_ids(3, 12, 3, 2)
    r = _routing(gpu_lib, ids, 3)
    offsets, order, _ = transpose(ids, 3)
    x, w, dy = _normal(1, 12, 16, dtype="f32"), _normal(2, 3, 8, 16, dtype="f32"), _normal(3, 24, 8, dtype="f32")
    dx, dw = gpu_lib.expert_product_backward(dy.cuda(), x.cuda(), w.cuda(), r)
    f = lambda a, b: (product(a, b, ids, offsets, order)[0] * _np(dy))[:offsets[-1]].sum()  # noqa: E731
    rng = np.random.default_rng(0)
    for _ in range(20):
        u, v = rng.standard_normal((12, 16)), rng.standard_normal((3, 8, 16))
        h = 1e-4  # the function is linear in each argument: differences have no error of their own
        dfx = (f(_np(x) + h * u, _np(w)) - f(_np(x) - h * u, _np(w))) / (2 * h)
        dfw = (f(_np(x), _np(w) + h * v) - f(_np(x), _np(w) - h * v)) / (2 * h)
        assert abs((_np(dx) * u).sum() - dfx) <= 1e-4 * (1 + abs(dfx))
        assert abs((_np(dw) * v).sum() - dfw) <= 1e-4 * (1 + abs(dfw))


def test_product_strides_and_streams(gpu_lib):
    """Column slices, padded group strides and a side stream."""
    import torch
    ids = _random_ids(8, 200, 6, 2)
    r = _routing(gpu_lib, ids, 6)
    offsets, order, _ = transpose(ids, 6)
    for pad in (8, 3):  # rows on 16-byte boundaries, and not
        xb, wb = _normal(1, 200, 128 + pad), _normal(2, 7, 100, 128 + pad)
        x, w = xb[:, :128], wb[:6, 4:84, :128]
        want, mag = product(_np(x), _np(w), ids, offsets, order)
        xc, wc = xb.cuda(), wb.cuda()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y = gpu_lib.expert_product(xc[:, :128], wc[:6, 4:84, :128], r, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert np.all(np.abs(_np(y) - want) <= rounding("bf16", want) + SUM * 128 * mag)


@pytest.mark.parametrize("d", [117, 120, 121, 3, 8])
def test_rows_that_end_with_the_storage(gpu_lib, d):
    """The last row has no padding behind it (its 16-byte pieces may not be read whole), others have NaN."""
    import torch
    ids = _random_ids(8, 700, 3, 2)
    r = _routing(gpu_lib, ids, 3)
    stride = (d + 7) // 8 * 8 + 8
    flat = torch.full((699 * stride + d,), float("nan"), dtype=torch.bfloat16).cuda()
    x = flat.as_strided((700, d), (stride, 1))
    dense = _normal(1, 700, d).cuda()
    x.copy_(dense)
    w, dy = _normal(2, 3, 40, (d + 7) // 8 * 8).cuda()[:, :, :d], _normal(3, 1400, 40).cuda()
    assert torch.equal(gpu_lib.expert_product(x, w, r), gpu_lib.expert_product(dense, w, r))
    got, want = gpu_lib.expert_product_backward(dy, x, w, r), gpu_lib.expert_product_backward(dy, dense.clone(), w, r)
    near = lambda a, b: ((a.double() - b.double()).abs() <= 2 * U["bf16"] * b.double().abs() + 1e-4).all()  # noqa: E731
    assert near(got[0], want[0]) and near(got[1], want[1])
    gpu_lib.grouped_status()


def _busy(torch):
    """Some tens of milliseconds of ordinary work on the current stream."""
    a = torch.ones(8192, 8192, device="cuda", dtype=torch.bfloat16)
    for _ in range(30):
        a @ a


def test_calls_on_a_side_stream_wait_for_no_other(gpu_lib):
    """Default weights are filled on the call's stream, not behind what the current one has under way."""
    import torch
    ids = _random_ids(8, 3000, 6, 2)
    ids_c, y = torch.tensor(ids).cuda(), _normal(1, 6000, 64).cuda()
    want = gpu_lib.combine(y, gpu_lib.group_rows(ids_c, 6))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):  # what a recycled block would hold
        for size in ((3000, 2), (6000,)):
            torch.full(size, 7.0, device="cuda")
    torch.full((3000, 2), 7.0, device="cuda")
    torch.cuda.synchronize()
    _busy(torch)
    r = gpu_lib.group_rows(ids_c, 6, stream=side)
    out = gpu_lib.combine(y, r, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # the current stream is still busy: nothing waited for it
    with torch.cuda.stream(side):
        assert torch.equal(out.clone(), want)
    torch.cuda.synchronize()


def test_outputs_of_a_side_stream_are_its_own(gpu_lib):
    """The current stream still writes to a tensor that is given up: its memory is not the side stream's output."""
    import torch
    ids = _random_ids(8, 2000, 6, 2)
    r = _routing(gpu_lib, ids, 6)
    x, w = _normal(1, 2000, 128).cuda(), _normal(2, 6, 512, 128).cuda()
    want = gpu_lib.expert_product(x, w, r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    _busy(torch)
    given_up = torch.zeros(4000, 512, device="cuda", dtype=torch.bfloat16)
    block = given_up.data_ptr()
    del given_up
    y = gpu_lib.expert_product(x, w, r, stream=side)
    side.synchronize()
    assert y.data_ptr() != block
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_inputs_of_a_side_stream_are_kept(gpu_lib):
    """An input that is given up after the call is not handed out while the side stream has yet to read it."""
    import torch
    ids = _random_ids(8, 2000, 6, 2)
    r = _routing(gpu_lib, ids, 6)
    x, w = _normal(1, 2000, 128).cuda(), _normal(2, 6, 512, 128).cuda()
    want = gpu_lib.expert_product(x, w, r)
    side = torch.cuda.Stream()
    mine = x.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _busy(torch)
    y = gpu_lib.expert_product(mine, w, r, stream=side)
    block = mine.data_ptr()
    del mine
    other = torch.full_like(x, float("nan"))
    assert other.data_ptr() != block
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_outputs_past_32_bit_offsets(gpu_lib):
    """More than 2^31 elements in y: rows at the start, around the boundary and at the end."""
    import torch
    tokens, k, d, n, groups = 270_000, 4, 64, 2048, 9
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.rand(tokens, groups, device="cuda", generator=g).topk(k, 1).indices.sort(1).values.int()
    r = gpu_lib.group_rows(ids, groups)
    x = torch.randn(tokens, d, device="cuda", generator=g).bfloat16()
    w = torch.randn(groups, n, d, device="cuda", generator=g).bfloat16()
    y = gpu_lib.expert_product(x, w, r)
    assert y.numel() > 1 << 31
    edge = (1 << 31) // n
    at = torch.tensor([0, 1, edge - 1, edge, edge + 1, tokens * k - 2, tokens * k - 1], device="cuda")
    slot = r.order[at].long()
    xr, wr = x[slot // k].double(), w[ids.reshape(-1)[slot].long()].double()
    want = torch.einsum("pd,pnd->pn", xr, wr)
    mag = torch.einsum("pd,pnd->pn", xr.abs(), wr.abs())
    assert ((y[at].double() - want).abs() <= U["bf16"] * want.abs() + SUM * d * mag).all()
    out = gpu_lib.combine(y, r)
    last = y[r.position[tokens - 1].long()].double()
    assert ((out[tokens - 1].double() - last.sum(0)).abs() <= U["bf16"] * last.sum(0).abs() + SUM * k * last.abs().sum(0)).all()
    gpu_lib.grouped_status()


def test_masked_values_stay_in_their_rows(gpu_lib):
    """A NaN or infinite row of x reaches only its own slots, in every product."""
    import torch
    ids = _random_ids(4, 150, 4, 2)
    r = _routing(gpu_lib, ids, 4)
    x, w = _normal(1, 150, 64), _normal(2, 4, 48, 64)
    clean = gpu_lib.expert_product(x.cuda(), w.cuda(), r)
    x[7], x[99, 3] = float("nan"), INF
    y = gpu_lib.expert_product(x.cuda(), w.cuda(), r)
    hit = torch.zeros(300, dtype=torch.bool)
    pos = r.position.cpu()
    for t in (7, 99):
        hit[pos[t][pos[t] >= 0].long()] = True
    assert torch.equal(y.cpu()[~hit], clean.cpu()[~hit])
    assert not torch.isfinite(y.cpu()[hit].float()).all(1).any()
    # the gradient of one group's weights sees its own rows only
    dy = _normal(3, 300, 48)
    _, dw = gpu_lib.expert_product_backward(dy.cuda(), x.cuda(), w.cuda(), r, need_dx=False)
    bad = {int(g) for t in (7, 99) for g in ids[t] if g >= 0}
    for g in range(4):
        assert torch.isfinite(dw[g].float()).all().item() == (g not in bad)


# ---- weighted sums -----------------------------------------------------------------------------
@pytest.mark.parametrize("tokens,groups,top_k,n", [(1, 1, 1, 8), (5, 4, 3, 40), (300, 16, 6, 264), (77, 9, 2, 33), (9, 32, 32, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_combine_and_gradients(gpu_lib, tokens, groups, top_k, n, dtype):
    import torch
    ids = _random_ids(tokens, tokens, groups, top_k)
    weights = np.random.default_rng(1).random(ids.shape).astype(np.float32)
    r = _routing(gpu_lib, ids, groups, weights)
    offsets, order, position = transpose(ids, groups)
    y, dout = _normal(1, ids.size, n, dtype=dtype), _normal(2, tokens, n, dtype=dtype)
    y[offsets[-1]:] = float("nan")
    out = gpu_lib.combine(y.cuda(), r)
    dy, dweights = gpu_lib.combine_backward(dout.cuda(), y.cuda(), r)
    yd, dd = _np(y), _np(dout)
    for t in range(tokens):
        js = [j for j in range(top_k) if position[t, j] >= 0]
        terms = np.array([weights[t, j] * yd[position[t, j]] for j in js]).reshape(len(js), n)
        want = terms.sum(0)
        assert np.all(np.abs(_np(out[t]) - want) <= rounding(dtype, want) + SUM * top_k * np.abs(terms).sum(0))
        for j in range(top_k):
            p = position[t, j]
            if p < 0:
                assert dweights[t, j] == 0
                continue
            assert abs(float(dweights[t, j]) - dd[t] @ yd[p]) <= SUM * n * (np.abs(dd[t]) @ np.abs(yd[p])) + 1e-30
            want = weights[t, j] * dd[t]
            assert np.all(np.abs(_np(dy[p]) - want) <= rounding(dtype, want) + 2.0 ** -24 * np.abs(want))
    assert torch.all(dy[offsets[-1]:] == 0)


@pytest.mark.parametrize("tokens,groups,top_k,d,n,dtype", [
    (4096, 8, 4, 2048, 1024, "bf16"), (509, 16, 2, 1024, 776, "f16"), (70, 5, 2, 264, 33, "bf16")])
def test_gradient_of_the_weights_from_32_bit_rows(gpu_lib, tokens, groups, top_k, d, n, dtype):
    """The chain with rows in 32 bits and everything else in 16: dweights of the unrounded product."""
    import torch
    ids = _random_ids(tokens, tokens, groups, top_k)
    weights = np.random.default_rng(1).random(ids.shape).astype(np.float32)
    r = _routing(gpu_lib, ids, groups, weights)
    x, w = _normal(1, tokens, d, dtype=dtype).cuda(), _normal(2, groups, n, d, dtype=dtype, std=d ** -0.5).cuda()
    dout = _normal(3, tokens, n, dtype=dtype).cuda()
    y = gpu_lib.expert_product(x, w, r, out_dtype=torch.float32)
    out = gpu_lib.combine(y, r, out_dtype=x.dtype)
    dy, dweights = gpu_lib.combine_backward(dout, y, r)
    assert out.dtype == dy.dtype == x.dtype and dweights.dtype == torch.float32
    same, _ = gpu_lib.combine_backward(dout, y.to(x.dtype), r)
    assert torch.equal(dy, same)
    want = torch.zeros(tokens, top_k, dtype=torch.float64, device="cuda")
    for g in range(groups):
        at = (torch.tensor(ids).cuda() == g).nonzero()
        want[at[:, 0], at[:, 1]] = (dout[at[:, 0]].double() * (x[at[:, 0]].double() @ w[g].double().t())).sum(1)
    assert float((dweights.double() - want).norm() / want.norm()) <= 1e-5
    dx, dw = gpu_lib.expert_product_backward(dy, x, w, r)  # the rest of the chain takes it
    assert dx.dtype == dw.dtype == x.dtype


@pytest.mark.parametrize("dout_type,y_type", [("f32", "bf16"), ("bf16", "f16"), ("f16", "f32")])
def test_combine_backward_of_mixed_types(gpu_lib, dout_type, y_type):
    r = _routing(gpu_lib, _random_ids(3, 50, 4, 2), 4)
    dout, y = _normal(1, 50, 40, dtype=dout_type).cuda(), _normal(2, 100, 40, dtype=y_type).cuda()
    dy, dweights = gpu_lib.combine_backward(dout, y, r)
    ref_dy, ref = gpu_lib.combine_backward(dout.float(), y.float(), r)
    assert dy.dtype == dout.dtype and (dy == ref_dy.to(dout.dtype)).all()
    mag = (dout.float().abs().amax() * y.float().abs().amax()).item() * 40
    assert (dweights - ref).abs().max() <= SUM * 40 * mag


def test_gradient_of_the_weights_without_columns(gpu_lib):
    """A scalar product of no terms is 0, whatever the output's memory held."""
    import torch
    r = _routing(gpu_lib, _random_ids(3, 50, 4, 2), 4)
    dout, y = torch.empty(50, 0, device="cuda"), torch.empty(100, 0, device="cuda")
    for _ in range(3):
        torch.full((50, 2), 7.0, device="cuda")  # the block that the output gets
        dy, dweights = gpu_lib.combine_backward(dout, y, r)
        assert dy.shape == (100, 0) and torch.all(dweights == 0)


# ---- the gated layer -----------------------------------------------------------------------------
@pytest.mark.parametrize("tokens,groups,top_k,d,hidden,n", [
    (1, 1, 1, 8, 8, 8), (1, 16, 4, 64, 96, 64), (9, 8, 3, 72, 40, 136), (200, 6, 2, 128, 64, 200), (700, 4, 2, 264, 328, 128),
    (64, 64, 6, 256, 128, 256), (31, 5, 2, 37, 19, 41), (600, 3, 3, 512, 256, 512),
])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_experts(gpu_lib, tokens, groups, top_k, d, hidden, n, dtype):
    ids = _random_ids(tokens + 1, tokens, groups, top_k, empty=(0,) if groups > 4 else ())
    weights = np.random.default_rng(1).random(ids.shape).astype(np.float32)
    r = _routing(gpu_lib, ids, groups, weights)
    x = _normal(1, tokens, d, dtype=dtype)
    up, down = _normal(2, groups, 2 * hidden, d, dtype=dtype, std=d ** -0.5), _normal(3, groups, n, hidden, dtype=dtype, std=hidden ** -0.5)
    out = _np(gpu_lib.experts(x.cuda(), up.cuda(), down.cuda(), r))
    xd, ud, dd = _np(x), _np(up), _np(down)
    want, tol = np.zeros((tokens, n)), np.zeros((tokens, n))
    for t in range(tokens):
        for j in range(top_k):
            g = ids[t, j]
            if g < 0:
                continue
            pre, mag = ud[g] @ xd[t], np.abs(ud[g]) @ np.abs(xd[t])
            gate, u = pre[:hidden], pre[hidden:]
            sig = 1 / (1 + np.exp(-gate))
            h = gate * sig * u
            # errors of the two products through silu (slope at most 1.1), exp and division, one rounding of h
            eh = SUM * d * (1.1 * np.abs(u) * mag[:hidden] + np.abs(gate * sig) * mag[hidden:]) + (U[dtype] + 2.0 ** -20) * np.abs(h)
            want[t] += weights[t, j] * (dd[g] @ h)
            tol[t] += weights[t, j] * (np.abs(dd[g]) @ (eh + SUM * (hidden + top_k) * np.abs(h)))
    small = TINY[dtype] * hidden  # roundings of h below the type's normal range
    assert np.all(np.abs(out - want) <= rounding(dtype, want) + 1.01 * tol + small)
    gpu_lib.grouped_status()


@pytest.mark.parametrize("tokens,groups,top_k,d,hidden", [(1594, 65, 4, 448, 504), (700, 30, 3, 192, 72), (2500, 9, 2, 1000, 136)])
def test_no_wait_runs_out_over_many_calls(gpu_lib, tokens, groups, top_k, d, hidden):
    """Groups of very different sizes, so that a slice is dealt over fewer copies than there are warps to
    issue them, call after call without a pause: every call gives the first one's bits and no wait expires."""
    import torch
    ids = _random_ids(tokens, tokens, groups, top_k)
    weights = np.random.default_rng(1).random(ids.shape).astype(np.float32)
    r = _routing(gpu_lib, ids, groups, weights)
    x = _normal(1, tokens, d).cuda()
    up, down = _normal(2, groups, 2 * hidden, d, std=d ** -0.5).cuda(), _normal(3, groups, d, hidden, std=hidden ** -0.5).cuda()
    dy = _normal(4, ids.size, 2 * hidden).cuda()
    first = gpu_lib.experts(x, up, down, r)
    dx, dw = gpu_lib.expert_product_backward(dy, x, up, r)
    for _ in range(40):
        out = gpu_lib.experts(x, up, down, r)
        again = gpu_lib.expert_product_backward(dy, x, up, r)
        assert torch.equal(out, first) and torch.equal(again[0], dx) and torch.equal(again[1], dw)
    outs = [gpu_lib.experts(x, up, down, r) for _ in range(20)]
    assert all(torch.equal(o, first) for o in outs)
    gpu_lib.grouped_status()


@pytest.mark.parametrize("hidden", [8, 9])  # on the tensor cores, on the CUDA cores
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_range_of_the_hidden_row(gpu_lib, hidden, dtype):
    """It is held in x's type: in f16 a value past 65504 is infinite and reaches out, in bf16 it is not."""
    import torch
    ids = np.zeros((20, 1), np.int32)
    r = _routing(gpu_lib, ids, 1)
    x = torch.ones(20, 16, dtype=_t(dtype))
    x[::2] *= 0.875
    up = torch.zeros(1, 2 * hidden, 16, dtype=_t(dtype))
    up[:, :hidden] = 4.0  # gate 64 (56): silu(64) = 64
    up[:, hidden:] = 70.0  # up 1120 (980): hidden value 71680 (54880)
    down = torch.full((1, 24, hidden), 2.0 ** -6, dtype=_t(dtype))
    out = _np(gpu_lib.experts(x.cuda(), up.cuda(), down.cuda(), r))
    want = np.where(np.arange(20) % 2 == 0, 54880.0, 71680.0)[:, None] * hidden / 64
    loud = np.abs(want) * 64 / hidden > 65504
    if dtype == "f16":
        assert np.all(np.isinf(out[loud[:, 0]]))
        want, out = want[~loud[:, 0]], out[~loud[:, 0]]
    assert np.all(np.abs(out - want) <= 2.02 * U[dtype] * want)  # roundings of the hidden value and of out


@pytest.mark.parametrize("rank", [8, 7])  # on the tensor cores, on the CUDA cores
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_range_of_the_row_between_an_adapters_products(gpu_lib, rank, dtype):
    """On the tensor cores it is held in x's type (f16: infinite past 65504), on the CUDA cores in 32 bits."""
    import torch
    ids = torch.arange(20, dtype=torch.int32) % 2
    x, w = torch.ones(20, 64, dtype=_t(dtype)), torch.ones(24, 64, dtype=_t(dtype))
    a = torch.full((2, rank, 64), 1100.0, dtype=_t(dtype))  # 70400, in bf16 from 1104: 70656
    a[1] = 500.0
    b = torch.full((2, 24, rank), 2.0 ** -4, dtype=_t(dtype))
    y = _np(gpu_lib.adapted_product(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda()))
    want = 64 + np.where(np.arange(20) % 2 == 0, 64 * float(a[0, 0, 0]), 32000.0)[:, None] * rank / 16
    if dtype == "f16" and rank == 8:
        assert np.all(np.isinf(y[::2]))
        want, y = want[1::2], y[1::2]
    assert np.all(np.abs(y - want) <= 2.02 * U[dtype] * want)


# ---- adapters ------------------------------------------------------------------------------------
@pytest.mark.parametrize("tokens,adapters,rank,d,n", [
    (1, 1, 8, 64, 64), (1, 3, 16, 128, 72), (5, 2, 8, 40, 136), (64, 48, 16, 256, 264), (300, 3, 64, 512, 128),
    (777, 5, 24, 200, 520), (140, 4, 128, 96, 64), (33, 4, 200, 64, 48), (50, 3, 7, 37, 21), (260, 1024, 8, 64, 64),
])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("mixed", [False, True])
def test_adapted_product(gpu_lib, tokens, adapters, rank, d, n, dtype, mixed):
    import torch
    rng = np.random.default_rng(tokens)
    if mixed:  # any order of adapters
        ids = rng.integers(-1, adapters, tokens).astype(np.int32)
    else:  # runs of requests, one of them without an adapter
        ids = np.sort(rng.integers(-1, adapters, tokens)).astype(np.int32)
    x, w = _normal(1, tokens, d, dtype=dtype), _normal(2, n, d, dtype=dtype, std=d ** -0.5)
    a, b = _normal(3, adapters, rank, d, dtype=dtype, std=d ** -0.5), _normal(4, adapters, n, rank, dtype=dtype, std=0.3)
    scale = torch.rand(adapters, generator=_gen(9)) + 0.5
    y = _np(gpu_lib.adapted_product(x.cuda(), w.cuda(), a.cuda(), b.cuda(), torch.tensor(ids).cuda(), scale.cuda()))
    xd, wd, ad, bd = _np(x), _np(w), _np(a), _np(b)
    want, tol = xd @ wd.T, SUM * (d + rank) * (np.abs(xd) @ np.abs(wd).T)
    for t in range(tokens):
        if ids[t] >= 0:
            g, s = ids[t], float(scale[ids[t]])
            v, mv = ad[g] @ xd[t], np.abs(ad[g]) @ np.abs(xd[t])
            want[t] += s * (bd[g] @ v)
            # v is rounded to the inputs' type once between the two small products
            tol[t] += s * (np.abs(bd[g]) @ (SUM * (d + rank) * mv + (U[dtype] + 2.0 ** -22) * np.abs(v)))
    assert np.all(np.abs(y - want) <= rounding(dtype, want) + 1.01 * tol)
    gpu_lib.grouped_status()


def test_adapters_without_scale_and_with_nan_rows(gpu_lib):
    """No scale means ones; a row of NaN reaches no other row; unused adapters may hold anything."""
    import torch
    ids = torch.tensor([0, 2, -1, 2, 0, 1] * 20, dtype=torch.int32)
    x, w = _normal(1, 120, 64), _normal(2, 48, 64, std=0.1)
    a, b = _normal(3, 4, 16, 64, std=0.1), _normal(4, 4, 48, 16)
    a[3], b[3] = float("nan"), float("nan")
    y = gpu_lib.adapted_product(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda())
    ones = gpu_lib.adapted_product(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(), torch.ones(4).cuda())
    assert torch.equal(y, ones) and torch.isfinite(y.float()).all()
    x[5] = float("nan")
    z = gpu_lib.adapted_product(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda())
    keep = torch.arange(120) != 5
    assert torch.equal(z.cpu()[keep], y.cpu()[keep]) and torch.isnan(z[5].float()).all()


def test_results_repeat_bit_for_bit(gpu_lib):
    import torch
    l = _normal(1, 3000, 32, dtype="f32").cuda()
    x, w = _normal(2, 3000, 128).cuda(), _normal(3, 32, 96, 128).cuda()
    first = None
    for _ in range(3):
        r = gpu_lib.route(l, 4)
        y = gpu_lib.expert_product(x, w, r)
        out = gpu_lib.combine(y, r)
        dy, dwt = gpu_lib.combine_backward(out, y, r)
        dx, dw = gpu_lib.expert_product_backward(dy, x, w, r)
        now = [r.ids, r.weights, r.order, y, out, dy, dwt, dx, dw]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("tokens", [6, 700])
def test_calls_replay_as_a_graph(gpu_lib, tokens):
    """A layer of all calls, captured and replayed on new inputs: the bits of the direct calls, again and again."""
    import torch
    experts, top_k, d, hidden = 12, 3, 256, 128
    w_in, a, b = _normal(1, d, d, std=1 / 16).cuda(), _normal(2, 4, 16, d, std=1 / 16).cuda(), _normal(3, 4, d, 16).cuda()
    scale, bias = torch.rand(4, generator=_gen(4)).cuda(), torch.zeros(experts).cuda()
    router = _normal(5, experts, d, std=1 / 16).cuda()
    up, down = _normal(6, experts, 2 * hidden, d, std=1 / 16).cuda(), _normal(7, experts, d, hidden, std=1 / 11).cuda()
    w = _normal(8, experts, d, d, std=1 / 16).cuda()

    def layer(x, which):
        h = gpu_lib.adapted_product(x, w_in, a, b, which, scale)
        l = (h @ router.t()).float()
        r = gpu_lib.route(l, top_k, bias=bias, score="sigmoid", groups=4, groups_kept=2, group_score="top2")
        out = gpu_lib.experts(h, up, down, r)
        y = gpu_lib.expert_product(h, w, r)
        s = gpu_lib.combine(y, r)
        dy, dweights = gpu_lib.combine_backward(out, y, r)
        dx, dw = gpu_lib.expert_product_backward(dy, h, w, r)
        dl = gpu_lib.route_backward(l, r, dweights)
        again = gpu_lib.group_rows(r.ids, experts)
        return [h, r.ids, r.weights, r.order, out, y, s, dy, dweights, dx, dw, dl, again.position]

    x, which = _normal(9, tokens, d).cuda(), torch.randint(-1, 4, (tokens,), generator=_gen(10)).int().cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, which)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = layer(x, which)
    for seed in (11, 12, 11):
        x.copy_(_normal(seed, tokens, d))
        which.copy_(torch.randint(-1, 4, (tokens,), generator=_gen(seed)).int())
        for _ in range(3):
            g.replay()
        got = [t.clone() for t in held]
        want = layer(x, which)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    gpu_lib.grouped_status()


def test_no_silent_end_of_a_graph(gpu_lib):
    """An input that wants a gradient does not lose it without a word."""
    import torch
    l = _normal(1, 6, 8, dtype="f32").cuda().requires_grad_()
    r = gpu_lib.route(l, 2)
    x, w = _normal(2, 6, 16).cuda().requires_grad_(), _normal(3, 8, 24, 16).cuda()
    up, down = _normal(6, 8, 48, 16).cuda(), _normal(7, 8, 24, 24).cuda()
    a, b = _normal(8, 3, 4, 16).cuda(), _normal(9, 3, 24, 4).cuda().requires_grad_()
    which = torch.zeros(6, dtype=torch.int32, device="cuda")
    plain = gpu_lib.route(l.detach(), 2)
    y = gpu_lib.expert_product(x, w, plain)
    for name, out in (("route", r.weights), ("expert_product", y), ("combine", gpu_lib.combine(y, plain)),
                      ("combine", gpu_lib.combine(y.detach(), r)), ("experts", gpu_lib.experts(x, up, down, plain)),
                      ("adapted_product", gpu_lib.adapted_product(x.detach(), w[0], a, b, which))):
        with pytest.raises(RuntimeError, match=name + " takes no part in autograd"):
            (out.float().sum() * 2).backward()
    assert torch.equal(r.ids, plain.ids) and torch.equal(r.weights, plain.weights)
    with torch.no_grad():
        assert not gpu_lib.expert_product(x, w, plain).requires_grad
    assert not gpu_lib.expert_product(x.detach(), w, plain).requires_grad
    # the same parameters, their gradients formed by hand
    dy, _ = gpu_lib.combine_backward(_normal(4, 6, 24).cuda(), y.detach(), plain)
    x.grad = gpu_lib.expert_product_backward(dy, x.detach(), w, plain)[0]
    assert x.grad.shape == x.shape


def test_routing_as_sparse_matrices(gpu_lib):
    """The choice and its transpose as CSR, multiplied by the library's SpGEMM: how often two experts
    serve the same token."""
    ids = _random_ids(5, 400, 12, 3)
    r = _routing(gpu_lib, ids, 12)
    rp, col, val = gpu_lib.multiply(r.transposed_csr(), r.to_csr()).to_host()
    got = np.zeros((12, 12))
    for i in range(12):
        got[i, col[rp[i]:rp[i + 1]]] = val[rp[i]:rp[i + 1]]
    one = np.zeros((400, 12))
    for t in range(400):
        one[t, ids[t][ids[t] >= 0]] = 1
    assert np.array_equal(got, one.T @ one)


def test_refusals(gpu_lib):
    import torch
    l = torch.zeros(4, 8, device="cuda")
    for kw in (dict(top_k=9), dict(top_k=0), dict(top_k=2, groups=3), dict(top_k=2, groups=2, groups_kept=3),
               dict(top_k=2, scale=INF)):
        with pytest.raises(gpu_lib.SpgemmError) as e:
            gpu_lib.route(l, **kw)
        assert e.value.code == -1
    with pytest.raises(ValueError):
        gpu_lib.route(l, 2, score="relu")
    with pytest.raises(TypeError):
        gpu_lib.route(l.double(), 2)
    with pytest.raises(ValueError):
        gpu_lib.route(l.t(), 2)
    r = gpu_lib.route(l, 2)
    x, w = torch.zeros(4, 16, device="cuda"), torch.zeros(8, 24, 16, device="cuda")
    with pytest.raises(gpu_lib.SpgemmError):
        gpu_lib.expert_product(x, w[:7], r)
    with pytest.raises(gpu_lib.SpgemmError):
        gpu_lib.expert_product(x, w.half(), r)
    with pytest.raises(gpu_lib.SpgemmError):
        gpu_lib.expert_product(x[:3], w, r)
    with pytest.raises(gpu_lib.SpgemmError):
        gpu_lib.experts(x, w, w, r)
    with pytest.raises(gpu_lib.SpgemmError):
        gpu_lib.combine(torch.zeros(7, 24, device="cuda"), r)
    with pytest.raises(ValueError):
        gpu_lib.adapted_product(x, w[0], w[:, :2], w[:, :, :2], torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.expert_product(x.cpu(), w, r)
    with pytest.raises(ValueError):
        gpu_lib.route_backward(l, gpu_lib.group_rows(r.ids, 8), torch.zeros(4, 2, device="cuda"))


def test_expanded_and_overlapping_inputs_are_refused(gpu_lib):
    """Every matrix of every call: rows that share storage are refused before any device work, copies are taken."""
    import torch
    l = _normal(1, 6, 8, dtype="f32").cuda()
    r = gpu_lib.route(l, 2)
    x, w = _normal(2, 6, 16).cuda(), _normal(3, 8, 24, 16).cuda()
    y, dout = _normal(4, 12, 24).cuda(), _normal(5, 6, 24).cuda()
    up, down = _normal(6, 8, 48, 16).cuda(), _normal(7, 8, 24, 24).cuda()
    a, b, which = _normal(8, 3, 4, 16).cuda(), _normal(9, 3, 24, 4).cuda(), torch.zeros(6, dtype=torch.int32, device="cuda")
    wide = lambda t: t[..., :1, :].expand(t.shape)  # noqa: E731  one row for all
    slide = lambda t: t.reshape(-1).as_strided(t.shape, t.stride()[:-2] + (t.shape[-1] - 1, 1))  # noqa: E731
    for f in (wide, slide):
        for call in (lambda: gpu_lib.route(f(l), 2), lambda: gpu_lib.route_backward(f(l), r, torch.zeros(6, 2, device="cuda")),
                     lambda: gpu_lib.expert_product(f(x), w, r), lambda: gpu_lib.expert_product(x, f(w), r),
                     lambda: gpu_lib.expert_product_backward(f(y), x, w, r), lambda: gpu_lib.expert_product_backward(y, f(x), w, r),
                     lambda: gpu_lib.expert_product_backward(y, x, f(w), r), lambda: gpu_lib.combine(f(y), r),
                     lambda: gpu_lib.combine_backward(f(dout), y, r), lambda: gpu_lib.combine_backward(dout, f(y), r),
                     lambda: gpu_lib.experts(f(x), up, down, r), lambda: gpu_lib.experts(x, f(up), down, r),
                     lambda: gpu_lib.experts(x, up, f(down), r), lambda: gpu_lib.adapted_product(f(x), w[0], a, b, which),
                     lambda: gpu_lib.adapted_product(x, f(w[0]), a, b, which), lambda: gpu_lib.adapted_product(x, w[0], f(a), b, which),
                     lambda: gpu_lib.adapted_product(x, w[0], a, f(b), which)):
            with pytest.raises(ValueError, match="overlap"):
                call()
    # the gradient of a sum over tokens is such a tensor: copied, it is taken; one matrix for all groups is taken as it is
    got = gpu_lib.combine_backward(wide(dout).contiguous(), y, r)
    again = gpu_lib.combine_backward(dout[:1].repeat(6, 1), y, r)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    one = w[:1].expand(8, 24, 16)
    assert torch.equal(gpu_lib.expert_product(x, one, r), gpu_lib.expert_product(x, one.contiguous(), r))


def test_a_wait_that_runs_out_is_reported(gpu_lib):
    """A withheld announcement makes a wait run out in every kind of tensor-core kernel: the status says
    so, and the same calls are right afterwards."""
    import torch
    lib = gpu_lib.load()
    ids = _random_ids(2, 600, 2, 2)
    few = _random_ids(3, 6, 4, 2)
    r, rf = _routing(gpu_lib, ids, 2), _routing(gpu_lib, few, 4)
    x, w = _normal(1, 600, 256).cuda(), _normal(2, 2, 256, 256, std=1 / 16).cuda()
    xf, wf = _normal(3, 6, 256).cuda(), _normal(4, 4, 128, 256).cuda()
    dy = _normal(5, 1200, 256).cuda()
    a, b = _normal(6, 3, 16, 256, std=1 / 16).cuda(), _normal(7, 3, 256, 16).cuda()
    which = torch.randint(0, 3, (600,), generator=_gen(8)).int().cuda()
    calls = [lambda: gpu_lib.expert_product(x, w, r), lambda: gpu_lib.expert_product(xf, wf, rf),
             lambda: gpu_lib.experts(x, w, w[:, :, :128].contiguous(), r),
             lambda: gpu_lib.expert_product_backward(dy, x, w, r, need_dw=False)[0],
             lambda: gpu_lib.expert_product_backward(dy, x, w, r, need_dx=False)[1],
             lambda: gpu_lib.adapted_product(x, w[0], a, b, which),
             lambda: gpu_lib.adapted_product(xf, w[0], a, b, which[:6].contiguous())]
    for call in calls:
        before = call().clone()
        gpu_lib.grouped_status()
        try:
            assert lib.spgemm_grouped_debug(1, 500) == 0
            call()
            with pytest.raises(gpu_lib.SpgemmError) as e:
                gpu_lib.grouped_status()
            assert e.value.code == -6 and "wait" in str(e.value)
        finally:
            lib.spgemm_grouped_debug(0, 0)
        assert torch.equal(call(), before)
        gpu_lib.grouped_status()


def test_the_hook_of_one_thread_leaves_the_others_alone(gpu_lib):
    import threading

    import torch
    lib = gpu_lib.load()
    r = _routing(gpu_lib, _random_ids(2, 600, 2, 2), 2)
    x, w = _normal(1, 600, 256).cuda(), _normal(2, 2, 256, 256, std=1 / 16).cuda()
    want = gpu_lib.expert_product(x, w, r)
    got = []

    def other():
        got.append(gpu_lib.expert_product(x, w, r))
        gpu_lib.grouped_status()

    try:
        assert lib.spgemm_grouped_debug(1, 500) == 0
        t = threading.Thread(target=other)
        t.start()
        t.join()
    finally:
        lib.spgemm_grouped_debug(0, 0)
    assert len(got) == 1 and torch.equal(got[0], want)
    gpu_lib.grouped_status()
