"""Every shape of the tensor-core grouped products (width of a tile, two blocks to a tile, depth split over
blocks) against the formulas in 64 bits, at sizes that end inside every tile."""
import contextlib

import numpy as np
import pytest

from _grouped_ref import SUM, TINY, U, transpose

pytestmark = pytest.mark.gpu

SHAPES = [(16, 0), (32, 0), (64, 0), (128, 0), (256, 0), (256, 1)]


@contextlib.contextmanager
def forced(gpu_lib, width, pair=0, split=0):
    lib = gpu_lib.load()
    assert lib.spgemm_grouped_force(width, pair, split) == 0
    try:
        yield
    finally:
        lib.spgemm_grouped_force(0, 0, 0)


def normal(seed, *shape, dtype="bf16", std=1.0):
    import torch
    t = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(t).cuda()


def near(got, want, dtype, slack):
    """Half a spacing of the type (f32: none) and `slack`."""
    import torch
    one = torch.zeros_like(want) if dtype == "f32" else torch.clamp(U[dtype] * want.abs(), min=TINY[dtype])
    over = (got.double() - want).abs() - one - slack
    assert (over <= 0).all(), float(over.max())


def choice(tokens, groups, top_k, seed=0):
    """Distinct ascending groups of very different sizes, some slots and one group left out."""
    rng = np.random.default_rng(seed + tokens)
    p = np.exp(-1.2 * np.arange(groups))
    if groups > 2:
        p[1] = 0.0
    p = np.maximum(p, 1e-3) if groups <= 2 else np.where(p > 0, np.maximum(p, 1e-3), 0)
    k = min(top_k, int((p > 0).sum()))
    ids = np.full((tokens, top_k), -1, np.int32)
    for t in range(tokens):
        n = k if rng.random() < 0.85 else int(rng.integers(0, k + 1))
        ids[t, :n] = np.sort(rng.choice(groups, n, replace=False, p=p / p.sum()))
    return ids


# many rows per group (laid out first) and few (gathered)
CASES = [(900, 5, 3, 328, 392), (70, 40, 2, 200, 136)]


@pytest.mark.parametrize("tokens,groups,top_k,d,n", CASES)
@pytest.mark.parametrize("width,pair", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_products(gpu_lib, tokens, groups, top_k, d, n, width, pair, dtype):
    import torch
    ids = choice(tokens, groups, top_k)
    r = gpu_lib.group_rows(torch.tensor(ids).cuda(), groups)
    offsets, order, _ = transpose(ids, groups)
    x, w, dy = normal(1, tokens, d, dtype=dtype), normal(2, groups, n, d, dtype=dtype), normal(3, ids.size, n, dtype=dtype)
    dy[offsets[-1]:] = float("nan")
    with forced(gpu_lib, width, pair):
        y = gpu_lib.expert_product(x, w, r)
        y32 = gpu_lib.expert_product(x, w, r, out_dtype=torch.float32)
        dx, dw = gpu_lib.expert_product_backward(dy, x, w, r)
    gpu_lib.grouped_status()
    xd, wd, dyd = x.double(), w.double(), dy.double()
    wx, mx = torch.zeros_like(xd), torch.zeros_like(xd)
    for g in range(groups):
        a, b = int(offsets[g]), int(offsets[g + 1])
        tok = torch.tensor(order[a:b] // top_k).cuda()
        want, mag = xd[tok] @ wd[g].t(), xd[tok].abs() @ wd[g].abs().t()
        near(y[a:b], want, dtype, SUM * d * mag)
        near(y32[a:b], want, "f32", SUM * d * mag)
        wx.index_add_(0, tok, dyd[a:b] @ wd[g])
        mx.index_add_(0, tok, dyd[a:b].abs() @ wd[g].abs())
        near(dw[g], dyd[a:b].t() @ xd[tok], dtype, SUM * max(b - a, 1) * (dyd[a:b].abs().t() @ xd[tok].abs()))
    near(dx, wx, dtype, SUM * (n + top_k) * mx)
    assert (y[offsets[-1]:] == 0).all() and (y32[offsets[-1]:] == 0).all()


@pytest.mark.parametrize("tokens,groups,top_k,d,hidden", [(900, 5, 3, 328, 200), (70, 40, 2, 200, 72)])
@pytest.mark.parametrize("width,pair", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gated_layer(gpu_lib, tokens, groups, top_k, d, hidden, width, pair, dtype):
    import torch
    ids = choice(tokens, groups, top_k)
    weights = torch.rand(tokens, top_k, generator=torch.Generator().manual_seed(4)).cuda()
    r = gpu_lib.group_rows(torch.tensor(ids).cuda(), groups, weights=weights)
    x = normal(1, tokens, d, dtype=dtype)
    up, down = normal(2, groups, 2 * hidden, d, dtype=dtype, std=d ** -0.5), normal(3, groups, d, hidden, dtype=dtype, std=hidden ** -0.5)
    with forced(gpu_lib, width, pair):
        out = gpu_lib.experts(x, up, down, r)
    gpu_lib.grouped_status()
    xd, ud, dd = x.double(), up.double(), down.double()
    want, tol = torch.zeros_like(xd), torch.zeros_like(xd)
    for g in range(groups):
        at = (torch.tensor(ids).cuda() == g).nonzero()
        tok, wt = at[:, 0], weights[at[:, 0], at[:, 1], None].double()
        pre, mag = xd[tok] @ ud[g].t(), xd[tok].abs() @ ud[g].abs().t()
        gate, u = pre[:, :hidden], pre[:, hidden:]
        act = gate * torch.sigmoid(gate)
        h = act * u
        # the two products' errors through silu (slope at most 1.1), exp and division, one rounding of h
        eh = SUM * d * (1.1 * u.abs() * mag[:, :hidden] + act.abs() * mag[:, hidden:]) + (U[dtype] + 2.0 ** -20) * h.abs() + TINY[dtype]
        want.index_add_(0, tok, wt * (h @ dd[g].t()))
        tol.index_add_(0, tok, wt * ((eh + SUM * (hidden + top_k) * h.abs()) @ dd[g].abs().t()))
    near(out, want, dtype, 1.01 * tol)


ADAPTED = SHAPES + [(16, 0, 2), (32, 0, 4), (64, 0, 2), (64, 0, 4), (64, 0, 8)]


@pytest.mark.parametrize("tokens,adapters,rank,d,n,mixed", [
    (600, 5, 24, 1096, 264, False), (600, 13, 72, 1096, 136, True), (61, 3, 16, 1096, 520, True), (61, 1, 8, 1032, 72, False)])
@pytest.mark.parametrize("shape", ADAPTED)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_adapters(gpu_lib, tokens, adapters, rank, d, n, mixed, shape, dtype):
    import torch
    rng = np.random.default_rng(tokens)
    ids = rng.integers(-1, adapters, tokens).astype(np.int32)
    ids = torch.tensor(ids if mixed else np.sort(ids)).cuda()
    x, w = normal(1, tokens, d, dtype=dtype), normal(2, n, d, dtype=dtype, std=d ** -0.5)
    a, b = normal(3, adapters, rank, d, dtype=dtype, std=d ** -0.5), normal(4, adapters, n, rank, dtype=dtype, std=0.3)
    scale = torch.rand(adapters, generator=torch.Generator().manual_seed(9)).cuda() + 0.5
    with forced(gpu_lib, *shape):
        y = gpu_lib.adapted_product(x, w, a, b, ids, scale)
    gpu_lib.grouped_status()
    xd, wd = x.double(), w.double()
    want, tol = xd @ wd.t(), SUM * (d + rank) * (xd.abs() @ wd.abs().t())
    for i in range(adapters):
        t, s = (ids == i).nonzero()[:, 0], float(scale[i])
        v, mv = xd[t] @ a[i].double().t(), xd[t].abs() @ a[i].double().abs().t()
        want[t] += s * (v @ b[i].double().t())
        # v is rounded to the inputs' type once between the two small products
        tol[t] += (s * (SUM * (d + rank) * mv + (U[dtype] + 2.0 ** -22) * v.abs()) + TINY[dtype]) @ b[i].double().abs().t()
    near(y, want, dtype, 1.01 * tol)


@pytest.mark.parametrize("tokens,adapters,rank,d,n", [(600, 5, 24, 1096, 264), (61, 3, 16, 1096, 136)])
@pytest.mark.parametrize("shape", ADAPTED)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_broken_adapter_reaches_its_own_rows_only(gpu_lib, tokens, adapters, rank, d, n, shape, dtype):
    """Infinite and NaN values in an adapter that is used: rows of other adapters and of none stay what they are,
    its own become what the formula says, whatever else is in their tile."""
    import torch
    ids = torch.tensor(np.random.default_rng(5).integers(-1, adapters, tokens).astype(np.int32)).cuda()
    x, w = normal(1, tokens, d, dtype=dtype), normal(2, n, d, dtype=dtype, std=d ** -0.5)
    a, b = normal(3, adapters, rank, d, dtype=dtype, std=d ** -0.5), normal(4, adapters, n, rank, dtype=dtype, std=0.3)
    b[1, 7, 3], b[1, 20:40, 0], b[1, n - 1] = float("nan"), float("inf"), float("-inf")
    x[tokens // 2] = float("nan")  # and a broken row
    with forced(gpu_lib, *shape):
        y = gpu_lib.adapted_product(x, w, a, b, ids)
    gpu_lib.grouped_status()
    xd, wd = x.double(), w.double()
    want, tol = xd @ wd.t(), SUM * (d + rank) * (xd.abs() @ wd.abs().t())
    for i in range(adapters):
        t = (ids == i).nonzero()[:, 0]
        v, mv = xd[t] @ a[i].double().t(), xd[t].abs() @ a[i].double().abs().t()
        want[t] += v @ b[i].double().t()
        tol[t] += (SUM * (d + rank) * mv + (U[dtype] + 2.0 ** -22) * v.abs() + TINY[dtype]) @ b[i].double().abs().t()
    fine = torch.isfinite(want)
    clean = (ids != 1) & (torch.arange(tokens, device="cuda") != tokens // 2)
    assert fine[clean].all() and not fine[(ids == 1)][:, n - 1].any()
    assert torch.equal(torch.isfinite(y), fine)
    near(y[fine], want[fine], dtype, 1.01 * tol[fine])


@pytest.mark.parametrize("shape", [(256, 1), (256, 0), (64, 0, 8), (64, 0, 2), (16, 0, 2)])
def test_a_wait_that_runs_out_is_reported(gpu_lib, shape):
    """In the kernels of two blocks to a tile and of split depth too: the status says so, later calls are right."""
    import torch
    lib = gpu_lib.load()
    r = gpu_lib.group_rows(torch.tensor(choice(600, 2, 2)).cuda(), 2)
    x, w, dy = normal(1, 600, 1024), normal(2, 2, 256, 1024, std=1 / 32), normal(5, 1200, 256)
    a, b = normal(6, 3, 16, 1024, std=1 / 32), normal(7, 3, 256, 16)
    which = torch.randint(0, 3, (600,), generator=torch.Generator().manual_seed(8)).int().cuda()
    up, down = normal(8, 2, 256, 1024, std=1 / 32), normal(9, 2, 64, 128)
    calls = [lambda: gpu_lib.adapted_product(x, w[0], a, b, which)]
    if len(shape) == 2:
        calls += [lambda: gpu_lib.expert_product(x, w, r), lambda: gpu_lib.experts(x, up, down, r),
                  lambda: gpu_lib.expert_product_backward(dy, x, w, r, need_dw=False)[0],
                  lambda: gpu_lib.expert_product_backward(dy, x, w, r, need_dx=False)[1]]
    with forced(gpu_lib, *shape):
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
