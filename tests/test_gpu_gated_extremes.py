"""The gated product with its checkpoint at the ends of its range, in each type."""
import numpy as np
import pytest

from _grouped_ref import rounding
from _quantised_ref import held, silu
from test_gpu_quantised import f64, few, torch_type

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
GATES = [-INF, -200.0, -104.0, -103.0, -89.0, -88.5, -88.0, -87.5, -87.0, -60.0, -17.0, -1.2784, -0.0, 0.0, 1e-3, 17.0, 88.0, 200.0, INF, NAN]
UPS = {"f32": [1.0, -3.0, 0.0, 1e30, -1e-30, INF, NAN], "bf16": [1.0, -3.0, 0.0, 1e30, -1e-30, INF, NAN], "f16": [1.0, -3.0, 0.0, 65504.0, -6e-8, INF, NAN]}


def pairs(dtype):
    import torch
    g, u = torch.tensor(GATES), torch.tensor(UPS[dtype])
    return g.repeat_interleave(len(u)), u.repeat(len(g))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_forward(gpu_lib, dtype):
    """One pair to a row, so that no number is brought to 8 bits beside a larger one."""
    import torch
    g, u = pairs(dtype)
    pre = torch.stack([g, u], 1).to(torch_type(dtype)).cuda()
    h, gate8, up8 = gpu_lib.gated8(pre)
    g, u = f64(pre)[:, 0], f64(pre)[:, 1]
    with np.errstate(all="ignore"):
        # 32-bit numbers end at 2^128 and exp(-g) with them: from there on silu is -0, and with an infinity NaN
        s = np.where(g > -88.72, silu(g), np.where(np.isfinite(g), -0.0, np.nan))
        s = np.where(g == INF, INF, s)
        want = s * u
    got = f64(h)[:, 0]
    top = {"f32": 3.4028235e38, "bf16": 3.3895314e38, "f16": 65504.0}[dtype]
    assert np.array_equal(np.isnan(got), np.isnan(want)), (g[np.isnan(got) != np.isnan(want)], u[np.isnan(got) != np.isnan(want)])
    with np.errstate(all="ignore"):
        big = ~np.isnan(want) & (np.abs(want) > top * (1 + 2.0 ** -9))
        assert np.array_equal(got[big], np.copysign(INF, want[big]))
        ok = ~np.isnan(want) & ~big
        # the factor s of silu where it is below 32 bits' normal range: held to half its smallest step, a few of them
        low = 8 * 2.0 ** -149 * np.abs(g * u)
        over = np.abs(got - want) - few(dtype) * np.abs(want) - rounding(dtype, want) - low - 2.0 ** -149
    assert np.all(over[ok] <= 0), (g[ok][over[ok] > 0], u[ok][over[ok] > 0], got[ok][over[ok] > 0], want[ok][over[ok] > 0])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_backward(gpu_lib, dtype):
    import torch
    g, u = pairs(dtype)
    pre = torch.stack([g, u], 1).to(torch_type(dtype)).cuda()
    _, gate8, up8 = gpu_lib.gated8(pre)
    dh = torch.full((len(g), 1), -0.5, device="cuda").to(torch_type(dtype))
    dpre, again = gpu_lib.gated8_backward(dh, gate8, up8)
    with np.errstate(all="ignore"):
        g, u = held(f64(pre)[:, :1])[:, 0], held(f64(pre)[:, 1:])[:, 0]
        s = np.where(np.isnan(g), np.nan, np.where(g > -88.72, 1.0 / (1.0 + np.exp(-g)), 0.0))
        low = 8 * 2.0 ** -149
        top = {"f32": 3.4028235e38, "bf16": 3.3895314e38, "f16": 65504.0}[dtype]
        for got, want, part, tiny in ((f64(again)[:, 0], g * s * u, None, np.abs(g * u)), (f64(dpre)[:, 1], -0.5 * g * s, None, np.abs(g)),
                                      (f64(dpre)[:, 0], -0.5 * u * s * (1 + g * (1 - s)), np.abs(u) * s * (1 + np.abs(g) * (1 - s)),
                                       np.abs(u) * (1 + np.abs(g)))):
            lost = np.isnan(g) if tiny is not None and np.array_equal(tiny, np.abs(g), equal_nan=True) else np.isnan(g) | np.isnan(u)
            assert np.array_equal(np.isnan(got), lost)
            big = ~lost & (np.abs(want) > top * (1 + 2.0 ** -9))
            assert np.array_equal(got[big], np.copysign(INF, want[big]))
            ok = ~lost & ~big
            over = np.abs(got - want) - few(dtype) * (np.abs(want) if part is None else part) - rounding(dtype, want) - low * tiny - 2.0 ** -149
            assert np.all(over[ok] <= 0), (g[ok][over[ok] > 0], u[ok][over[ok] > 0], got[ok][over[ok] > 0], want[ok][over[ok] > 0])
