"""The whole-layer call where its answer could depend on the path that a number of tokens takes."""
import numpy as np
import pytest

from test_gpu_quantised import f64, layer_ref, normal, silu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens", [1, 3, 12, 32, 33])
def test_infinities_in_the_down_matrix(gpu_lib, tokens, dtype):
    """An infinite entry gives an infinity of the sign of its hidden value, and NaN where two experts' signs differ, on every
    path; the other columns keep their bits."""
    x, router = normal((tokens, 128), dtype), normal((8, 128), dtype, seed=1, std=1 / 11)
    up, down = normal((8, 96, 128), dtype, seed=2, std=1 / 11), normal((8, 72, 48), dtype, seed=3, std=1 / 7)
    clean, ids, weights = gpu_lib.expert_layer(x, router, up, down, 2)
    at, signs = {5: 7, 6: 9, 70: 0, 33: 47}, {5: 1, 6: -1, 70: 1, 33: -1}  # column of the result: hidden value
    for n, k in at.items():
        down[:, n, k] = signs[n] * float("inf")
    out, gi, gw = gpu_lib.expert_layer(x, router, up, down, 2)
    gpu_lib.grouped_status()
    assert (gi == ids).all() and (gw == weights).all()
    keep = [n for n in range(72) if n not in at]
    assert (out[:, keep] == clean[:, keep]).all()
    got, e = f64(out), ids.cpu().numpy()
    x, up = f64(x), f64(up)
    for n, k in at.items():
        for t in range(tokens):
            pre = up[e[t]] @ x[t]
            h = silu(pre[:, k]) * pre[:, 48 + k]
            assert np.all(np.abs(h) > 1e-6)  # no sign hangs on a rounding
            with np.errstate(invalid="ignore"):
                want = np.sum(np.sign(h) * signs[n] * np.inf)
            assert np.array_equal(got[t, n], want, equal_nan=True), (t, n, got[t, n], want)
