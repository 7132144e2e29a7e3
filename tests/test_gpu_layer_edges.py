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


def test_layers_of_several_host_threads(gpu_lib):
    """Calls that take different amounts of shared memory, at once on four threads: none is refused, all are right."""
    import threading

    import torch

    from sparse_gemm_irregular_gb300.grouped import _dense, _pack_rule
    x, router = normal((64, 64), "bf16"), normal((512, 64), "bf16", seed=1, std=1 / 8)
    up8 = gpu_lib.quantise_weights(normal((512, 32, 64), "bf16", seed=2, std=1 / 8))
    down8 = gpu_lib.quantise_weights(normal((512, 48, 16), "bf16", seed=3, std=1 / 4))
    sizes = (64, 60, 64, 7)
    want = {t: gpu_lib.expert_layer(x[:t], router, up8, down8, 16) for t in sizes}
    torch.cuda.synchronize()
    lib, go, refused, got = gpu_lib.load(), threading.Barrier(len(sizes)), [], {}

    def calls(i, t):
        s = torch.cuda.Stream()
        out, ids, weights = (torch.empty_like(v) for v in want[t])
        # the entry point itself, which lets the other threads run: through the Python layer calls hardly meet
        args = (_dense(x[:t], "x"), _dense(router, "w_router"), _pack_rule(16, 0, 1, 1, 0, 1, 1.0, 0), None, None, None, up8._packed(),
                down8._packed(), _dense(out, "out"), ids.data_ptr(), weights.data_ptr(), s.cuda_stream)
        torch.cuda.synchronize()
        go.wait()
        for _ in range(4000):
            rc = lib.spgemm_expert_layer(*args)
            if rc:
                refused.append((t, rc, gpu_lib.spgemm_last_error()))
                break
        s.synchronize()
        got[i] = out, ids, weights

    threads = [threading.Thread(target=calls, args=a) for a in enumerate(sizes)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not refused, refused
    for i, t in enumerate(sizes):
        assert all(torch.equal(p, q) for p, q in zip(got[i], want[t]))
    gpu_lib.grouped_status()
