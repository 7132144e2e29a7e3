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


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_token_in_another_row_of_each_expert(gpu_lib, dtype, bits):
    """Token 3 is the first, second, third and fourth of the experts that it chooses, one after the other: its sums pass from lane to
    lane of the warps that form them."""
    import torch
    tokens, experts, top_k, d, hidden, n = 4, 16, 8, 256, 48, 144
    chosen = [[e for e in range(8) if t == 3 or e % 4 > t] for t in range(tokens)]
    chosen = [c + list(range(8 + t, 8 + t + top_k - len(c))) for t, c in enumerate(chosen)]
    assert all(len(c) == top_k and max(c) < experts for c in chosen)
    x, router = normal((tokens, d), dtype), torch.zeros(experts, d)
    x[:, :tokens] = torch.eye(tokens) * 4
    for t, c in enumerate(chosen):
        for i, e in enumerate(c):
            router[e, t] = 1 + i / 16  # no two alike
    router = router.to(x)
    up, down = normal((experts, 2 * hidden, d), dtype, seed=2, std=d ** -0.5), normal((experts, n, hidden), dtype, seed=3, std=hidden ** -0.5)
    if bits == 8:
        up, down = gpu_lib.quantise_weights(up), gpu_lib.quantise_weights(down)
        u64, d64 = (f64(gpu_lib.dequantise(w, torch.float32)) for w in (up, down))
    else:
        u64, d64 = f64(up), f64(down)
    want, ids, weights, err, gap = layer_ref(f64(x), f64(router), u64, d64, dtype, top_k, None, parts=2)
    assert gap > 1e-6 and [list(i) for i in ids] == chosen
    first, gi, _ = gpu_lib.expert_layer(x, router, up, down, top_k)
    assert np.array_equal(gi.cpu().numpy(), ids)
    assert np.all(np.abs(f64(first) - want) <= err)
    for _ in range(50):
        assert torch.equal(gpu_lib.expert_layer(x, router, up, down, top_k)[0], first)
