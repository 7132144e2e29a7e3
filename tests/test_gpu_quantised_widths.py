"""The 8-bit product in every width of tile that its rule chooses from, of one block and of two, on matrices whose scales differ
from block to block."""
import contextlib

import numpy as np
import pytest

from _grouped_ref import SUM
from _quantised_ref import BLOCK, spread
from test_gpu_grouped_shapes import choice
from test_gpu_quantised import f64, normal, powers, product_ref

pytestmark = pytest.mark.gpu

WIDTHS = [(w, p) for p in (0, 1) for w in range(64, 241, 16)]


@contextlib.contextmanager
def forced(gpu_lib, width, pair):
    lib = gpu_lib.load()
    assert lib.spgemm_quantised_force(width, pair) == 0
    try:
        yield
    finally:
        lib.spgemm_quantised_force(0, 0)


# tiles that begin and end anywhere in the blocks of 128 columns, groups of more rows than a pair's tile and of fewer, an odd number
# of slices and more of them than stages, columns off 16 bytes
SIZES = [(420, 3, 2, 328, 1010), (300, 2, 1, 1300, 701), (50, 20, 3, 130, 256)]


@pytest.fixture(scope="module")
def problems(gpu_lib):
    import torch
    made = []
    for tokens, groups, top_k, d, n in SIZES:
        ids = choice(tokens, groups, top_k)
        r = gpu_lib.group_rows(torch.tensor(ids).cuda(), groups)
        q, qw = gpu_lib.quantise_rows(normal((tokens, d), "bf16", seed=d)), gpu_lib.quantise_weights(normal((groups, n, d), "bf16", seed=n))
        kb, nb = -(-d // BLOCK), -(-n // BLOCK)
        sx, sw = powers((kb, tokens), 4).t(), powers((groups, nb, kb), 6)
        x = f64(q.values.float()) * spread(f64(sx), 1, tokens, d)
        w = np.stack([f64(qw.values[g].float()) * spread(f64(sw[g]), BLOCK, n, d) for g in range(groups)])
        made.append((r, gpu_lib.Rows8(q.values, sx, torch.bfloat16), gpu_lib.Weights8(qw.values, sw), *product_ref(x, w, ids), d))
    return made


@pytest.mark.parametrize("width,pair", WIDTHS)
@pytest.mark.parametrize("which", range(len(SIZES)))
def test_every_width(gpu_lib, problems, which, width, pair):
    import torch
    r, x8, w8, want, mag, d = problems[which]
    with forced(gpu_lib, width, pair):
        y = gpu_lib.expert_product8(x8, w8, r, out_dtype=torch.float32)
        y16 = gpu_lib.expert_product8(x8, w8, r)
    gpu_lib.grouped_status()
    err = (d + 4) * SUM * mag
    assert np.all(np.abs(f64(y) - want) <= err)
    assert y16.dtype is torch.bfloat16 and torch.equal(y16, y.bfloat16())  # one rounding of the same sums
    assert torch.equal(y, gpu_lib.expert_product8(x8, w8, r, out_dtype=torch.float32))  # no shape differs from the rule's own
    assert not y[int(r.offsets[-1]):].any()


@pytest.mark.parametrize("width,pair", [(64, 1), (112, 1), (176, 1), (144, 0)])
def test_waits_of_narrow_tiles_run_out_and_say_so(gpu_lib, problems, width, pair):
    """As for the widths of the other hook: an announcement that never comes ends as an error, and the next call is right."""
    import torch
    lib, (r, x8, w8, *_) = gpu_lib.load(), problems[0]
    with forced(gpu_lib, width, pair):
        before = gpu_lib.expert_product8(x8, w8, r)
        gpu_lib.grouped_status()
        try:
            assert lib.spgemm_grouped_debug(1, 500) == 0
            gpu_lib.expert_product8(x8, w8, r)
            with pytest.raises(gpu_lib.SpgemmError, match="wait"):
                gpu_lib.grouped_status()
        finally:
            lib.spgemm_grouped_debug(0, 0)
        assert torch.equal(gpu_lib.expert_product8(x8, w8, r), before)
        gpu_lib.grouped_status()
