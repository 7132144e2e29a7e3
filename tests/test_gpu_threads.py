"""Sparse products on several host threads at once, a handle and a stream each: kernels that the threads' products share take
different amounts of shared memory."""
import threading

import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu


def test_products_of_several_host_threads(gpu_lib):
    import torch
    # different chunk widths, thresholds and row lengths, so that one kernel's blocks differ in size from thread to thread
    jobs = [(synth.rmat(11, 8, seed=3), gpu_lib.options(tau=128, chunk_width=64, chunks_max=4)), (synth.rmat(11, 8, seed=4), gpu_lib.options(tau=512, chunk_width=256)),
            (synth.config(1), None), (synth.rmat(10, 16, seed=5), gpu_lib.options(tau=64, chunk_width=128))]
    mats = [gpu_lib.DeviceCSR.from_host(a) for a, _ in jobs]
    want = [gpu_lib.multiply(m, m, opts=o).to_host() for m, (_, o) in zip(mats, jobs)]
    # sums may be added in another order: 1e-12 of the sum of the terms' magnitudes, as for every product
    sizes = [gpu_lib.multiply(a, a, opts=o).to_host()[2] for a, (_, o) in
             ((gpu_lib.DeviceCSR(m.rows, m.cols, m.row_ptr, m.col, m.val.abs()), j) for m, j in zip(mats, jobs))]
    torch.cuda.synchronize()
    go, failed = threading.Barrier(len(jobs)), []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                go.wait()
                for _ in range(15):
                    row_ptr, col, val = gpu_lib.multiply(mats[i], mats[i], stream=stream, opts=jobs[i][1]).to_host()
                    assert np.array_equal(row_ptr, want[i][0]) and np.array_equal(col, want[i][1])
                    assert np.all(np.abs(val - want[i][2]) <= 1e-12 * sizes[i])
        except Exception as e:  # noqa: BLE001  told by the thread that asserts
            failed.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
