"""Orthogonalisations issued by several host threads at once.

The kernels of all sizes up to a short side of 128 take their shared memory by
the size of the matrix; a call of one thread must not change what the launch of
another may use.
"""
import ctypes
import threading

import numpy as np
import pytest

from tests.gpu_common import cuda

pytestmark = pytest.mark.gpu

# a large and a small matrix of the same kernel: tensor-core products, in one block and in a
# cluster; fp32 sums of 4 and of 8 rows
PAIRS = [((1, 128, 256), (1, 48, 48)), ((1, 64, 1920), (1, 40, 96)), ((1, 4, 4096), (1, 4, 1700)), ((1, 8, 1024), (1, 8, 800))]


@pytest.mark.parametrize("large,small", PAIRS)
def test_threads_of_different_sizes(large, small):
    """Plain calls of the C interface in a row, which leave the interpreter's lock for
    nearly all of their time, so that the threads are inside at once."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from equivariant_mlip_tensor_b200 import api, lib
    rng = np.random.default_rng(large[1])
    inputs = [cuda(rng.standard_normal(s).astype(np.float32)) for s in (large, small)]
    wanted = [api.orthogonalise(t, steps=1) for t in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [torch.empty_like(inputs[k % 2]) for k in range(4)]
    failures, start, run = [], threading.Barrier(4), lib().cgtp_orthogonalise

    def work(k):
        batch, m, n = inputs[k % 2].shape
        args = (batch, m, n, 1, ctypes.c_float(1.0), ctypes.c_void_p(inputs[k % 2].data_ptr()),
                ctypes.c_void_p(outs[k].data_ptr()), None, 0, ctypes.c_void_p(streams[k].cuda_stream))
        start.wait(timeout=60)
        for i in range(4000):
            status = run(*args)
            if status != 0:
                failures.append((k, i, status, lib().cgtp_last_cuda_error()))
                return

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    for k in range(4):
        assert torch.equal(outs[k], wanted[k % 2])
