"""The table's gradient has one order of its sums for given numbers of tokens,
rows and columns: the strides and alignments of the rows change no bit of it."""
import numpy as np
import pytest

from tests.gpu_common import cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from equivariant_mlip_tensor_b200 import api as a
    return a


# runs within one chunk, joined by one worker, by a block of 256 threads and by one of 1 024
@pytest.mark.parametrize("n,rows", [(7680, 16), (7680, 1), (9001, 700), (70000, 2)])
@pytest.mark.parametrize("width", [4, 8, 16, 24, 64, 100, 128, 132, 256])
def test_strides_and_alignments_change_no_bit(api, n, rows, width):
    import torch
    rng = np.random.default_rng(n + width)
    order = api.token_sort(cuda(rng.integers(-1, rows, n).astype(np.int32)), rows)
    g = cuda(rng.standard_normal((n, width)).astype(np.float32))
    want = api.embed_backward(order, g)
    for stride, first in ((width + 4, 0), (width + 1, 0), (width + 4, 2), (3 * width, 1)):
        wide = torch.full((n, stride), float("nan"), device="cuda")
        wide[:, first:first + width] = g
        assert torch.equal(api.embed_backward(order, wide[:, first:first + width]), want), (stride, first)
    # a gradient table off a 16-byte boundary
    flat = torch.empty(rows * width + 1, device="cuda")
    out = flat[1:].view(rows, width)
    assert torch.equal(api.embed_backward(order, g, out=out), want)
