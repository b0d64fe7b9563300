"""Statistics of long samples and wide groups whose first part is unlike the rest.

The split by tiles joins the means and squared deviations of a sample's parts.
A sample may start on the last row of a tile, so that its first part is one
row; what that row holds must not cost the others their digits.

Tolerances, with u = 2^-24 and K = 96 rounded operations in a row at most (8 rows a
thread, trees of 3 + 5 levels, 32 warps and at most 13 slots a thread, two operations each):
a part's mean c is off by d <= K u mean|x| of the part, and so is the mean of the sample, by
K u mean|x| over its group and half a step for each of two last additions.
The squared deviations are sums of terms of one sign, off by K u of themselves, and
deviations from c instead of the part's own mean leave out 2 n d (c - mean) of each
part, by Cauchy at most 2 K u rms|x| sd per value.  So the variance is off by
K u (1 + 2 rms|x| / sd) of itself and rstd by K u (1 + rms|x| rstd).
"""
import numpy as np
import pytest

from oracle import norm as onorm
from tests.gpu_common import cuda, host

pytestmark = pytest.mark.gpu
U, K, EPS = 2.0 ** -24, 96, 1e-5


@pytest.fixture(scope="module")
def api():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from equivariant_mlip_tensor_b200 import api as a
    return a


def _check(api, x, ptr, groups, max_rows, k=K):
    p = cuda(np.asarray(ptr, dtype=np.int32))
    y, mean, rstd = api.group_norm_forward(cuda(x), None, None, groups, graph_ptr=p, eps=EPS, max_rows=max_rows)
    want, om, orstd = onorm.forward(x, None, None, groups, ptr, EPS, None)
    n, c = x.shape
    for s, (lo, hi) in enumerate(zip(ptr[:-1], ptr[1:])):
        v = x[lo:hi].reshape(hi - lo, groups, c // groups).astype(np.float64)
        size, rms = np.abs(v).mean(axis=(0, 2)), np.sqrt((v * v).mean(axis=(0, 2)))
        off_mean = np.abs(host(mean)[s] - om[s])
        assert (off_mean <= k * U * size + 2 * U * np.abs(om[s])).all(), (s, off_mean)
        off_rstd = np.abs(host(rstd)[s] / orstd[s] - 1)
        assert (off_rstd <= k * U * (1 + rms * orstd[s])).all(), (s, off_rstd)
    return host(y), want


# rows of 132 channels in one group: tiles of 64 rows
@pytest.mark.parametrize("first", [63, 62, 40, 64])
@pytest.mark.parametrize("value,offset", [(100.0, 0.0), (1e4, 0.0), (-3e3, 5.0), (0.0, 1000.0)])
def test_first_row_unlike_the_others(api, first, value, offset):
    """One long sample: the first row begins on the last row of a tile, before it and after it."""
    rng = np.random.default_rng(first)
    n, c = 4000, 132
    x = (rng.standard_normal((n, c)) + offset).astype(np.float32)
    x[first, 0] = value
    y, want = _check(api, x, [0, first, n], 1, 0)
    assert np.isfinite(y).all()


@pytest.mark.parametrize("value", [1e3, -1e4])
def test_many_samples_with_such_rows(api, value):
    """Samples of a few parts, joined by a warp each."""
    rng = np.random.default_rng(5)
    ptr = np.concatenate([[0], np.arange(63, 63 + 128 * 21, 128)])
    x = rng.standard_normal((int(ptr[-1]), 132)).astype(np.float32)
    x[ptr[1:-1], 0] = value
    _check(api, x, ptr, 1, 128)


def test_long_sample_of_narrow_groups(api):
    """The size of a bulk cell's read-out: enough values for the tiles, groups of 8 channels."""
    rng = np.random.default_rng(6)
    n, c = 140000, 128
    x = rng.standard_normal((n, c)).astype(np.float32)
    ptr = [0, 1023, n]
    x[1023, ::8] = 1e4
    # eight register loads of 8 rows a thread and their joins instead of one: 5 operations each
    _check(api, x, ptr, 16, 0, K + 40)
