"""Orthogonalised updates against the fp64 oracle.

Tolerance: a step maps X to a X + (b X X^T + c (X X^T)^2) X.  On singular values
in [0, 1.21] the derivative of its polynomial is at most 3.9, so an error of
step k is at the end at most 3.9^(steps - k - 1) times itself (Frobenius norm).
The step's own error: three fp32-accurate products, each within 2^-21 of the
product of the norms (operands and sums of a product in 22 bits or more), with
spectral norms |X|, |X X^T| <= 1.45 and |b X X^T + c (X X^T)^2| <= 2.9, so
that the errors of the Gram matrix pass through |b| + 2 |c| 1.45 < 11 and one
more factor 1.21: below 2^-21 (11 x 1.21 x 1.45 + 2.9 x 1.21 + 3.45) < 27 x
2^-21 of |X_k|_F in all.  Errors of independent roundings add up like their root
mean square, not their sum, which leaves this bound with a wide margin.
"""
import numpy as np
import pytest

from oracle import ortho as oortho
from tests.gpu_common import cuda, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from equivariant_mlip_tensor_b200 import api as a
    return a


def _check(got, g, steps=5, scale=1.0):
    for z in range(g.shape[0]):
        xs = oortho.iterates(g[z], steps)
        want = scale * (xs[-1].T if g.shape[1] > g.shape[2] else xs[-1])
        bound = 27 * 2.0 ** -21 * sum(3.9 ** (steps - k - 1) * np.linalg.norm(xs[k]) for k in range(steps))
        off = np.linalg.norm(got[z] - want)
        assert off <= abs(scale) * bound, (z, off, bound)
        # and close in the ordinary sense: no direction is lost
        assert off <= 1e-3 * max(np.linalg.norm(want), 1e-30), (z, off)


SHAPES = [(1, 1, 1), (1, 1, 7), (2, 7, 1), (5, 8, 8), (3, 4, 100), (2, 100, 4), (15, 32, 16), (2, 33, 65), (4, 64, 64),
          (1, 64, 1920), (3, 128, 128), (2, 127, 129), (2, 129, 127), (2, 128, 96), (1, 130, 260), (2, 256, 192),
          (1, 300, 77), (1, 256, 512), (1, 520, 530), (150, 12, 20), (1, 40, 2100), (1, 1920, 64), (2, 128, 257)]


@pytest.mark.parametrize("batch,m,n", SHAPES)
def test_matches_the_oracle(api, batch, m, n):
    rng = np.random.default_rng(batch + m + n)
    g = (1e-3 * rng.standard_normal((batch, m, n))).astype(np.float32)
    _check(host(api.orthogonalise(cuda(g))), g)


@pytest.mark.parametrize("m,n", [(8, 8), (64, 48), (128, 128), (96, 300), (200, 180)])
@pytest.mark.parametrize("steps,scale", [(1, 1.0), (2, -0.5), (5, 2.0), (11, 1.0)])
def test_steps_and_scale(api, m, n, steps, scale):
    rng = np.random.default_rng(m + n + steps)
    g = rng.standard_normal((2, m, n)).astype(np.float32)
    got = host(api.orthogonalise(cuda(g), steps=steps, scale=scale))
    if steps > 5:  # errors no longer grow: values move inside the attracting interval, where |p'| < 1.2
        s = np.linalg.svd(got[0], compute_uv=False)
        assert s.max() < 1.21 and s.min() > 0.6
    else:
        _check(got, g, steps, scale)


@pytest.mark.parametrize("m,n", [(8, 12), (128, 128), (64, 700), (260, 200)])
def test_scales_from_tiny_to_huge(api, m, n):
    """The norm neither overflows nor vanishes; below the floor 1e-7 the update
    is divided by the floor."""
    rng = np.random.default_rng(m)
    g = rng.standard_normal((4, m, n)).astype(np.float32)
    g[0] *= np.float32(1e-12)
    g[1] *= np.float32(1e30)
    g[2] *= np.float32(3e-9)
    _check(host(api.orthogonalise(cuda(g))), g)


@pytest.mark.parametrize("m,n", [(8, 8), (128, 128), (64, 700), (260, 200)])
def test_zero_one_and_nonfinite_matrices(api, m, n):
    """A matrix of zeros gives zeros, a single entry keeps its place, and a NaN
    or an infinity spoils its own matrix only."""
    rng = np.random.default_rng(m)
    g = rng.standard_normal((6, m, n)).astype(np.float32)
    good = host(api.orthogonalise(cuda(g)))
    g[1] = 0
    g[2] = 0
    g[2, m - 1, n - 1] = -3.0
    g[3, 0, 0] = np.nan
    g[4, 1, 2] = np.inf
    got = host(api.orthogonalise(cuda(g)))
    assert np.array_equal(got[0], good[0]) and np.array_equal(got[5], good[5])
    assert not got[1].any()
    _check(got[2:3], g[2:3])
    assert np.count_nonzero(got[2]) == 1
    assert np.isnan(got[3]).all() and np.isnan(got[4]).all()


@pytest.mark.parametrize("m,n", [(8, 8), (128, 128), (96, 64), (64, 1920), (200, 260)])
def test_in_place_low_rank_and_equal_bits(api, m, n):
    import torch
    rng = np.random.default_rng(m + n)
    k = max(1, min(m, n) // 4)
    g = (rng.standard_normal((2, m, k)) @ rng.standard_normal((2, k, n)) + 1e-2 * rng.standard_normal((2, m, n)))
    g = g.astype(np.float32)
    a = api.orthogonalise(cuda(g))
    _check(host(a), g)
    assert torch.equal(a, api.orthogonalise(cuda(g)))
    t = cuda(g)
    assert api.orthogonalise(t, out=t).data_ptr() == t.data_ptr()
    assert torch.equal(t, a)
    assert torch.equal(api.orthogonalise(cuda(g)[1]), a[1])  # a matrix alone: the same bits


@pytest.mark.parametrize("m,n", [(32, 32), (128, 200), (64, 1920), (300, 300)])
def test_streams_and_graph_replay(api, m, n):
    import torch
    g = torch.zeros((3, m, n), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            out = api.orthogonalise(g)
        for seed in (1, 2):
            h = np.random.default_rng(seed).standard_normal((3, m, n)).astype(np.float32)
            g.copy_(cuda(h))
            graph.replay()
            s.synchronize()
            _check(host(out), h)


def test_empty_and_refusals(api):
    import torch
    assert api.orthogonalise(torch.empty((0, 4, 4), device="cuda")).shape == (0, 4, 4)
    assert api.orthogonalise(torch.empty((2, 0, 4), device="cuda")).shape == (2, 0, 4)
    x = torch.zeros((4, 8), device="cuda")
    for bad in (lambda: api.orthogonalise(x.half()), lambda: api.orthogonalise(x.t()), lambda: api.orthogonalise(x[0]),
                lambda: api.orthogonalise(x.cpu()), lambda: api.orthogonalise(x, out=x[:2])):
        with pytest.raises(ValueError):
            bad()
    from equivariant_mlip_tensor_b200 import CGTPError
    for kw in ({"steps": 0}, {"steps": 65}):
        with pytest.raises(CGTPError):
            api.orthogonalise(x, **kw)
