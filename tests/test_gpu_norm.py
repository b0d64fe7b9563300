"""Per-graph group norm with its activation against the fp64 oracle.

Tolerances, with u = 2^-24 (half a step of fp32) and K = 96, a bound on the
rounded operations in a row that a value passes through at these sizes (a sum
of at most 8 values, trees of 8 + 5 + 8 levels and at most 48 slots a thread,
the join, and some 20 operations around them): the mean is off by K u max|x|
over its group, a deviation x - mean by (K + 1) u max|x| more, and rstd, a
function of sums of squared deviations, by K u + 2 K u max|x| rstd of itself
(d rstd / rstd = -d sigma / sigma).  With D = max|x - mean| <= 2 max|x| the
normalised value h is off by at most 2 K u M with M = rstd max|x| (1 + |h|),
and y = act(gamma h + beta) by 1.1 (|gamma| 2 K u M + 3 u |z|) + 4 u |y|, since
|SiLU'| < 1.1.  Gradients: the library's measure, max|diff| / max|oracle| <= 1e-4,
at inputs of ordinary scale, where the same bound times
the few products of the chain stays below it (K u x 10 = 6e-5).
"""
import numpy as np
import pytest

from oracle import norm as onorm
from tests.gpu_common import GRAD_TOL, cuda, host, rel_err

pytestmark = pytest.mark.gpu
U, K, EPS = 2.0 ** -24, 96, 1e-5


@pytest.fixture(scope="module")
def api():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from equivariant_mlip_tensor_b200 import api as a
    return a


def _ptr(rng, n, samples, kind):
    if kind is None:
        return None
    if kind == "equal":
        return np.arange(samples + 1) * n // samples
    cuts = np.sort(rng.integers(0, n + 1, samples - 1))
    if samples > 3:
        cuts[1] = cuts[0]  # a graph without rows
    ptr = np.concatenate([[0], cuts, [n]])
    if kind == "inner":  # rows before the first graph and behind the last one
        ptr = np.clip(ptr, n // 10, n - n // 8)
    return ptr


def _inside(ptr, n):
    m = np.ones(n, bool)
    if ptr is not None:
        m[:ptr[0]] = False
        m[ptr[-1]:] = False
    return m


def _i32(a):
    return None if a is None else cuda(np.asarray(a, dtype=np.int32))


def _forward_bound(x, gamma, beta, groups, ptr, activation):
    """Elementwise bound of the module's comment."""
    y, mean, rstd = onorm.forward(x, gamma, beta, groups, ptr, EPS, activation)
    n, c = x.shape
    cpg, bound = c // groups, np.zeros((n, c))
    for s, (lo, hi) in enumerate([(0, n)] if ptr is None else zip(ptr[:-1], ptr[1:])):
        if hi == lo:
            continue
        v = np.abs(x[lo:hi].reshape(hi - lo, groups, cpg))
        top = np.repeat(v.max(axis=(0, 2)), cpg)
        r, m = np.repeat(rstd[s], cpg), np.repeat(mean[s], cpg)
        h = np.abs(x[lo:hi] - m) * r
        z = gamma * (x[lo:hi] - m) * r + beta
        off = 2 * K * U * r * top * (1 + h)
        bound[lo:hi] = 1.1 * (np.abs(gamma) * off + 3 * U * np.abs(z)) + 4 * U * np.abs(y[lo:hi]) + 1e-30
    return y, mean, rstd, bound


CASES = [(1, 1, 4, 1, None), (1, 1, 1, 1, None), (5, 1, 12, 3, None), (70, 1, 128, 8, None), (700, 1, 96, 32, "equal"),
         (240, 8, 128, 8, "equal"), (240, 8, 64, 1, "equal"), (300, 10, 128, 128, "equal"), (333, 17, 36, 4, "ragged"),
         (500, 90, 13, 1, "ragged"), (64, 64, 16, 4, "equal"), (1500, 7, 260, 4, "ragged"), (900, 6, 20, 5, "inner"),
         (4000, 2, 8, 2, "ragged"), (200, 3, 1028, 2, "ragged"), (130, 5, 33, 11, "inner")]


@pytest.mark.parametrize("n,samples,c,groups,kind", CASES)
@pytest.mark.parametrize("activation", [None, "silu"])
@pytest.mark.parametrize("hint", [0, 1])
def test_both_directions_match_the_oracle(api, n, samples, c, groups, kind, activation, hint):
    rng = np.random.default_rng(n + c + samples)
    ptr = _ptr(rng, n, samples, kind)
    x = (rng.standard_normal((n, c)) * (0.5 + rng.random(c)) + rng.standard_normal(c)).astype(np.float32)
    gamma, beta = (1 + 0.3 * rng.standard_normal(c)).astype(np.float32), rng.standard_normal(c).astype(np.float32)
    gy = rng.standard_normal((n, c)).astype(np.float32)
    longest = n if ptr is None else int(np.diff(ptr).max())
    kw = dict(graph_ptr=_i32(ptr), activation=activation, max_rows=longest if hint else 0)
    y, mean, rstd = api.group_norm_forward(cuda(x), cuda(gamma), cuda(beta), groups, eps=EPS, **kw)
    want, om, orstd, bound = _forward_bound(x, gamma, beta, groups, ptr, activation)
    m = _inside(ptr, n)
    assert (np.abs(host(y) - want)[m] <= bound[m]).all()
    assert np.allclose(host(rstd), orstd, rtol=2e-5 * max(1.0, float(orstd.max())), atol=0)
    assert rel_err(host(mean), om) <= K * U * 4
    gx, gg, gb = api.group_norm_backward(cuda(x), cuda(gamma), cuda(beta), groups, mean, rstd, cuda(gy), **kw)
    wx, wg, wb = onorm.backward(x, gamma, beta, groups, ptr, EPS, activation, gy)
    # a group of one value has no gradient: what is left are roundings of rstd |t|, not of the (zero) result
    floor = GRAD_TOL * float(orstd.max()) * 1.1 * np.abs(gamma).max() * np.abs(gy).max() * (n * c // groups < 8 * samples)
    assert np.abs(host(gx) - wx)[m].max(initial=0) <= max(GRAD_TOL * np.abs(wx[m]).max(initial=0), floor)
    assert np.abs(host(gg) - wg).max() <= max(GRAD_TOL * np.abs(wg).max(), floor)
    assert rel_err(host(gb), wb) <= GRAD_TOL


LARGE = [(20000, 1, 128, 32, None), (9000, 2, 64, 4, "ragged"), (100003, 5, 260, 1, "ragged"), (60000, 700, 140, 1, "ragged"),
         (20000, 3, 70, 2, "ragged"), (131072, 1, 128, 4, None), (30000, 3000, 32, 4, "ragged"), (50000, 40, 36, 1, "inner")]


@pytest.mark.parametrize("n,samples,c,groups,kind", LARGE)
@pytest.mark.parametrize("hint", [0, 1])
def test_long_samples_and_many_samples(api, n, samples, c, groups, kind, hint):
    """Rows beyond a block's registers, clusters, tiles of several register
    loads, samples that end inside a tile.  A value passes through more roundings in a row
    than at the sizes above: up to 8 register loads of 8 rows with a join each
    (5 operations), 64 slots a thread and the trees, 256 in all, so the bound grows by
    256 / K."""
    rng = np.random.default_rng(n + c)
    ptr = _ptr(rng, n, samples, kind)
    x = (rng.standard_normal((n, c)) * (0.5 + rng.random(c)) + rng.standard_normal(c)).astype(np.float32)
    gamma, beta = (1 + 0.3 * rng.standard_normal(c)).astype(np.float32), rng.standard_normal(c).astype(np.float32)
    gy = rng.standard_normal((n, c)).astype(np.float32)
    longest = n if ptr is None else int(np.diff(ptr).max())
    kw = dict(graph_ptr=_i32(ptr), activation="silu", max_rows=longest if hint else 0)
    y, mean, rstd = api.group_norm_forward(cuda(x), cuda(gamma), cuda(beta), groups, eps=EPS, **kw)
    want, om, orstd, bound = _forward_bound(x, gamma, beta, groups, ptr, "silu")
    m = _inside(ptr, n)
    assert (np.abs(host(y) - want)[m] <= (256 / K * bound)[m]).all()
    gx, gg, gb = api.group_norm_backward(cuda(x), cuda(gamma), cuda(beta), groups, mean, rstd, cuda(gy), **kw)
    wx, wg, wb = onorm.backward(x, gamma, beta, groups, ptr, EPS, "silu", gy)
    assert rel_err(host(gx)[m], wx[m]) <= GRAD_TOL and rel_err(host(gg), wg) <= GRAD_TOL and rel_err(host(gb), wb) <= GRAD_TOL


@pytest.mark.parametrize("width", [16, 10])
@pytest.mark.parametrize("hint", [0, 40])
def test_scalar_block_in_place_and_rows_left_alone(api, width, hint):
    """x[:, 0, :] of features, normalised in place: l > 0 blocks and the rows
    of no graph keep their values, in the gradient too."""
    import torch
    rng = np.random.default_rng(width)
    n, groups, ptr = 120, 2, [4, 40, 40, 79, 100]
    x = rng.standard_normal((n, 4, width)).astype(np.float32)
    gy = rng.standard_normal((n, 4, width)).astype(np.float32)
    gamma, beta = rng.standard_normal(width).astype(np.float32), rng.standard_normal(width).astype(np.float32)
    m = _inside(ptr, n)
    t, g = cuda(x), cuda(gy)
    kw = dict(graph_ptr=_i32(ptr), activation="silu", max_rows=hint)
    out, mean, rstd = api.group_norm_forward(t[:, 0], cuda(gamma), cuda(beta), groups, eps=EPS, out=t[:, 0], **kw)
    assert out.data_ptr() == t.data_ptr()
    want, _, _, bound = _forward_bound(x[:, 0], gamma, beta, groups, ptr, "silu")
    got = host(t)
    assert np.array_equal(got[:, 1:], x[:, 1:]) and np.array_equal(got[~m], x[~m])
    assert (np.abs(got[:, 0] - want)[m] <= bound[m]).all()
    gx, gg, gb = api.group_norm_backward(cuda(x)[:, 0], cuda(gamma), cuda(beta), groups, mean, rstd, g[:, 0],
                                         grad_x=g[:, 0], **kw)
    wx, wg, wb = onorm.backward(x[:, 0], gamma, beta, groups, ptr, EPS, "silu", gy[:, 0])
    got = host(g)
    assert np.array_equal(got[:, 1:], gy[:, 1:]) and np.array_equal(got[~m], gy[~m])
    assert rel_err(got[m, 0], wx[m]) <= GRAD_TOL and rel_err(host(gg), wg) <= GRAD_TOL and rel_err(host(gb), wb) <= GRAD_TOL


@pytest.mark.parametrize("hint", [0, 7, 30, 100000])
def test_hint_that_is_wrong_changes_no_result(api, hint):
    """max_rows below, at and above the longest graph."""
    rng = np.random.default_rng(11)
    n, c, groups, ptr = 5000, 64, 8, [0, 3, 33, 60, 4300, 5000]
    x, gy = (rng.standard_normal((n, c)).astype(np.float32) for _ in range(2))
    ones, zeros = np.ones(c, np.float32), np.zeros(c, np.float32)
    y, mean, rstd = api.group_norm_forward(cuda(x), None, None, groups, graph_ptr=_i32(ptr), activation="silu",
                                           max_rows=hint)
    want, _, _, bound = _forward_bound(x, ones, zeros, groups, ptr, "silu")
    assert (np.abs(host(y) - want) <= bound).all()
    gx, gg, gb = api.group_norm_backward(cuda(x), None, None, groups, mean, rstd, cuda(gy), graph_ptr=_i32(ptr),
                                         activation="silu", max_rows=hint)
    wx, wg, wb = onorm.backward(x, None, None, groups, ptr, EPS, "silu", gy)
    assert rel_err(host(gx), wx) <= GRAD_TOL and rel_err(host(gg), wg) <= GRAD_TOL and rel_err(host(gb), wb) <= GRAD_TOL


@pytest.mark.parametrize("hint", [0, 64])
def test_large_common_offset(api, hint):
    """Deviations are taken before they are squared: an offset of 1000 costs
    the mean's rounding (2^-24 x 1000 x rstd), not the variance."""
    rng = np.random.default_rng(12)
    n, c, groups = 256, 32, 4
    x = (rng.standard_normal((n, c)) + 1000).astype(np.float32)
    ptr = np.arange(0, n + 1, 64)
    _, mean, rstd = api.group_norm_forward(cuda(x), None, None, groups, graph_ptr=_i32(ptr), max_rows=hint)
    _, om, orstd = onorm.forward(x, None, None, groups, ptr, EPS, None)
    assert np.abs(host(rstd) / orstd - 1).max() <= 2 * K * U + (K * U * 1000) ** 2
    assert np.abs(host(mean) - om).max() <= K * U * 1000


@pytest.mark.parametrize("hint", [0, 20])
def test_nonfinite_values_stay_in_their_graph_and_group(api, hint):
    import torch
    rng = np.random.default_rng(13)
    x = rng.standard_normal((60, 16)).astype(np.float32)
    ptr = [0, 20, 40, 60]
    good, _, _ = api.group_norm_forward(cuda(x), None, None, 4, graph_ptr=_i32(ptr), activation="silu", max_rows=hint)
    x[25, 5] = np.nan
    x[50, 15] = np.inf
    y, mean, rstd = api.group_norm_forward(cuda(x), None, None, 4, graph_ptr=_i32(ptr), activation="silu", max_rows=hint)
    bad = np.zeros((60, 16), bool)
    bad[20:40, 4:8] = True
    bad[40:60, 12:16] = True
    assert np.array_equal(host(y)[~bad], host(good)[~bad])
    assert np.isnan(host(y)[20:40, 4:8]).all() and not np.isfinite(host(y)[40:60, 12:16]).any()
    # a NaN gradient of one graph reaches the parameters but no other graph's rows
    gy = np.ones((60, 16), np.float32)
    gy[3, 0] = np.nan
    y, mean, rstd = api.group_norm_forward(good, None, None, 4, graph_ptr=_i32(ptr), max_rows=hint)
    gx, gg, gb = api.group_norm_backward(good, None, None, 4, mean, rstd, cuda(gy), graph_ptr=_i32(ptr), max_rows=hint)
    assert np.isnan(host(gx)[:20, :4]).all() and np.isfinite(host(gx)[20:]).all() and np.isfinite(host(gx)[:, 4:]).all()
    assert np.isnan(host(gb)[0]) and np.isfinite(host(gb)[1:]).all()


def test_infinite_value_leaves_no_number_in_its_group_of_a_long_sample(api):
    """Enough rows for the split by tiles: the variance of a group that holds an
    infinity is no number, and so are its rstd and every result."""
    rng = np.random.default_rng(8)
    n, c = 140000, 128
    ptr = np.array([0, n // 2, n])
    x = rng.standard_normal((n, c)).astype(np.float32)
    x[n // 2 + 4321, 70] = np.inf
    y, mean, rstd = api.group_norm_forward(cuda(x), None, None, 2, graph_ptr=_i32(ptr))
    assert np.isnan(host(rstd)[1, 1]) and np.isfinite(host(rstd)).sum() == 3
    assert np.isnan(host(y)[n // 2:, 64:]).all() and np.isfinite(host(y)).sum() == n * c - n // 2 * 64


@pytest.mark.parametrize("c", [132, 520, 35])
@pytest.mark.parametrize("ptr", [[3, 40, 40, 700, 900], [0, 0, 1000, 1000], [998, 999], list(range(5, 991, 5))])
def test_rows_outside_every_sample_of_wide_groups(api, c, ptr):
    """Groups wider than a fused slab (tiles): rows before, behind and between what
    belongs to a graph may hold anything, and are left as they were; in place and with a row stride."""
    rng = np.random.default_rng(c)
    n, wide = 1000, c + 4
    x, gy = (rng.standard_normal((n, wide)).astype(np.float32) for _ in range(2))
    m = _inside(ptr, n)
    x[~m], gy[~m] = np.nan, np.inf
    gamma, beta = rng.standard_normal(c).astype(np.float32), rng.standard_normal(c).astype(np.float32)
    kw = dict(graph_ptr=_i32(ptr), activation="silu")
    t, g = cuda(x), cuda(gy)
    y, mean, rstd = api.group_norm_forward(t[:, :c], cuda(gamma), cuda(beta), 1, eps=EPS, **kw)
    gx, gg, gb = api.group_norm_backward(t[:, :c], cuda(gamma), cuda(beta), 1, mean, rstd, g[:, :c], grad_x=g[:, :c], **kw)
    clean = np.where(m[:, None], x, 0)[:, :c], np.where(m[:, None], gy, 0)[:, :c]
    want, _, _, bound = _forward_bound(clean[0], gamma, beta, 1, ptr, "silu")
    assert (np.abs(host(y) - want)[m] <= bound[m]).all()
    wx, wg, wb = onorm.backward(clean[0], gamma, beta, 1, ptr, EPS, "silu", clean[1])
    got = host(g)
    assert np.array_equal(got[~m], gy[~m]) and np.array_equal(got[:, c:], gy[:, c:])
    # graphs of one row and few channels: the gradient is what cancels, measured against its terms
    scale = max(np.abs(wx[m]).max(), 0.1 * np.abs(gy[m][:, :c]).max() * np.abs(gamma).max())
    assert np.abs(got[m][:, :c] - wx[m]).max() <= GRAD_TOL * scale
    assert rel_err(host(gg), wg) <= GRAD_TOL and rel_err(host(gb), wb) <= GRAD_TOL


def test_gradient_against_differences(api):
    """Directional differences of the kernel's own forward.

    With step h in a direction d of unit entries the central difference is off by
    h^2/6 |f'''| (f''' of order |d|^3) and by the forward's roundings over h.
    """
    rng = np.random.default_rng(14)
    n, c, groups, ptr = 96, 32, 4, [0, 10, 50, 96]
    x, gy, d = (rng.standard_normal((n, c)).astype(np.float32) for _ in range(3))
    gamma, beta = rng.standard_normal(c).astype(np.float32), rng.standard_normal(c).astype(np.float32)
    kw = dict(graph_ptr=_i32(ptr), activation="silu")

    def f(x):
        y, mean, rstd = api.group_norm_forward(cuda(x.astype(np.float32)), cuda(gamma), cuda(beta), groups, **kw)
        return np.sum(host(y).astype(np.float64) * gy), mean, rstd

    _, mean, rstd = f(x)
    gx, _, _ = api.group_norm_backward(cuda(x), cuda(gamma), cuda(beta), groups, mean, rstd, cuda(gy), **kw)
    h = 2.0 ** -7
    hi, lo = (x + h * d).astype(np.float32), (x - h * d).astype(np.float32)
    want = np.sum(host(gx).astype(np.float64) * (hi.astype(np.float64) - lo))
    # the same difference of the exact forward bounds the truncation; roundings add 16 u sum |y gy| of the two values
    o = lambda x: np.sum(onorm.forward(x, gamma, beta, groups, ptr, EPS, "silu")[0] * gy)
    exact = np.sum(onorm.backward(x, gamma, beta, groups, ptr, EPS, "silu", gy)[0] * (hi.astype(np.float64) - lo))
    truncation = abs(o(hi) - o(lo) - exact)
    roundings = 2 * np.sum(_forward_bound(x, gamma, beta, groups, ptr, "silu")[3] * np.abs(gy))
    assert abs(f(hi)[0] - f(lo)[0] - want) <= truncation + roundings + GRAD_TOL * np.abs(want)


@pytest.mark.parametrize("hint", [0, 33])
def test_streams_graph_replay_and_equal_bits(api, hint):
    import torch
    rng = np.random.default_rng(15)
    n, c, groups, ptr = 900, 64, 8, [0, 30, 63, 63, 90, 500, 900]
    x, gy = (torch.zeros((n, c), device="cuda") for _ in range(2))
    p = _i32(ptr)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            y, mean, rstd = api.group_norm_forward(x, None, None, groups, graph_ptr=p, activation="silu", max_rows=hint)
            gx, gg, gb = api.group_norm_backward(x, None, None, groups, mean, rstd, gy, graph_ptr=p, activation="silu",
                                                 max_rows=hint)
        for _ in range(2):
            xh, gh = (rng.standard_normal((n, c)).astype(np.float32) for _ in range(2))
            x.copy_(cuda(xh))
            gy.copy_(cuda(gh))
            graph.replay()
            s.synchronize()
            wx, wg, wb = onorm.backward(xh, None, None, groups, ptr, EPS, "silu", gh)
            assert rel_err(host(gx), wx) <= GRAD_TOL and rel_err(host(gg), wg) <= GRAD_TOL
            assert rel_err(host(gb), wb) <= GRAD_TOL
            again = api.group_norm_backward(x, None, None, groups, mean, rstd, gy, graph_ptr=p, activation="silu",
                                            max_rows=hint)
            for a, b in zip(again, (gx, gg, gb)):
                assert torch.equal(a, b)


def test_row_offsets_beyond_32_bits(api):
    """70 000 rows, 32 768 floats apart: the last one starts at 2.3e9 floats."""
    import torch
    rng = np.random.default_rng(17)
    n, c, groups, stride = 70000, 8, 2, 32768
    xh, gh = (rng.standard_normal((n, c)).astype(np.float32) for _ in range(2))
    x, g = (torch.empty((n, stride), device="cuda")[:, :c] for _ in range(2))
    x.copy_(cuda(xh))
    g.copy_(cuda(gh))
    ptr = [0, 69990, n]
    for hint in (0, n):
        y, mean, rstd = api.group_norm_forward(x, None, None, groups, graph_ptr=_i32(ptr), activation="silu", max_rows=hint)
        gx, gg, gb = api.group_norm_backward(x, None, None, groups, mean, rstd, g, graph_ptr=_i32(ptr), activation="silu",
                                             max_rows=hint, grad_x=g if hint else None)
        want = onorm.forward(xh, None, None, groups, ptr, EPS, "silu")[0]
        wx, wg, wb = onorm.backward(xh, None, None, groups, ptr, EPS, "silu", gh)
        # sums of 280 000 values: in runs of a few hundred (tiles, chunks of registers) joined by trees
        assert rel_err(host(y), want) <= 4 * K * U
        assert rel_err(host(gx), wx) <= GRAD_TOL and rel_err(host(gg), wg) <= GRAD_TOL and rel_err(host(gb), wb) <= GRAD_TOL


def test_requested_outputs_alone_and_empty(api):
    import torch
    rng = np.random.default_rng(16)
    x, gy = (cuda(rng.standard_normal((50, 8)).astype(np.float32)) for _ in range(2))
    y, mean, rstd = api.group_norm_forward(x, None, None, 2)
    full = api.group_norm_backward(x, None, None, 2, mean, rstd, gy)
    a = api.group_norm_backward(x, None, None, 2, mean, rstd, gy, want_params=False)
    b = api.group_norm_backward(x, None, None, 2, mean, rstd, gy, want_x=False)
    assert a[1] is None and a[2] is None and b[0] is None
    assert torch.equal(a[0], full[0]) and torch.equal(b[1], full[1]) and torch.equal(b[2], full[2])
    none = torch.empty((0, 8), device="cuda")
    for ptr, samples in ((None, 1), (_i32([0, 0, 0]), 2), (_i32([0]), 0)):
        y, mean, rstd = api.group_norm_forward(none, None, None, 2, graph_ptr=ptr)
        assert y.shape == (0, 8) and mean.shape == (samples, 2) and not mean.any()
        assert np.allclose(host(rstd), 1 / np.sqrt(EPS))
        gx, gg, gb = api.group_norm_backward(none, None, None, 2, mean, rstd, none, graph_ptr=ptr)
        assert gx.shape == (0, 8) and not gg.any() and not gb.any()


def test_refusals(api):
    import torch
    x = torch.zeros((6, 8), device="cuda")
    v = torch.zeros(8, device="cuda")
    s = torch.zeros((1, 2), device="cuda")
    for bad in (lambda: api.group_norm_forward(x[:, :0], None, None, 1), lambda: api.group_norm_forward(x, v, v, 3), lambda: api.group_norm_forward(x, v, v, 0),
                lambda: api.group_norm_forward(x.half(), v, v, 2), lambda: api.group_norm_forward(x.cpu(), v, v, 2),
                lambda: api.group_norm_forward(x, v[:4], v, 2), lambda: api.group_norm_forward(x.t(), None, None, 2),
                lambda: api.group_norm_forward(x, v, v, 2, activation="relu"),
                lambda: api.group_norm_forward(x, v, v, 2, graph_ptr=torch.zeros(2, dtype=torch.int64, device="cuda")),
                lambda: api.group_norm_forward(x, v, v, 2, out=torch.zeros((6, 7), device="cuda")),
                lambda: api.group_norm_backward(x, v, v, 2, s[:, :1].contiguous(), s, x),
                lambda: api.group_norm_backward(x, v, v, 2, s, s, x[:5])):
        with pytest.raises(ValueError):
            bad()
    from equivariant_mlip_tensor_b200 import CGTPError
    with pytest.raises(CGTPError):
        api.group_norm_forward(x, v, v, 2, eps=0.0)
