"""Token sort, embedding and its table gradient against the fp64 oracle.

Tolerances, with u = 2^-24 (half a step of fp32): the forward is one rounded
product, so it equals the fp32 product bit for bit.  In the gradient each
term passes through fewer than count + 2 rounded operations (its additions and
the scale), so an entry is off by at most (count + 2) u scale sum |grad_out|
to first order; 1.01 covers the higher orders up to count = 100 000.
"""
import numpy as np
import pytest

from oracle import embed as oembed
from tests.gpu_common import cuda, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def api():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from equivariant_mlip_tensor_b200 import api as a
    return a


def _tokens(rng, n, rows, kind):
    if kind == "one":
        t = np.full(n, rows - 1)
    elif kind == "skew":
        t = (rows * rng.random(n) ** 4).astype(np.int64)
    elif kind == "none":
        t = np.where(rng.random(n) < 0.5, -1, rows)  # no token is a row
    else:
        t = rng.integers(0, rows, n)
        t[rng.random(n) < 0.1] = -1
        t[rng.random(n) < 0.05] = 2 ** 31 - 1
    return t.astype(np.int32)


def _check_backward(got, tok, rows, g, scale):
    want = oembed.backward(tok, rows, g, scale)
    mag = oembed.backward(tok, rows, np.abs(g), abs(scale))
    count = np.bincount(tok[(tok >= 0) & (tok < rows)], minlength=rows)[:, None]
    bad = np.abs(host(got) - want) > 1.01 * (count + 2) * U * mag
    assert not bad.any(), np.argwhere(bad)[:4]


@pytest.mark.parametrize("n,rows", [(1, 1), (5, 3), (31, 300), (4096, 255), (4097, 256), (9001, 70000), (20000, 3),
                                    (60000, 17000000), (33, 2 ** 31 - 1)])
def test_sort_is_stable(api, n, rows):
    rng = np.random.default_rng(n)
    for kind in ("mixed", "skew", "one"):
        tok = _tokens(rng, n, rows, kind)
        o = api.token_sort(cuda(tok), rows)
        order, srt = oembed.sort(tok, rows)
        assert np.array_equal(host(o.order), order) and np.array_equal(host(o.sorted), srt)


def test_sort_beyond_the_repeated_tile_sums(api):
    """More than 256 tiles of 4 096 tokens: the sort's prefix launches."""
    tok = np.random.default_rng(7).integers(-5, 1000, 1_100_003).astype(np.int32)
    o = api.token_sort(cuda(tok), 998)
    order, srt = oembed.sort(tok, 998)
    assert np.array_equal(host(o.order), order) and np.array_equal(host(o.sorted), srt)


@pytest.mark.parametrize("n,rows,width", [(1, 1, 1), (1, 5, 4), (7, 3, 8), (33, 70, 13), (257, 4, 128), (513, 1000, 96),
                                          (1000, 16, 260), (2049, 5, 3), (65, 9, 1028), (3000, 600, 64)])
@pytest.mark.parametrize("kind", ["mixed", "skew", "one", "none"])
def test_both_directions_match_the_oracle(api, n, rows, width, kind):
    rng = np.random.default_rng(n + rows + width)
    tok = _tokens(rng, n, rows, kind)
    table = rng.standard_normal((rows, width)).astype(np.float32)
    g = rng.standard_normal((n, width)).astype(np.float32)
    out = host(api.embed_forward(cuda(tok), cuda(table), scale=0.7))
    valid = (tok >= 0) & (tok < rows)
    want = np.where(valid[:, None], np.float32(0.7) * table[np.where(valid, tok, 0)], np.float32(0))
    assert np.array_equal(out, want)
    got = api.embed_backward(api.token_sort(cuda(tok), rows), cuda(g), scale=-0.7)
    _check_backward(got, tok, rows, g, float(np.float32(-0.7)))


@pytest.mark.parametrize("width", [8, 6, 128])
def test_scalar_block_of_features_in_place(api, width):
    """Rows with a stride: only the l = 0 block is written, and read."""
    import torch
    rng = np.random.default_rng(width)
    n, rows = 90, 11
    tok = _tokens(rng, n, rows, "mixed")
    table = rng.standard_normal((rows, width)).astype(np.float32)
    x = torch.full((n, 9, width), 5.0, device="cuda")
    api.embed_forward(cuda(tok), cuda(table), out=x[:, 0, :])
    assert bool((x[:, 1:] == 5.0).all())
    assert np.array_equal(host(x[:, 0]), oembed.forward(tok, table, 1.0).astype(np.float32))
    g = rng.standard_normal((n, 9, width)).astype(np.float32)
    got = api.embed_backward(api.token_sort(cuda(tok), rows), cuda(g)[:, 0, :])
    _check_backward(got, tok, rows, g[:, 0], 1.0)
    # a view that starts off a 16-byte boundary takes the scalar path
    wide = torch.zeros((n, width + 1), device="cuda")
    api.embed_forward(cuda(tok), cuda(table), out=wide[:, 1:])
    assert np.array_equal(host(wide[:, 1:]), oembed.forward(tok, table, 1.0).astype(np.float32))
    assert not bool(wide[:, 0].any())


@pytest.mark.parametrize("rows,width", [(40000, 12), (40003, 7), (300007, 8), (64, 260)])
@pytest.mark.parametrize("n", [1, 40, 9000])
def test_rows_without_a_token_are_cleared(api, rows, width, n):
    """More rows than the clearing blocks search at once, in whole pieces of 32 rows and between tokens."""
    import torch
    rng = np.random.default_rng(rows + n)
    tok = rng.integers(0, rows, n).astype(np.int32)
    g = rng.standard_normal((n, width)).astype(np.float32)
    out = torch.full((rows, width), float("nan"), device="cuda")
    api.embed_backward(api.token_sort(cuda(tok), rows), cuda(g), out=out)
    assert not out[torch.from_numpy(np.setdiff1d(np.arange(rows), tok)).cuda()].any()
    _check_backward(out, tok, rows, g, 1.0)


def test_long_sums_cross_many_chunks(api):
    """One row takes nearly every token: its sum is joined from hundreds of chunks."""
    rng = np.random.default_rng(3)
    n, rows, width = 70000, 40, 16
    tok = np.where(rng.random(n) < 0.995, 7, rng.integers(0, rows, n)).astype(np.int32)
    g = rng.standard_normal((n, width)).astype(np.float32)
    o = api.token_sort(cuda(tok), rows)
    got = api.embed_backward(o, cuda(g))
    _check_backward(got, tok, rows, g, 1.0)
    assert np.array_equal(host(got), host(api.embed_backward(o, cuda(g))))  # the same bits again


@pytest.mark.parametrize("width", [3, 8, 64, 128, 130])
def test_runs_that_end_around_every_join_length(api, width):
    """Rows whose tokens fill a given number of 16-position chunks, one less and one
    more: joined by one worker alone, or by a block's workers together."""
    rng = np.random.default_rng(width)
    lengths = [16 * k + d for k in (0, 1, 2, 14, 15, 16, 17, 18, 30, 31, 32, 33, 34, 60) for d in (-1, 0, 1) if 16 * k + d >= 0]
    rng.shuffle(lengths)
    rows = len(lengths)
    tok = rng.permutation(np.repeat(np.arange(rows), lengths)).astype(np.int32)
    g = rng.standard_normal((tok.size, width)).astype(np.float32)
    o = api.token_sort(cuda(tok), rows)
    got = api.embed_backward(o, cuda(g), scale=0.5)
    _check_backward(got, tok, rows, g, 0.5)
    assert np.array_equal(host(got), host(api.embed_backward(o, cuda(g), scale=0.5)))


def test_gradient_against_differences(api):
    """The gradient is the forward's: <embed(table + h d), g> grows by h <grad, d>."""
    rng = np.random.default_rng(4)
    n, rows, width = 200, 12, 20
    tok = cuda(_tokens(rng, n, rows, "mixed"))
    table, d = (rng.standard_normal((rows, width)).astype(np.float32) for _ in range(2))
    g = rng.standard_normal((n, width)).astype(np.float32)
    grad = host(api.embed_backward(api.token_sort(tok, rows), cuda(g), scale=1.5)).astype(np.float64)
    f = lambda t: np.sum(host(api.embed_forward(tok, cuda(t), scale=1.5)).astype(np.float64) * g)
    hi, lo = (table + 0.5 * d).astype(np.float32), (table - 0.5 * d).astype(np.float32)
    want = np.sum(grad * (hi.astype(np.float64) - lo))
    # linear in the table: only roundings, u per entry of either side and (count + 2) u in the gradient
    mag = 1.5 * np.sum(np.abs(host(api.embed_forward(tok, cuda(np.abs(hi) + np.abs(lo))))) * np.abs(g))
    assert abs(f(hi) - f(lo) - want) <= (n + 4) * U * mag


def test_empty_and_zero_sized(api):
    import torch
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    table = torch.ones((3, 4), device="cuda")
    assert api.embed_forward(none, table).shape == (0, 4)
    o = api.token_sort(none, 3)
    out = torch.full((3, 4), 9.0, device="cuda")
    assert not api.embed_backward(o, torch.empty((0, 4), device="cuda"), out=out).any()
    # a table without rows: every token is padding
    tok = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert not api.embed_forward(tok, torch.empty((0, 4), device="cuda")).any()
    assert api.embed_backward(api.token_sort(tok, 0), torch.ones((5, 4), device="cuda")).shape == (0, 4)
    assert api.embed_forward(tok, torch.empty((3, 0), device="cuda")).shape == (5, 0)


def test_disordered_order_stays_in_bounds(api):
    """Entries out of range are left out; the untouched sums stay right."""
    import torch
    rng = np.random.default_rng(5)
    g = cuda(rng.standard_normal((100, 8)).astype(np.float32))
    order = torch.arange(100, dtype=torch.int32, device="cuda")
    srt = torch.arange(100, dtype=torch.int32, device="cuda") // 10
    want = api.embed_backward(api.TokenOrder(10, order, srt), g)
    bad = order.clone()
    bad[3], bad[95] = -7, 1 << 30
    got = api.embed_backward(api.TokenOrder(10, bad, srt), g)
    assert torch.equal(got[1:9], want[1:9])
    far = srt.clone()
    far[90:] = 1 << 30
    got = api.embed_backward(api.TokenOrder(10, order, far), g)
    assert torch.equal(got[:9], want[:9]) and not got[9].any()


def test_nonfinite_values_stay_in_their_row(api):
    import torch
    tok = torch.tensor([0, 1, -1, 2, 1], dtype=torch.int32, device="cuda")
    table = torch.tensor([[1.0, 2], [float("inf"), float("nan")], [3, 4]], device="cuda")
    out = api.embed_forward(tok, table, scale=2.0)
    assert torch.equal(out[[0, 2, 3]], torch.tensor([[2.0, 4], [0, 0], [6, 8]], device="cuda"))
    assert torch.isinf(out[1, 0]) and torch.isnan(out[4, 1])
    g = torch.ones((5, 2), device="cuda")
    g[2] = float("nan")  # the gradient of padding
    g[3, 0] = float("inf")
    grad = api.embed_backward(api.token_sort(tok, 3), g)
    assert torch.equal(grad[:2], torch.tensor([[1.0, 1], [2, 2]], device="cuda"))
    assert torch.isinf(grad[2, 0]) and grad[2, 1] == 1


def test_offsets_beyond_32_bits(api):
    """Rows 32 768 floats apart (the last starts at 2.3e9), as features, as the
    gradient of features and as rows of the table."""
    import torch
    rng = np.random.default_rng(8)
    n, rows, width, stride = 70000, 50, 8, 32768
    tok = _tokens(rng, n, rows, "mixed")
    table, gh = (rng.standard_normal(s).astype(np.float32) for s in ((rows, width), (n, width)))
    wide = torch.empty((n, stride), device="cuda")
    api.embed_forward(cuda(tok), cuda(table), out=wide[:, :width])
    valid = (tok >= 0) & (tok < rows)
    assert np.array_equal(host(wide[:, :width].contiguous()), np.where(valid[:, None], table[np.where(valid, tok, 0)], 0))
    wide[:, :width].copy_(cuda(gh))
    _check_backward(api.embed_backward(api.token_sort(cuda(tok), rows), wide[:, :width]), tok, rows, gh, 1.0)
    few = torch.tensor([69999, 0, 69999], dtype=torch.int32, device="cuda")
    out = api.embed_forward(few, wide)
    assert torch.equal(out[0], wide[69999]) and torch.equal(out[1], wide[0])
    grad = api.embed_backward(api.token_sort(few, n), out, out=wide)  # the table's own storage
    assert torch.equal(grad[69999], out[0] + out[2]) and torch.equal(grad[0], out[1])
    assert not grad[1:69999].any()


def test_streams_and_graph_replay(api):
    """On another stream than the default one, and captured once, replayed on new inputs."""
    import torch
    rng = np.random.default_rng(6)
    n, rows, width = 5000, 700, 32
    s = torch.cuda.Stream()
    tok, g = (torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty((n, width), device="cuda"))
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        tok.zero_(), g.zero_()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            got = api.embed_backward(api.token_sort(tok, rows), g)
        for seed in (1, 2):
            t = _tokens(np.random.default_rng(seed), n, rows, "mixed")
            gh = rng.standard_normal((n, width)).astype(np.float32)
            tok.copy_(cuda(t))
            g.copy_(cuda(gh))
            graph.replay()
            s.synchronize()
            _check_backward(got, t, rows, gh, 1.0)


def test_refusals(api):
    import torch
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    table = torch.zeros((3, 8), device="cuda")
    for bad in (lambda: api.embed_forward(tok.long(), table), lambda: api.embed_forward(tok.cpu(), table),
                lambda: api.embed_forward(tok, table.half()), lambda: api.embed_forward(tok, table[0]),
                lambda: api.embed_forward(tok, table, out=torch.zeros((4, 9), device="cuda")),
                lambda: api.embed_forward(tok, table, out=torch.zeros((8, 4), device="cuda").t()),
                lambda: api.embed_forward(tok, table, out=torch.zeros((1, 8), device="cuda").expand(4, 8)),
                lambda: api.embed_backward(api.token_sort(tok, 3), torch.zeros((5, 8), device="cuda")),
                lambda: api.embed_backward(api.token_sort(tok, 3), torch.zeros((4, 8), device="cuda"),
                                           out=torch.zeros((4, 8), device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    from equivariant_mlip_tensor_b200 import CGTPError
    with pytest.raises(CGTPError):
        api.token_sort(tok, -1)
    with pytest.raises(CGTPError):
        api.token_sort(tok.repeat(5000), 3, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
