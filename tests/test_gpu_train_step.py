"""One training step through the library: species -> embedding -> fully
connected convolution -> per-graph group norm with SiLU -> energy, its gradient back to
the embedding table, the norm's parameters and the mixing matrices, and the
orthogonalised update of the latter, each against the fp64 oracle's chain.

Tolerances: the library's measures for forward values (1e-5 of the largest)
and gradients (1e-4); the loss is a sum of n x mult_out terms, so it is held to
1e-5 of the sum of their magnitudes.
"""
import numpy as np
import pytest

from oracle import conv as oconv
from oracle import embed as oembed
from oracle import graph as ograph
from oracle import norm as onorm
from oracle import ortho as oortho
from tests.gpu_common import FWD_TOL, GRAD_TOL, cuda, host, rel_err

pytestmark = pytest.mark.gpu

L, MULT, MULT_OUT, SPECIES, GROUPS, EPS = (1, 1, 1), 16, 32, 5, 4, 1e-5
GRAPHS, ATOMS = 6, 11


@pytest.fixture(scope="module")
def api():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from equivariant_mlip_tensor_b200 import api as a
    return a


def _inputs(seed=0):
    rng = np.random.default_rng(seed)
    n = GRAPHS * ATOMS
    d = {"pos": (rng.random((n, 3)) * 4.0).astype(np.float32),
         "ptr": np.arange(0, n + 1, ATOMS, dtype=np.int32),
         "species": rng.integers(0, SPECIES, n).astype(np.int32)}
    d["gid"] = np.repeat(np.arange(GRAPHS, dtype=np.int32), ATOMS)
    d["species"][[3, 40]] = -1  # atoms whose features come from elsewhere
    n_paths = 5
    d["table"] = rng.standard_normal((SPECIES, MULT)).astype(np.float32)
    d["mix"] = (rng.standard_normal((n_paths, MULT, MULT_OUT)) / np.sqrt(MULT)).astype(np.float32)
    d["gamma"] = (1 + 0.2 * rng.standard_normal(MULT_OUT)).astype(np.float32)
    d["beta"] = (0.2 * rng.standard_normal(MULT_OUT)).astype(np.float32)
    d["cot"] = rng.standard_normal((n, MULT_OUT)).astype(np.float32)  # dE/dy
    o = ograph.neighbour_list(d["pos"], 3.0, None, d["gid"])
    d["o"] = o
    d["w"] = rng.standard_normal((o["col"].size, n_paths, MULT)).astype(np.float32)
    return d


def _step(api, d, table=None):
    """(loss, every gradient, the orthogonalised update) on the GPU."""
    import torch
    n = d["pos"].shape[0]
    plan = api.Plan(*L, MULT)
    g = api.build_graph(cuda(d["pos"]), 3.0, graph_ptr=cuda(d["ptr"]))
    table = cuda(d["table"] if table is None else table)
    w, mix, gamma, beta, cot, ptr, tok = (cuda(d[k]) for k in ("w", "mix", "gamma", "beta", "cot", "ptr", "species"))
    x = torch.zeros((n, 4, MULT), device="cuda")
    api.embed_forward(tok, table, scale=2.0, out=x[:, 0])
    f = plan.uvw_forward(g, x, w, mix)
    y, mean, rstd = api.group_norm_forward(f[:, 0], gamma, beta, GROUPS, graph_ptr=ptr, eps=EPS, activation="silu",
                                           max_rows=ATOMS)
    loss = (y.double() * cot.double()).sum().item()
    gf = torch.zeros_like(f)
    _, ggamma, gbeta = api.group_norm_backward(f[:, 0], gamma, beta, GROUPS, mean, rstd, cot, graph_ptr=ptr,
                                               activation="silu", max_rows=ATOMS, grad_x=gf[:, 0])
    gx, _, gmix, _ = plan.uvw_backward(g, x, w, mix, gf)
    gtable = api.embed_backward(api.token_sort(tok, SPECIES), gx[:, 0], scale=2.0)
    return {"loss": loss, "y": y, "ggamma": ggamma, "gbeta": gbeta, "gmix": gmix, "gtable": gtable,
            "update": api.orthogonalise(gmix)}


def _oracle(d):
    o, n = d["o"], d["pos"].shape[0]
    x = np.zeros((n, 4, MULT))
    x[:, 0] = oembed.forward(d["species"], d["table"], 2.0)
    f = oconv.conv_uvw_forward(o["row_ptr"], o["col"], o["edge_vec"], x, d["w"], d["mix"], *L)
    y, _, _ = onorm.forward(f[:, 0], d["gamma"], d["beta"], GROUPS, d["ptr"], EPS, "silu")
    gf = np.zeros_like(f)
    gf[:, 0], ggamma, gbeta = onorm.backward(f[:, 0], d["gamma"], d["beta"], GROUPS, d["ptr"], EPS, "silu", d["cot"])
    gx, _, gmix, _ = oconv.conv_uvw_backward(o["row_ptr"], o["col"], o["edge_vec"], x, d["w"], d["mix"], gf, *L)
    return {"loss": np.sum(y * d["cot"]), "scale": np.sum(np.abs(y * d["cot"])), "y": y, "ggamma": ggamma, "gbeta": gbeta,
            "gmix": gmix, "gtable": oembed.backward(d["species"], SPECIES, gx[:, 0], 2.0)}


def test_step_matches_the_oracle_chain(api):
    d = _inputs()
    got, want = _step(api, d), _oracle(d)
    assert abs(got["loss"] - want["loss"]) <= FWD_TOL * want["scale"]
    assert rel_err(host(got["y"]), want["y"]) <= FWD_TOL * 10  # through a norm of sums: their error over their spread
    for k in ("ggamma", "gbeta", "gmix", "gtable"):
        assert rel_err(host(got[k]), want[k]) <= GRAD_TOL, k
    # the update of the kernel's own gradient (its bound: test_gpu_ortho)
    for p in range(got["gmix"].shape[0]):
        want = oortho.orthogonalise(host(got["gmix"][p]))
        assert np.linalg.norm(host(got["update"][p]) - want) <= 1e-3 * max(1e-30, np.linalg.norm(want))


def test_table_gradient_against_differences_of_the_step(api):
    """The loss along a direction of the table, by central differences of the
    step's own forward; the truncation is the oracle's at the same points."""
    d = _inputs(1)
    rng = np.random.default_rng(2)
    v = rng.standard_normal(d["table"].shape)
    h = 2.0 ** -6
    hi, lo = (d["table"] + h * v).astype(np.float32), (d["table"] - h * v).astype(np.float32)
    step = hi.astype(np.float64) - lo
    got = _step(api, d, hi)["loss"] - _step(api, d, lo)["loss"]
    along = np.sum(host(_step(api, d)["gtable"]).astype(np.float64) * step)
    ohi, olo, o = _oracle({**d, "table": hi}), _oracle({**d, "table": lo}), _oracle(d)
    truncation = abs(ohi["loss"] - olo["loss"] - np.sum(o["gtable"] * step))
    assert abs(got - along) <= truncation + 2 * FWD_TOL * o["scale"] + GRAD_TOL * np.sum(np.abs(o["gtable"] * step))


def test_step_captured_and_replayed(api):
    """The whole step as a graph: equal bits on the same inputs, and new inputs
    give what the eager step gives."""
    import torch
    d = _inputs(3)
    n, plan = d["pos"].shape[0], api.Plan(*L, MULT)
    g = api.build_graph(cuda(d["pos"]), 3.0, graph_ptr=cuda(d["ptr"]))
    table, w, mix, gamma, beta, cot, ptr, tok = (cuda(d[k]) for k in ("table", "w", "mix", "gamma", "beta", "cot", "ptr",
                                                                      "species"))
    x, gf = torch.zeros((n, 4, MULT), device="cuda"), torch.zeros((n, 4, MULT_OUT), device="cuda")

    def step():
        api.embed_forward(tok, table, scale=2.0, out=x[:, 0])
        f = plan.uvw_forward(g, x, w, mix)
        y, mean, rstd = api.group_norm_forward(f[:, 0], gamma, beta, GROUPS, graph_ptr=ptr, activation="silu")
        _, gg, gb = api.group_norm_backward(f[:, 0], gamma, beta, GROUPS, mean, rstd, cot, graph_ptr=ptr,
                                            activation="silu", grad_x=gf[:, 0])
        gx, _, gmix, _ = plan.uvw_backward(g, x, w, mix, gf)
        return (y, gg, gb, gmix, api.embed_backward(api.token_sort(tok, SPECIES), gx[:, 0], scale=2.0),
                api.orthogonalise(gmix))

    eager = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            out = step()
        graph.replay()
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
        rng = np.random.default_rng(4)
        table.copy_(cuda(rng.standard_normal(d["table"].shape).astype(np.float32)))
        tok.copy_(cuda(rng.integers(0, SPECIES, n).astype(np.int32)))
        graph.replay()
        s.synchronize()
        again = step()
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_two_streams_at_once(api):
    """The same calls on two streams with their own tensors do not disturb one another."""
    import torch
    rng = np.random.default_rng(5)
    cases = []
    for k in range(2):
        n, rows = 3000 + 1000 * k, 60
        cases.append((cuda(rng.integers(0, rows, n).astype(np.int32)), rows,
                      cuda(rng.standard_normal((n, 64)).astype(np.float32)),
                      cuda(rng.standard_normal((4, 96, 80 + 200 * k)).astype(np.float32))))

    def work(c):
        tok, rows, g, m = c
        y, mean, rstd = api.group_norm_forward(g, None, None, 8, activation="silu")
        return (api.embed_backward(api.token_sort(tok, rows), g), y,
                *api.group_norm_backward(g, None, None, 8, mean, rstd, y, activation="silu"), api.orthogonalise(m))

    want = [work(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        got = []
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(work(c))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


FIRST_CALLS = """
import torch
from equivariant_mlip_tensor_b200 import api
s = torch.cuda.Stream()
tok = torch.arange(20000, dtype=torch.int32, device="cuda") % 7
g = torch.ones((20000, 8), device="cuda")
m = [torch.randn(2, *k, device="cuda") for k in ((8, 8), (16, 600), (150, 160))]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=s):
    x = api.embed_forward(tok, g[:7])
    t = api.embed_backward(api.token_sort(tok, 7), g)
    few = api.embed_backward(api.token_sort(tok[:500].contiguous(), 7), g[:500])
    y, mean, rstd = api.group_norm_forward(g, None, None, 2, activation="silu")
    b = api.group_norm_backward(g, None, None, 2, mean, rstd, x, activation="silu")
    o = [api.orthogonalise(k) for k in m]
graph.replay()
torch.cuda.synchronize()
want = torch.bincount(tok.long()).float()[:, None].expand(7, 8)
assert torch.equal(t, want) and torch.equal(x, g) and not y.any() and all(torch.isfinite(k).all() for k in o)
assert torch.equal(few.sum(0), torch.full((8,), 500.0, device="cuda"))
print("captured")
"""


def test_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
