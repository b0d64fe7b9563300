"""The training-side operators of the library, as a user's program calls them.

Three operators, each in every direction it has: the embedding lookup with its
gradient by sorted tokens, the per-graph group norm with SiLU over channels-last
scalars, and the Newton-Schulz orthogonalisation of an update of the mixing
matrices.  ``run`` is one pass: in elementary torch operations where ``own`` is
false, through the library's entry points where it is true.
"""
import math

import torch

own = False

# quintic of the orthogonalisation and the floor of its norm
NS_A, NS_B, NS_C, NS_EPS = 3.4445, -4.7750, 2.0315, 1e-7
NORM_EPS = 1e-5


def listed():
    return [
        # species of 32 atoms into the scalar block of l <= 1 features: latency
        {"name": "embed_forward_tiny", "op": "embed_forward", "n": 32, "rows": 4, "width": 8, "lmax": 1},
        # a large vocabulary, one row per token
        {"name": "embed_forward_large", "op": "embed_forward", "n": 131072, "rows": 65536, "width": 256, "lmax": 0},
        # species gradient of 256 molecules of 30 atoms: few rows, long sums, scalar block of l <= 2 features
        {"name": "embed_backward_molecules", "op": "embed_backward", "n": 7680, "rows": 16, "width": 128, "lmax": 2},
        # many tokens over a large vocabulary: short and long sums mixed
        {"name": "embed_backward_large", "op": "embed_backward", "n": 200003, "rows": 50021, "width": 256, "lmax": 0},
        # scalars of 256 molecules of 30 atoms between two convolutions
        {"name": "norm_forward_molecules", "op": "norm_forward", "n": 7680, "samples": 256, "channels": 128, "groups": 8,
         "lmax": 2, "ragged": False},
        # read-out scalars of one periodic cell of 20000 atoms: one long sample
        {"name": "norm_forward_bulk", "op": "norm_forward", "n": 20000, "samples": 1, "channels": 128, "groups": 32,
         "lmax": 0, "ragged": False},
        # the training pass of the molecules
        {"name": "norm_backward_molecules", "op": "norm_backward", "n": 7680, "samples": 256, "channels": 128,
         "groups": 8, "lmax": 2, "ragged": False},
        # graphs of very different sizes, empty ones among them
        {"name": "norm_backward_ragged", "op": "norm_backward", "n": 131101, "samples": 61, "channels": 256, "groups": 32,
         "lmax": 0, "ragged": True},
        # mixing matrices of the smallest workload: latency
        {"name": "orthogonalise_tiny", "op": "orthogonalise", "batch": 5, "m": 8, "n": 8},
        # mixing matrices of the l <= 2 interaction with harmonics to l = 4, multiplicity 128
        {"name": "orthogonalise_mixing", "op": "orthogonalise", "batch": 15, "m": 128, "n": 128},
        # the radial network's output weights of the same layer: short and wide
        {"name": "orthogonalise_radial", "op": "orthogonalise", "batch": 1, "m": 64, "n": 1920},
        # two large dense layers
        {"name": "orthogonalise_large", "op": "orthogonalise", "batch": 2, "m": 1024, "n": 1024},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed_forward", "embed_backward", "norm_forward", "norm_backward", "orthogonalise"])
    if op.startswith("embed"):
        width = rng.choice([1, 1, 4, 4, 4]) * _spread(rng, 1, 128)
        n = min(_spread(rng, 1, 200000), 50000000 // width)
        rows = min(_spread(rng, 1, 100000), 12000000 // width)
        return {"op": op, "n": n, "rows": rows, "width": width, "lmax": rng.choice([0, 0, 1, 2])}
    if op.startswith("norm"):
        groups = rng.choice([1, 2, 4, 8, 16, 32])
        channels = groups * _spread(rng, 1, 32)
        n = min(_spread(rng, 1, 130000), 33000000 // channels)
        return {"op": op, "n": n, "samples": _spread(rng, 1, max(1, min(2000, n))), "channels": channels,
                "groups": groups, "lmax": rng.choice([0, 0, 1, 2]), "ragged": rng.random() < 0.6}
    m, n = _spread(rng, 4, 1024), _spread(rng, 4, 1024)
    if rng.random() < 0.5:  # multiplicities come in multiples of 4
        m, n = max(4, m // 4 * 4), max(4, n // 4 * 4)
    return {"op": op, "batch": min(_spread(rng, 1, 64), max(1, 2 * 1024 ** 3 // (m * n * min(m, n)))), "m": m, "n": n}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _tokens(case, g):
    """Tokens of a batch: frequent and rare rows (a power law), and some -1, which stand for no token."""
    u = torch.rand(case["n"], device="cuda", generator=g)
    t = (case["rows"] * u ** 3).to(torch.int32).clamp_(max=case["rows"] - 1)
    pad = torch.rand(case["n"], device="cuda", generator=g) < 0.02
    t = torch.where(pad, torch.full_like(t, -1), t)
    t[0] = case["rows"] - 1
    return t


def _features(n, lmax, width, g):
    return torch.randn((n, (lmax + 1) ** 2, width), device="cuda", generator=g)


def _samples(case, g):
    """Start rows of the graphs: equal ones, or random cuts (empty and one-row graphs among them)."""
    n, b = case["n"], case["samples"]
    if case["ragged"]:
        cuts = torch.randint(0, n + 1, (b - 1,), device="cuda", generator=g).sort().values
        if b > 8:
            cuts[2] = cuts[1]  # an empty graph
    else:
        cuts = torch.arange(1, b, device="cuda") * n // b
    ends = torch.tensor([0, n], device="cuda")
    return torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)


def prepare(case, seed):
    g, op, s = _generator(seed), case["op"], dict(case)
    if op.startswith("embed"):
        s["tokens"], s["scale"] = _tokens(case, g), math.sqrt(case["width"])
        if op == "embed_forward":
            s["table"] = torch.randn((case["rows"], case["width"]), device="cuda", generator=g) / math.sqrt(case["width"])
            s["x"] = torch.zeros((case["n"], (case["lmax"] + 1) ** 2, case["width"]), device="cuda")
        else:
            s["grad_x"] = _features(case["n"], case["lmax"], case["width"], g)
    elif op.startswith("norm"):
        c = case["channels"]
        x = _features(case["n"], case["lmax"], c, g)
        s["x"] = x * (0.5 + torch.rand(c, device="cuda", generator=g)) + 0.5 * torch.randn(c, device="cuda", generator=g)
        s["gamma"] = 1 + 0.2 * torch.randn(c, device="cuda", generator=g)
        s["beta"] = 0.2 * torch.randn(c, device="cuda", generator=g)
        s["ptr"] = _samples(case, g)
        s["max_rows"] = int((s["ptr"][1:] - s["ptr"][:-1]).max())  # the graphs' sizes are known where they are made
        if op == "norm_backward":
            s["grad_y"] = _features(case["n"], case["lmax"], c, g)
            s["mean"], s["rstd"] = _statistics(s["x"][:, 0], s["ptr"], case["groups"], torch.float64)
            s["mean"], s["rstd"] = s["mean"].float(), s["rstd"].float()
    else:
        # gradients of the mixing matrices: channels of unequal strength
        rows = torch.exp(0.3 * torch.randn((case["batch"], case["m"], 1), device="cuda", generator=g))
        s["update"] = rows * 1e-3 * torch.randn((case["batch"], case["m"], case["n"]), device="cuda", generator=g)
    return s


def _row_sample(ptr, n):
    """The graph of each row."""
    return torch.bucketize(torch.arange(n, device=ptr.device, dtype=ptr.dtype), ptr[1:], right=True)


def _per_sample(v, sample, b):
    """Sums over the rows of each graph, in 64 bits (graphs may be long)."""
    return torch.zeros((b,) + v.shape[1:], dtype=torch.float64, device=v.device).index_add_(0, sample, v.double())


def _statistics(x, ptr, groups, dtype):
    n, b = x.shape[0], ptr.numel() - 1
    sample = _row_sample(ptr, n)
    v = x.reshape(n, groups, -1)
    count = ((ptr[1:] - ptr[:-1]).double() * v.shape[2]).clamp(min=1)[:, None]
    mean = _per_sample(v.to(dtype).sum(2), sample, b) / count
    d = v.to(dtype) - mean.to(dtype)[sample][:, :, None]
    var = _per_sample((d * d).sum(2), sample, b) / count
    return mean.to(dtype), (1 / torch.sqrt(var + NORM_EPS)).to(dtype)


def _plain_embed_forward(s):
    valid = ((s["tokens"] >= 0) & (s["tokens"] < s["rows"]))[:, None]
    s["x"][:, 0] = torch.where(valid, s["scale"] * s["table"][s["tokens"].clamp(0, s["rows"] - 1)], 0.0)
    return s["x"][:, 0]


def _plain_embed_backward(s):
    # one spare row takes what belongs to no token; the long sums of frequent rows in 64 bits
    row = torch.where((s["tokens"] >= 0) & (s["tokens"] < s["rows"]), s["tokens"], s["rows"])
    total = torch.zeros((s["rows"] + 1, s["width"]), dtype=torch.float64, device=row.device)
    total.index_add_(0, row, s["grad_x"][:, 0].double())
    return (s["scale"] * total[:-1]).float()


def _plain_norm_forward(s):
    x, n = s["x"][:, 0], s["n"]
    mean, rstd = _statistics(x, s["ptr"], s["groups"], torch.float32)
    sample = _row_sample(s["ptr"], n)
    h = ((x.reshape(n, s["groups"], -1) - mean[sample][:, :, None]) * rstd[sample][:, :, None]).reshape(n, -1)
    z = s["gamma"] * h + s["beta"]
    return z / (1 + torch.exp(-z)), mean, rstd


def _plain_norm_backward(s):
    x, gy, n, b, groups = s["x"][:, 0], s["grad_y"][:, 0], s["n"], s["samples"], s["groups"]
    sample = _row_sample(s["ptr"], n)
    mean, rstd = s["mean"][sample][:, :, None], s["rstd"][sample][:, :, None]
    h = (x.reshape(n, groups, -1) - mean) * rstd
    z = s["gamma"] * h.reshape(n, -1) + s["beta"]
    sig = 1 / (1 + torch.exp(-z))
    gz = gy * sig * (1 + z * (1 - sig))
    t = (s["gamma"] * gz).reshape(n, groups, -1)
    count = ((s["ptr"][1:] - s["ptr"][:-1]).double() * t.shape[2]).clamp(min=1)[:, None]
    m1 = (_per_sample(t.sum(2), sample, b) / count).float()[sample][:, :, None]
    m2 = (_per_sample((t * h).sum(2), sample, b) / count).float()[sample][:, :, None]
    gx = (rstd * (t - m1 - h * m2)).reshape(n, -1)
    # sums over every row: in 64 bits
    return gx, (gz * h.reshape(n, -1)).double().sum(0).float(), gz.double().sum(0).float()


def _plain_orthogonalise(s):
    x = s["update"]
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + NS_EPS)
    for _ in range(5):
        a = x @ x.transpose(1, 2)
        x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
    return x.transpose(1, 2).contiguous() if tall else x


_PLAIN = {"embed_forward": _plain_embed_forward, "embed_backward": _plain_embed_backward,
          "norm_forward": _plain_norm_forward, "norm_backward": _plain_norm_backward,
          "orthogonalise": _plain_orthogonalise}


def run(s):
    if not own:
        return _PLAIN[s["op"]](s)
    from equivariant_mlip_tensor_b200 import api
    op = s["op"]
    if op == "embed_forward":
        return api.embed_forward(s["tokens"], s["table"], scale=s["scale"], out=s["x"][:, 0])
    if op == "embed_backward":
        order = api.token_sort(s["tokens"], s["rows"])
        return api.embed_backward(order, s["grad_x"][:, 0], scale=s["scale"])
    if op == "norm_forward":
        return api.group_norm_forward(s["x"][:, 0], s["gamma"], s["beta"], s["groups"], graph_ptr=s["ptr"], eps=NORM_EPS,
                                      activation="silu", max_rows=s["max_rows"])
    if op == "norm_backward":
        return api.group_norm_backward(s["x"][:, 0], s["gamma"], s["beta"], s["groups"], s["mean"], s["rstd"],
                                       s["grad_y"][:, 0], graph_ptr=s["ptr"], activation="silu", max_rows=s["max_rows"])
    return api.orthogonalise(s["update"], steps=5)


def work(case):
    op = case["op"]
    if op == "embed_forward":
        values = case["n"] * case["width"]
        return {"bytes": 4 * (case["n"] + values + min(case["n"], case["rows"]) * case["width"]), "flops": values}
    if op == "embed_backward":
        values = case["n"] * case["width"]
        return {"bytes": 4 * (case["n"] + values + case["rows"] * case["width"]), "flops": values}
    if op.startswith("norm"):
        values, stats = case["n"] * case["channels"], case["samples"] * (2 * case["groups"] + 1)
        passes, terms = (2, 12) if op == "norm_forward" else (3, 25)
        return {"bytes": 4 * (passes * values + stats + 4 * case["channels"]), "flops": terms * values}
    k, long = sorted((case["m"], case["n"]))
    return {"bytes": 8 * case["batch"] * k * long, "flops": 5 * case["batch"] * (4 * k * k * long + 2 * k ** 3)}


def _segments(ptr):
    p = ptr.tolist()
    return list(zip(p[:-1], p[1:]))


def exact(case, seed):
    """The definitions in 64 bits, graph by graph and token by token."""
    s, op = prepare(case, seed), case["op"]
    if op == "embed_forward":
        padded = torch.cat([s["table"].double(), torch.zeros((1, case["width"]), dtype=torch.float64, device="cuda")])
        return s["scale"] * padded[torch.where(s["tokens"] < 0, case["rows"], s["tokens"]).long()]
    if op == "embed_backward":
        order = torch.argsort(s["tokens"], stable=True)
        g = s["grad_x"][:, 0].double()[order]
        total = torch.cat([torch.zeros((1, case["width"]), dtype=torch.float64, device="cuda"), g.cumsum(0)])
        cut = torch.searchsorted(s["tokens"][order], torch.arange(case["rows"] + 1, device="cuda", dtype=torch.int32))
        return s["scale"] * (total[cut[1:]] - total[cut[:-1]])
    if op.startswith("norm"):
        x, gamma, beta = s["x"][:, 0].double(), s["gamma"].double(), s["beta"].double()
        y, mean, rstd = torch.empty_like(x), [], []
        gx, ggamma, gbeta = torch.empty_like(x), torch.zeros_like(gamma), torch.zeros_like(beta)
        for lo, hi in _segments(s["ptr"]):
            v = x[lo:hi].reshape(hi - lo, case["groups"], case["channels"] // case["groups"])
            if hi == lo:
                mean.append(torch.zeros(case["groups"], dtype=torch.float64, device="cuda"))
                rstd.append(torch.full_like(mean[-1], 1 / math.sqrt(NORM_EPS)))
                continue
            mu = v.mean((0, 2))
            sd = torch.sqrt(((v - mu[:, None]) ** 2).mean((0, 2)) + NORM_EPS)
            mean.append(mu)
            rstd.append(1 / sd)
            h = (v - mu[:, None]) / sd[:, None]
            z = h.reshape(hi - lo, -1) * gamma + beta
            sig = torch.sigmoid(z)
            y[lo:hi] = z * sig
            if op == "norm_backward":
                gz = s["grad_y"][lo:hi, 0].double() * (sig + z * sig * (1 - sig))
                ggamma += (gz * h.reshape(hi - lo, -1)).sum(0)
                gbeta += gz.sum(0)
                t = (gz * gamma).reshape(v.shape)
                t = t - t.mean((0, 2))[:, None] - h * (t * h).mean((0, 2))[:, None]
                gx[lo:hi] = (t / sd[:, None]).reshape(hi - lo, -1)
        return (y, torch.stack(mean), torch.stack(rstd)) if op == "norm_forward" else (gx, ggamma, gbeta)
    u = s["update"].double()
    u = u / (torch.linalg.norm(u.flatten(1), dim=1)[:, None, None] + NS_EPS)
    left = case["m"] <= case["n"]
    for _ in range(5):
        gram = torch.einsum("bik,bjk->bij", u, u) if left else torch.einsum("bki,bkj->bij", u, u)
        poly = NS_B * gram + NS_C * gram.matmul(gram)
        u = NS_A * u + (poly.matmul(u) if left else u.matmul(poly))
    return u
