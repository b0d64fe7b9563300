"""Group norm with an activation, one normalisation per graph (fp64).

Test infrastructure only (see ``oracle/__init__``).

Over the rows of a graph and the channels of a group: h = (x - mean) /
sqrt(var + eps) with the biased variance, y = act(gamma h + beta).  The
backward is the chain rule written out: gz = grad_y act'(z), t = gamma gz,
grad_x = (t - mean(t) - h mean(t h)) / sqrt(var + eps).
"""
import numpy as np


def _act(z, activation):
    if activation is None:
        return z, np.ones_like(z)
    s = 1.0 / (1.0 + np.exp(-z))
    return z * s, s * (1.0 + z * (1.0 - s))


def _graphs(ptr, n):
    return [(0, n)] if ptr is None else list(zip(ptr[:-1], ptr[1:]))


def forward(x, gamma, beta, groups, ptr, eps, activation):
    """(y, mean, rstd); rows of y outside every graph are NaN."""
    x = np.asarray(x, dtype=np.float64)
    n, c = x.shape
    gamma = np.ones(c) if gamma is None else np.asarray(gamma, dtype=np.float64)
    beta = np.zeros(c) if beta is None else np.asarray(beta, dtype=np.float64)
    y = np.full((n, c), np.nan)
    graphs = _graphs(ptr, n)
    mean, rstd = np.zeros((len(graphs), groups)), np.full((len(graphs), groups), 1.0 / np.sqrt(eps))
    for s, (lo, hi) in enumerate(graphs):
        if hi == lo:
            continue
        v = x[lo:hi].reshape(hi - lo, groups, c // groups)
        mean[s] = v.mean(axis=(0, 2))
        rstd[s] = 1.0 / np.sqrt(v.var(axis=(0, 2)) + eps)
        h = ((v - mean[s][:, None]) * rstd[s][:, None]).reshape(hi - lo, c)
        y[lo:hi] = _act(gamma * h + beta, activation)[0]
    return y, mean, rstd


def backward(x, gamma, beta, groups, ptr, eps, activation, grad_y):
    """(grad_x, grad_gamma, grad_beta); rows of grad_x outside every graph are NaN."""
    x, grad_y = np.asarray(x, dtype=np.float64), np.asarray(grad_y, dtype=np.float64)
    n, c = x.shape
    gamma = np.ones(c) if gamma is None else np.asarray(gamma, dtype=np.float64)
    beta = np.zeros(c) if beta is None else np.asarray(beta, dtype=np.float64)
    _, mean, rstd = forward(x, gamma, beta, groups, ptr, eps, activation)
    gx, gg, gb = np.full((n, c), np.nan), np.zeros(c), np.zeros(c)
    for s, (lo, hi) in enumerate(_graphs(ptr, n)):
        if hi == lo:
            continue
        shape = (hi - lo, groups, c // groups)
        h = (x[lo:hi].reshape(shape) - mean[s][:, None]) * rstd[s][:, None]
        hf = h.reshape(hi - lo, c)
        gz = grad_y[lo:hi] * _act(gamma * hf + beta, activation)[1]
        gg += (gz * hf).sum(axis=0)
        gb += gz.sum(axis=0)
        t = (gamma * gz).reshape(shape)
        m1, m2 = t.mean(axis=(0, 2)), (t * h).mean(axis=(0, 2))
        gx[lo:hi] = ((t - m1[:, None] - h * m2[:, None]) * rstd[s][:, None]).reshape(hi - lo, c)
    return gx, gg, gb
