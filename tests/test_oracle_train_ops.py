"""Pins of the oracle's embedding, group norm and orthogonalisation, and the
host-side errors of their entry points (no GPU)."""
import ctypes

import numpy as np
import pytest

from oracle import embed, norm, ortho


def test_embedding_gradient_is_the_adjoint():
    rng = np.random.default_rng(0)
    tok = np.array([3, 0, 3, -1, 7, 2, 3, 5, 0])  # 7 and -1 are no rows of 6
    table, g = rng.standard_normal((6, 4)), rng.standard_normal((9, 4))
    lhs = np.sum(embed.forward(tok, table, 1.5) * g)
    assert np.isclose(lhs, np.sum(table * embed.backward(tok, 6, g, 1.5)), rtol=1e-13, atol=0)
    assert not embed.forward(tok, table, 1.5)[[3, 4]].any()
    order, srt = embed.sort(tok, 6)
    assert order.tolist() == [1, 8, 5, 0, 2, 6, 7, 3, 4] and srt.tolist() == [0, 0, 2, 3, 3, 3, 5, 6, 6]


@pytest.mark.parametrize("activation", [None, "silu"])
@pytest.mark.parametrize("ptr", [None, [0, 4, 4, 9], [1, 2, 8]])
def test_norm_gradient_against_differences(activation, ptr):
    rng = np.random.default_rng(1)
    n, c, groups, eps = 9, 6, 3, 1e-5
    x, gamma, beta = rng.standard_normal((n, c)), rng.standard_normal(c), rng.standard_normal(c)
    gy = rng.standard_normal((n, c))
    rows = slice(0, n) if ptr is None else slice(ptr[0], ptr[-1])

    def loss(x, gamma, beta):
        return np.sum((norm.forward(x, gamma, beta, groups, ptr, eps, activation)[0] * gy)[rows])

    got = norm.backward(x, gamma, beta, groups, ptr, eps, activation, gy)
    step = 1e-5
    for k, a in enumerate((x, gamma, beta)):
        num = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            hi, lo = [v.copy() for v in (x, gamma, beta)], [v.copy() for v in (x, gamma, beta)]
            hi[k][i] += step
            lo[k][i] -= step
            num[i] = (loss(*hi) - loss(*lo)) / (2 * step)
        want = np.nan_to_num(got[k])
        # central differences: truncation step^2 f'''/6 and cancellation 1e-16 |loss| / step
        assert np.allclose(num, want, rtol=0, atol=1e-6 * max(1.0, np.abs(want).max()))


def test_norm_normalises_each_graph_and_group():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((50, 8)) * 3 + 2
    y, mean, rstd = norm.forward(x, None, None, 2, [0, 20, 50], 1e-12, None)
    for lo, hi in ((0, 20), (20, 50)):
        for g in range(2):
            v = y[lo:hi, 4 * g:4 * g + 4]
            assert abs(v.mean()) < 1e-12 and abs(v.std() - 1) < 1e-9


@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (7, 3), (16, 16)])
def test_orthogonalisation_is_the_polynomial_of_the_singular_values(shape):
    g = np.random.default_rng(3).standard_normal(shape)
    assert np.allclose(ortho.orthogonalise(g), ortho.by_singular_values(g), atol=1e-10)
    s = np.linalg.svd(ortho.orthogonalise(g, 12), compute_uv=False)
    assert s.max() < 1.2026 and s.min() > 0.6  # the polynomial's attracting interval


def test_host_errors():
    """Refused before any device work."""
    from equivariant_mlip_tensor_b200 import lib
    L = lib()
    P, bad = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004)
    other = ctypes.c_void_p(0x2000)
    sz = ctypes.c_size_t()
    f = ctypes.c_float
    big = 1 << 40
    # sizes
    assert L.cgtp_token_sort_workspace_size(-1, 4, ctypes.byref(sz)) == 1
    assert L.cgtp_token_sort_workspace_size((1 << 30) + 1, 4, ctypes.byref(sz)) == 1
    assert L.cgtp_token_sort_workspace_size(4, -1, ctypes.byref(sz)) == 1
    assert L.cgtp_token_sort_workspace_size(4, 4, None) == 1
    assert L.cgtp_embed_backward_workspace_size(4, -1, ctypes.byref(sz)) == 1
    assert L.cgtp_group_norm_workspace_size(4, 1, 12, 5, 0, 0, ctypes.byref(sz)) == 1   # 12 channels, 5 groups
    assert L.cgtp_group_norm_workspace_size(4, 1, 12, 0, 0, 0, ctypes.byref(sz)) == 1
    assert L.cgtp_group_norm_workspace_size(4, 1, 0, 1, 0, 0, ctypes.byref(sz)) == 1
    assert L.cgtp_group_norm_workspace_size(4, 1, 12, 4, -1, 0, ctypes.byref(sz)) == 1
    assert L.cgtp_orthogonalise_workspace_size(1, 8193, 4, ctypes.byref(sz)) == 1
    assert L.cgtp_orthogonalise_workspace_size(65536, 4, 4, ctypes.byref(sz)) == 1
    # token sort: missing and aliased arrays, workspace
    assert L.cgtp_token_sort(4, 4, None, P, other, P, big, None) == 1
    assert L.cgtp_token_sort(4, 4, P, P, other, P, big, None) == 1
    assert L.cgtp_token_sort(4, 4, P, other, other, P, big, None) == 1
    third = ctypes.c_void_p(0x3000)
    assert L.cgtp_token_sort(10000, 4, P, other, third, None, 0, None) == 7
    assert L.cgtp_token_sort(10000, 4, P, other, third, P, 8, None) == 7
    assert L.cgtp_token_sort(10000, 4, P, other, third, bad, big, None) == 1      # misaligned workspace
    # embedding
    assert L.cgtp_embed_forward(4, 4, 8, P, None, f(1), P, 8, None) == 1
    assert L.cgtp_embed_forward(4, 4, 8, P, P, f(1), P, 7, None) == 1             # rows would overlap
    assert L.cgtp_embed_forward(-1, 4, 8, P, P, f(1), P, 8, None) == 1
    assert L.cgtp_embed_backward(4, 4, 8, P, P, P, 8, f(1), None, P, big, None) == 1
    assert L.cgtp_embed_backward(4, 4, 8, P, P, P, 7, f(1), P, P, big, None) == 1
    assert L.cgtp_embed_backward(4, 4, 8, P, P, P, 8, f(1), P, P, 8, None) == 7
    # group norm
    fwd, bwd = L.cgtp_group_norm_forward, L.cgtp_group_norm_backward
    assert fwd(4, 2, 8, 2, None, 0, P, 8, P, P, f(1e-5), 1, P, 8, P, P, P, big, None) == 1   # two samples, no offsets
    assert fwd(4, 1, 8, 3, None, 0, P, 8, P, P, f(1e-5), 1, P, 8, P, P, P, big, None) == 1
    assert fwd(4, 1, 8, 2, None, 0, P, 8, P, P, f(0), 1, P, 8, P, P, P, big, None) == 1      # eps
    assert fwd(4, 1, 8, 2, None, 0, P, 8, P, P, f(1e-5), 2, P, 8, P, P, P, big, None) == 1   # activation
    assert fwd(4, 1, 8, 2, None, 0, P, 16, P, P, f(1e-5), 1, P, 8, P, P, P, big, None) == 1  # in place, other stride
    assert fwd(4, 1, 8, 2, None, -1, P, 8, P, P, f(1e-5), 1, P, 8, P, P, P, big, None) == 1
    assert fwd(4, 1, 8, 2, None, 0, P, 8, P, P, f(1e-5), 1, P, 8, None, P, P, big, None) == 1
    assert fwd(1 << 20, 1, 8, 2, None, 0, P, 8, P, P, f(1e-5), 1, P, 8, P, P, P, 8, None) == 7
    assert bwd(4, 1, 8, 2, None, 0, P, 8, P, P, P, P, 1, None, 8, P, 8, P, P, P, big, None) == 1
    assert bwd(4, 1, 8, 2, None, 0, P, 8, P, P, P, P, 1, P, 8, P, 7, P, P, P, big, None) == 1
    assert bwd(4, 1, 8, 2, None, 0, P, 8, P, P, P, P, 1, P, 8, P, 8, P, P, None, 0, None) == 7
    # orthogonalisation
    ns = L.cgtp_orthogonalise
    assert ns(1, 4, 4, 0, f(1), P, P, P, big, None) == 1
    assert ns(1, 4, 4, 65, f(1), P, P, P, big, None) == 1
    assert ns(1, 4, 4, 5, f(1), None, P, P, big, None) == 1
    assert ns(1, 400, 400, 5, f(1), P, P, None, 0, None) == 7
    assert ns(0, 4, 4, 5, f(1), None, None, None, 0, None) == 0                   # nothing to do
