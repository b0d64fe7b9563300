"""The accuracy that the orthogonalisation claims, and that its test would see a lost part of it.

Bound: the error that fp64 iterates get when every entry of every product is moved
by delta(K) times the root mean square of the product's entries, and every entry of
X by 2^-22 of itself, with random signs.  delta(K) is what a product of fp16 pairs over K
terms may be off by:

  operands      each within 2^-23 of itself (pairs of 11 bits), low low (2^-22) left out: 2^-21
  sums          an accumulator adds 16 terms at a time and rounds towards zero, by less than 2^-23 and in
                the mean by 2^-24 of its running sum, which is at most its last one in the mean square:
                2^-24 min(K / 16, 48), for contractions beyond 768 are spread over several accumulators

and 2^-22 covers X as a pair and the three fp32 operations that make its next value.  (fp32
sums of the smallest matrices stay below that: half a step, 2^-24, at random for each of
at most 64 terms in a row.)  The errors pass through the further steps as they do in the
kernels.  Twice the size of that error is allowed, since roundings towards zero have one sign.

The CPU tests check the bound from the other side: with one of the two cross
terms low high and high low left out, in every product or in a single one of the
three, or with no low part, the same arithmetic in fp64 is beyond it.
"""
import numpy as np
import pytest

from oracle import ortho as oortho
from tests.gpu_common import cuda, host

A, B, C, EPS = oortho.A, oortho.B, oortho.C, oortho.EPS


def _start(g):
    x = np.asarray(g, dtype=np.float64)
    if x.shape[0] > x.shape[1]:
        x = x.T
    return x / (np.linalg.norm(x) + EPS)


def _rel(x, want):
    return np.linalg.norm(x - want) / np.linalg.norm(want)


def _allowed(g, steps):
    """fp64 result on the side with fewer rows, and the relative error allowed."""
    rng = np.random.default_rng(0)

    def signs(x):
        return rng.choice([-1.0, 1.0], x.shape)

    def product(a, b):
        p = a @ b
        delta = 2.0 ** -21 + 2.0 ** -24 * min(a.shape[1] / 16, 48)
        return p + delta * np.sqrt(np.mean(p * p)) * signs(p)

    x = _start(g)
    x = x + 2.0 ** -22 * x * signs(x)
    for _ in range(steps):
        gram = product(x, x.T)
        x = A * x + product(B * gram + C * product(gram, gram), x)
        x = x + 2.0 ** -22 * x * signs(x)
    want = oortho.iterates(g, steps)[-1]
    return want, 2 * _rel(x, want)


def _pair_steps(g, steps, kept):
    """The steps with products of fp16 pairs and diagonals outside them, all sums in
    fp64; kept: (low high, high low) of X X^T, A A and P X, 1 or 0."""
    def split(x):
        x = x * 2.0 ** 14
        high = x.astype(np.float16).astype(np.float64)
        return high * 2.0 ** -14, (x - high).astype(np.float16).astype(np.float64) * 2.0 ** -14

    def product(a, b, keep):
        (ah, al), (bh, bl) = split(a), split(b)
        return ah @ bh + keep[0] * (al @ bh) + keep[1] * (ah @ bl)

    x = _start(g)
    for _ in range(steps):
        r = product(x, x.T, kept[0])
        np.fill_diagonal(r, 0)
        d = (x * x).sum(1)
        square = product(r, r, kept[1]) + (d[:, None] + d[None, :]) * r + np.diag(d * d)
        p = B * (r + np.diag(d)) + C * square
        dp = np.diag(p).copy()
        np.fill_diagonal(p, 0)
        x = (A + dp)[:, None] * x + 2 * product(p / 2, x, kept[2])  # entries of P up to 3.45: half of them fit
    return x


def _matrix(shape, kind):
    rng = np.random.default_rng(sum(shape))
    m, n = shape[-2:]
    if kind == "low rank":
        k = max(1, min(m, n) // 4)
        g = rng.standard_normal(shape[:-2] + (m, k)) @ rng.standard_normal(shape[:-2] + (k, n))
        g += 1e-2 * rng.standard_normal(shape)
    elif kind == "unequal rows":
        g = np.exp(rng.standard_normal(shape[:-1] + (1,))) * rng.standard_normal(shape)
    else:
        g = 1e-3 * rng.standard_normal(shape)
    return g.astype(np.float32)


@pytest.mark.parametrize("m,n", [(8, 8), (33, 65), (64, 64), (64, 1920), (128, 128), (96, 300), (300, 77), (40, 2100),
                                 (256, 512)])
def test_bound_sees_a_lost_part(m, n):
    both, none = (1, 1), (0, 0)
    for steps in (5, 11):
        g = _matrix((m, n), "random")
        want, allowed = _allowed(g, steps)
        assert _rel(_pair_steps(g, steps, [both] * 3), want) < 0.1 * allowed
        lost = [[(0, 1)] * 3, [(1, 0)] * 3, [none] * 3]
        if steps == 11:  # A A, the smallest of the three, counts for little before the values have settled
            lost += [[keep if k == j else both for k in range(3)] for j in range(3) for keep in ((0, 1), (1, 0))]
        for kept in lost:
            assert _rel(_pair_steps(g, steps, kept), want) > allowed, (steps, kept)


SHAPES = [(2, 4, 4), (2, 8, 8), (2, 4, 100), (2, 32, 16), (2, 33, 65), (3, 64, 64), (1, 64, 1920), (2, 128, 128),
          (2, 127, 129), (2, 128, 257), (1, 130, 260), (2, 96, 300), (1, 256, 512), (2, 300, 77), (1, 40, 2100),
          (1, 64, 2432), (1, 520, 530)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("steps", [1, 5, 11])
def test_error_of_every_matrix(shape, steps):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from equivariant_mlip_tensor_b200 import api
    for kind in ("random", "low rank", "unequal rows"):
        g = _matrix(shape, kind)
        got = host(api.orthogonalise(cuda(g), steps=steps))
        for z in range(shape[0]):
            want, allowed = _allowed(g[z], steps)
            off = _rel(got[z].T if shape[1] > shape[2] else got[z], want)
            assert off <= allowed, (kind, z, off, allowed)
