"""Orthogonalisation of a matrix by Newton-Schulz products (fp64).

Test infrastructure only (see ``oracle/__init__``).

X = G / (|G|_F + 1e-7); each step X <- a X + (b A + c A A) X with A = X X^T and
(a, b, c) = (3.4445, -4.7750, 2.0315).  On the singular values this is the odd
polynomial a s + b s^3 + c s^5, so the result also follows from a singular
value decomposition (``by_singular_values``), which pins the products.
"""
import numpy as np

A, B, C, EPS = 3.4445, -4.7750, 2.0315, 1e-7


def iterates(g, steps):
    """[X_0, ..., X_steps] of one matrix, on the side with fewer rows."""
    x = np.asarray(g, dtype=np.float64)
    if x.shape[0] > x.shape[1]:
        x = x.T
    xs = [x / (np.linalg.norm(x) + EPS)]
    for _ in range(steps):
        gram = xs[-1] @ xs[-1].T
        xs.append(A * xs[-1] + (B * gram + C * gram @ gram) @ xs[-1])
    return xs


def orthogonalise(g, steps=5, scale=1.0):
    g = np.asarray(g, dtype=np.float64)
    x = scale * iterates(g, steps)[-1]
    return x.T if g.shape[0] > g.shape[1] else x


def by_singular_values(g, steps=5):
    u, s, vt = np.linalg.svd(np.asarray(g, dtype=np.float64), full_matrices=False)
    s = s / (np.linalg.norm(s) + EPS)
    for _ in range(steps):
        s = A * s + B * s ** 3 + C * s ** 5
    return (u * s) @ vt
