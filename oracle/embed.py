"""Token embedding and its table gradient by token (fp64).

Test infrastructure only (see ``oracle/__init__``).

* out[k] = scale * table[tokens[k]], a zero row for a token outside the table;
* grad_table[v] = scale * sum over {k: tokens[k] = v} of grad_out[k].
"""
import numpy as np


def sort(tokens, n_rows):
    """(order, sorted): the stable sort, tokens outside [0, n_rows) last as n_rows."""
    t = np.asarray(tokens, dtype=np.int64)
    key = np.where((t >= 0) & (t < n_rows), t, n_rows)
    order = np.argsort(key, kind="stable")
    return order, key[order]


def forward(tokens, table, scale):
    table = np.asarray(table, dtype=np.float64)
    out = np.zeros((len(tokens), table.shape[1]))
    for k, t in enumerate(tokens):
        if 0 <= t < table.shape[0]:
            out[k] = scale * table[t]
    return out


def backward(tokens, n_rows, grad_out, scale):
    grad = np.zeros((n_rows, grad_out.shape[1]))
    for t, g in zip(tokens, np.asarray(grad_out, dtype=np.float64)):
        if 0 <= t < n_rows:
            grad[t] += scale * g
    return grad
