"""CPU oracle of expert routing: the plan, rows to the segments and back, and the gradients
(numpy; float64 values). Test infrastructure only: it shares no code with the GPU path."""
import numpy as np


def rows_for(tokens, top_k, experts):
    """A row count that any choice fits: each expert in use pads to 32."""
    n = tokens * top_k
    return (n + 31 * min(experts, n)) // 32 * 32


def route(ids, experts, rows):
    """(offsets, row_of, entry_of) as mxfp8_route writes them for valid ids."""
    flat = np.asarray(ids).reshape(-1)
    row_of = np.full(flat.size, -1, np.int64)
    entry_of = np.full(rows, -1, np.int64)
    offsets, at = np.zeros(experts + 1, np.int64), 0
    segments = []
    for e in range(experts):
        mine = np.flatnonzero(flat == e)
        offsets[e] = at
        segments.append((at, mine))
        at += -(-len(mine) // 32) * 32
    offsets[experts] = rows
    if at > rows:                       # a plan of no entries
        offsets[:experts] = 0
        segments = []
    for start, mine in segments:
        row_of[mine] = start + np.arange(len(mine))
        entry_of[start:start + len(mine)] = mine
    return offsets, row_of.reshape(np.shape(ids)), entry_of


def dispatch(x, row_of, rows, weights=None):
    out = np.zeros((rows, x.shape[1]))
    for t, j in np.argwhere(row_of >= 0):
        out[row_of[t, j]] = x[t] * (1.0 if weights is None else float(weights[t, j]))
    return out


def combine(y, row_of, weights=None):
    """The sums, and the sums of the terms' magnitudes."""
    out = np.zeros((row_of.shape[0], y.shape[1]))
    mag = np.zeros_like(out)
    for t, j in np.argwhere(row_of >= 0):
        term = y[row_of[t, j]] * (1.0 if weights is None else float(weights[t, j]))
        out[t] += term
        mag[t] += np.abs(term)
    return out, mag


def combine_weights_grad(grad_out, y, row_of):
    """The weights' gradient, and the sums of the terms' magnitudes."""
    dw, mag = np.zeros(row_of.shape), np.zeros(row_of.shape)
    for t, j in np.argwhere(row_of >= 0):
        term = grad_out[t] * y[row_of[t, j]]
        dw[t, j], mag[t, j] = term.sum(), np.abs(term).sum()
    return dw, mag
