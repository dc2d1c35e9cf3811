"""Tokens' rows sorted by expert, and back with weights, pair by pair from their definitions (numpy, 64 bits)."""
import numpy as np


def route(ids, experts, first, align, max_rows):
    """(position, offsets, counts)."""
    lists = [[] for _ in range(experts)]
    for pair, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e - first < experts and e >= 0:
            lists[e - first].append(pair)
    position = np.full(ids.size, -1, dtype=np.int64)
    offsets, counts, at = [], [], 0
    for pairs in lists:
        kept = max(0, min(len(pairs), max_rows - at))
        position[pairs[:kept]] = at + np.arange(kept)
        offsets.append(min(at, max_rows))
        counts.append(kept)
        at += -(-len(pairs) // align) * align
    return position.reshape(ids.shape), np.array(offsets + [min(at, max_rows)]), np.array(counts)


def filled(offsets, counts):
    """The rows that fill experts up."""
    return [r for e, n in enumerate(counts.tolist()) for r in range(offsets[e] + n, offsets[e + 1])]


def dispatch(x, position, offsets, counts, rows):
    """rows (any type, as they were) with x's in them."""
    rows = rows.copy()
    rows[filled(offsets, counts)] = 0
    for t, j in zip(*np.nonzero(position >= 0)):
        rows[position[t, j]] = x[t]
    return rows


def combine(rows, position, weights):
    """(out, the sum of its terms' magnitudes)."""
    out = np.zeros((len(position), rows.shape[1]))
    size = np.zeros_like(out)
    for t, j in zip(*np.nonzero(position >= 0)):
        term = rows[position[t, j]].astype(np.float64) * (1.0 if weights is None else float(weights[t, j]))
        out[t] += term
        size[t] += np.abs(term)
    return out, size


def combine_backward(dout, rows, position, weights, offsets, counts, drows):
    """(drows, dweights, the sums of the magnitudes of dweights' terms)."""
    drows = drows.astype(np.float64).copy()
    drows[filled(offsets, counts)] = 0
    dweights, size = np.zeros(position.shape), np.zeros(position.shape)
    for t, j in zip(*np.nonzero(position >= 0)):
        r = position[t, j]
        drows[r] = dout[t].astype(np.float64) * float(weights[t, j])
        terms = dout[t].astype(np.float64) * rows[r].astype(np.float64)
        dweights[t, j], size[t, j] = terms.sum(), np.abs(terms).sum()
    return drows, dweights, size
