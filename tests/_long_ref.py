"""Plain 64-bit forms of the long-context calls, written from their definitions."""
import numpy as np


def visible(lengths, cu, mask, n, i):
    """Positions that node i of sequence n sees (mask as the tree calls take it)."""
    w = cu[n + 1] - cu[n]
    m = mask[cu[n] + i] if mask is not None else (2 << i) - 1
    return list(range(lengths[n])) + [lengths[n] + j for j in range(w) if (m >> j) & 1]


def key(pool, table, n, t):
    page = pool.shape[1]
    return pool[table[n][t // page], t % page]


def lse(q, pool, table, lengths, cu, mask, scale):
    """(lse [nodes, H], size [nodes, H]: the largest scale * sum|q c| of a row); float64."""
    q, pool = q.double().numpy(), pool.double().numpy()
    out, size = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    for n in range(len(cu) - 1):
        for i in range(cu[n + 1] - cu[n]):
            seen = visible(lengths, cu, mask, n, i)
            if not seen:
                continue
            keys = np.stack([key(pool, table, n, t) for t in seen])
            s = q[cu[n] + i] @ keys.T * scale
            top = s.max(-1, keepdims=True)
            out[cu[n] + i] = top[:, 0] + np.log(np.exp(s - top).sum(-1))
            size[cu[n] + i] = (np.abs(q[cu[n] + i]) @ np.abs(keys).T).max(-1) * scale
    return out, size


def weights(q, pool, table, lengths, cu, mask, node_weight, lse, scale, width):
    """(sum [n_seqs, width], and the bound of its error): what each position gets."""
    q, pool = q.double().numpy(), pool.double().numpy()
    out = np.zeros((len(cu) - 1, width))
    tol = np.zeros_like(out)
    for n in range(len(cu) - 1):
        w = cu[n + 1] - cu[n]
        rows = w * q.shape[1]
        for i in range(w):
            u = 1.0 if node_weight is None else node_weight[cu[n] + i]
            seen = visible(lengths, cu, mask, n, i)
            if u == 0 or not seen:
                continue
            keys = np.stack([key(pool, table, n, t) for t in seen])
            row = q[cu[n] + i]
            s = row @ keys.T * scale
            size = np.abs(row) @ np.abs(keys).T * scale
            p = u * np.exp(s - lse[cu[n] + i][:, None])
            # the score: an fp32 sum of 576 products, eight more roundings; the exponent in units of
            # log 2: two roundings of the score's and the lse's size; the power and its product; the sum
            e = 584 * 2.0**-24 * size + 2.0**-22 * (np.abs(s) + np.abs(lse[cu[n] + i])[:, None]) + (rows + 16) * 2.0**-24
            out[n, seen] += p.sum(0)
            tol[n, seen] += 1.02 * (np.abs(p) * e).sum(0)
    return out, tol


def choose(values, count, first, recent, most):
    """Taken indices, ascending: NaN below everything, the lower index first among equals."""
    if count <= most:
        return list(range(count))
    rank = lambda j: (0 if values[j] == values[j] else 1, -values[j] if values[j] == values[j] else 0, j)  # noqa: E731
    middle = sorted(range(first, count - recent), key=rank)[:most - first - recent]
    return list(range(first)) + sorted(middle) + list(range(count - recent, count))


def block_scores(q, keys, table, lengths, cu, page, scale):
    """(per sequence: scores of its full blocks, bound of their error)."""
    q, keys = q.double().numpy(), keys.double().numpy()
    out = []
    for n in range(len(cu) - 1):
        full, rows = lengths[n] // page, q[cu[n]:cu[n + 1]].reshape(-1, 576)
        if full == 0 or len(rows) == 0:
            out.append((np.zeros(0), np.zeros(0)))
            continue
        k = keys[table[n][:full]]
        s = rows @ k.T * scale
        size = (np.abs(rows) @ np.abs(k).T).max(-1, keepdims=True) * scale
        top = s.max(-1, keepdims=True)
        p = np.exp(s - top)
        p /= p.sum(-1, keepdims=True)
        # the score's error counts in the exponent and in the lse; the lse's own sum and logarithm
        e = 2 * 584 * 2.0**-24 * size + 2.0**-21 * (np.abs(top) + size + 1) + (full + len(rows) + 32) * 2.0**-24
        out.append((p.sum(0), 1.02 * (p * e).sum(0)))
    return out
