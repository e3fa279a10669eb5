"""Plain 64-bit forms of the tree-verification calls, written from their definitions: loops over
sequences, nodes and positions, no packing tricks and nothing shared with the library."""
import math

import numpy as np
import torch

LATENT, KEY = 512, 576


def path_to(parent, i):
    """Nodes from the root to i (parents of one sequence)."""
    p = []
    while i >= 0:
        p.append(i)
        i = parent[i]
    return p[::-1]


def masks(parents):
    """One sequence's visibility words (Python ints, two's complement 64-bit)."""
    out = []
    for i in range(len(parents)):
        m = sum(1 << j for j in path_to(parents, i))
        out.append(m - (1 << 64) if m >> 63 else m)
    return out


def random_parents(rng, w, root_share=0.1):
    return [-1 if i == 0 or rng.random() < root_share else int(rng.integers(max(0, i - 5), i))
            for i in range(w)]


def tree_attention(q, pool, table, lengths, cu, mask, scale):
    """(z [nodes, H, 512], unit, size): float64 numpy; unit is sum_t p_t |c_t|, what a relative
    error of the weights is multiplied by, and size [nodes, H, 1] the largest scale * sum|q c|."""
    q, pool = q.double().numpy(), pool.double().numpy()
    page = pool.shape[1]
    z = np.zeros(q.shape[:2] + (LATENT,))
    unit, size = np.zeros_like(z), np.zeros(q.shape[:2] + (1,))
    for n in range(len(cu) - 1):
        w = cu[n + 1] - cu[n]
        for i in range(w):
            m = mask[cu[n] + i] if mask is not None else (2 << i) - 1
            seen = list(range(lengths[n])) + [lengths[n] + j for j in range(w) if (m >> j) & 1]
            if not seen:
                continue
            keys = np.stack([pool[table[n][t // page], t % page] for t in seen])
            s = q[cu[n] + i] @ keys.T * scale
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            z[cu[n] + i] = p @ keys[:, :LATENT]
            unit[cu[n] + i] = p @ np.abs(keys[:, :LATENT])
            size[cu[n] + i, :, 0] = (np.abs(q[cu[n] + i]) @ np.abs(keys).T).max(-1) * scale
    return z, unit, size


def _silu(x):
    return x / (1 + np.exp(-x))


def _streams(x, w, tail, path, H, d, l2_eps, l2norm):
    """q, k, v [H, d] of the last node of a path."""
    taps = np.concatenate([tail, x[path]])[-4:]
    y = _silu((taps * w.T).sum(0)).reshape(3, H, d)
    q, k, v = y
    if l2norm:
        q, k = (t / np.sqrt((t ** 2).sum(-1, keepdims=True) + l2_eps) for t in (q, k))
    return q, k, v


def kda_tree(x, conv_w, conv_state, g, beta, state, slots, cu, parent, *, H, d, scale=1.0,
             l2_eps=1e-6, norm_eps=1e-6, g_min=-5.0, l2norm=True, gate=None, norm_w=None,
             accept=None):
    """Outputs of all nodes, and with `accept` the pool state and conv tails afterwards."""
    f = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    x, conv_w, conv_state, g, beta, state, gate, norm_w = map(
        f, (x, conv_w, conv_state, g, beta, state, gate, norm_w))
    out = np.zeros((x.shape[0], H, d))
    new_state, new_tail = state.copy(), conv_state.copy()
    for n in range(len(cu) - 1):
        lo, hi = cu[n], cu[n + 1]
        par, S = parent[lo:hi], []
        for i in range(hi - lo):
            path = path_to(par, i)
            q, k, v = _streams(x[lo:hi], conv_w, conv_state[slots[n]], path, H, d, l2_eps, l2norm)
            before = S[par[i]] if par[i] >= 0 else state[slots[n]]
            m = np.exp(np.maximum(g[lo + i], g_min))[:, :, None] * before
            u = beta[lo + i][:, None] * (v - np.einsum("hc,hcd->hd", k, m))
            m = m + k[:, :, None] * u[:, None, :]
            S.append(m)
            o = scale * np.einsum("hc,hcd->hd", q, m)
            if gate is not None:
                o = o / np.sqrt((o ** 2).mean(-1, keepdims=True) + norm_eps)
                o = o * (1 if norm_w is None else norm_w) / (1 + np.exp(-gate[lo + i]))
            out[lo + i] = o
        if accept is not None and accept[n] >= 0:
            new_state[slots[n]] = S[accept[n]]
            rows = np.concatenate([conv_state[slots[n]], x[lo:hi][path_to(par, accept[n])]])
            new_tail[slots[n]] = rows[-3:]
    return out, new_state, new_tail


class Pages:
    """The page bookkeeping as lists."""

    def __init__(self, n_pages, n_slots, max_pages, page_size):
        self.refs = [0] * n_pages
        self.table = [[-1] * max_pages for _ in range(n_slots)]
        self.held, self.lengths, self.page = [0] * n_slots, [0] * n_slots, page_size

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def free(self, slots):
        for s in slots:
            for j in range(self.held[s]):
                self.refs[self.table[s][j]] -= 1
                self.table[s][j] = -1
            if self.held[s]:
                self.lengths[s] = 0
            self.held[s] = 0

    def fork(self, src, dst, copies):
        """copies(old page, new page, rows) is told of every copy."""
        free, out_of = iter(self._free()), False
        children = [d for i, d in enumerate(dst) if self.held[d] == 0 and d not in dst[:i]]
        done, bad = [], False
        for i, (s, d) in enumerate(zip(src, dst)):
            if self.held[d] or d in dst[:i] or s in children:
                bad = True
                continue
            done.append((s, d))
        for s, d in done:
            n = self.lengths[s]
            full, part = divmod(n, self.page)
            new = next(free, None) if part else None
            if part and new is None:
                out_of = True
                continue
            for j in range(full):
                self.table[d][j] = self.table[s][j]
                self.refs[self.table[s][j]] += 1
            if part:
                self.table[d][full] = new
                self.refs[new] = 1
                copies(self.table[s][full], new, part)
            self.held[d], self.lengths[d] = full + (part > 0), n
        return bad, out_of

    def reserve(self, slots, extra):
        free, out_of = self._free(), False
        for s, e in zip(slots, extra):
            need = max(0, math.ceil((self.lengths[s] + e) / self.page) - self.held[s])
            if need and (out_of or need > len(free)):
                out_of = True
                continue
            for j in range(need):
                p = free.pop(0)
                self.refs[p] = 1
                self.table[s][self.held[s] + j] = p
            self.held[s] += need
        return out_of


def i32(x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)
