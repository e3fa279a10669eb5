"""The speculative-verification operators as a serving step uses them: what is timed, on which inputs.

Four operators, each with its plain form in elementary torch operations and, where `own` is set, the
library's call:

  tree     latent attention of a tree of drafted tokens (or of one token) over a paged cache
  pages    freeing, forking and reserving a sequence's pages (copy of the partly filled page)
  cache    writing drafted rows into the paged cache, then compacting the accepted path
  verify   the KDA layer's outputs for every node of a drafted tree, the pool state read once
  accept   the accepted path replayed into the KDA pool state and convolution tail

A case's "shape" number fixes its ragged sizes, trees and accepted nodes, so that the work of a case
does not depend on the seed; the seed fixes every value and the placement of the pages.
"""
import math
import random

import torch

own = False

DEV = "cuda"
LATENT, KEY = 512, 576
HD = 128                      # KDA head width
SCALE = 192 ** -0.5


def listed():
    return [
        # one user on one of four tensor-parallel ranks: 16 heads, a draft of four, a short prompt
        dict(name="tree_1x4_h16", op="tree", n=1, nodes=4, heads=16, length=700, page=16, shape=1),
        # ordinary decode of a full batch, one token a sequence, ragged lengths up to 4096
        dict(name="decode_256x1", op="tree", n=256, nodes=1, heads=64, length=4096, page=64, shape=2),
        # a batch verifying trees of eight drafted tokens
        dict(name="tree_64x8", op="tree", n=64, nodes=8, heads=64, length=4096, page=64, shape=3),
        # long contexts with wide trees: the cache is far larger than L2
        dict(name="tree_4x16_long", op="tree", n=4, nodes=16, heads=64, length=65536, page=64, shape=4),
        # one prompt forked for four samples
        dict(name="fork_1to4", op="pages", n=1, children=4, layers=9, length=300, page=64, shape=5),
        # a batch of prompts forked for parallel sampling over all latent layers
        dict(name="fork_64to256", op="pages", n=64, children=4, layers=9, length=1000, page=64, shape=6),
        # four users' drafted rows written and compacted, all latent layers
        dict(name="rows_4x4", op="cache", n=4, nodes=4, layers=9, length=500, page=16, shape=7),
        # a full batch's drafted rows
        dict(name="rows_256x8", op="cache", n=256, nodes=8, layers=9, length=500, page=64, shape=8),
        # one user's tree through a KDA layer
        dict(name="verify_1x12", op="verify", n=1, nodes=12, heads=64, shape=9),
        # a full batch of trees through a KDA layer
        dict(name="verify_256x8", op="verify", n=256, nodes=8, heads=64, shape=10),
        # the accepted paths of a few users, and of a full batch
        dict(name="accept_3x6", op="accept", n=3, nodes=6, heads=64, shape=11),
        dict(name="accept_256x8", op="accept", n=256, nodes=8, heads=64, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "pages", "cache", "verify", "accept"])
    shape = rng.randrange(1, 1 << 30)
    if op == "tree":
        heads, page = rng.choice([16, 32, 64]), rng.choice([16, 32, 64, 128])
        n, nodes = _log(rng, 1, 256), _log(rng, 1, 33)
        most = min(65536, (1 << 28) // (n * nodes * heads), (1 << 20) // n)
        return dict(op=op, n=n, nodes=nodes, heads=heads, length=_log(rng, 1, max(2, most)), page=page, shape=shape)
    if op == "pages":
        return dict(op=op, n=_log(rng, 1, 64), children=rng.randint(1, 4), layers=rng.choice([1, 9]), length=_log(rng, 1, 1000),
                    page=rng.choice([16, 32, 64, 128]), shape=shape)
    if op == "cache":
        return dict(op=op, n=_log(rng, 1, 256), nodes=rng.randint(1, 8), layers=rng.choice([1, 9]), length=_log(rng, 1, 500),
                    page=rng.choice([16, 32, 64]), shape=shape)
    n = _log(rng, 1, 256)
    return dict(op=op, n=n, nodes=_log(rng, 1, max(1, min(32, 2048 // n))), heads=rng.choice([16, 32, 64]), shape=shape)


# ---- the sizes that a case's shape number stands for ----------------------------------------

def _sizes(case):
    """(lengths, nodes of each sequence, parents of every node, accepted node of each sequence)"""
    r = random.Random(case["shape"])
    n = case["n"]
    lengths = [case["length"] - r.randrange(case["length"] // 2 + 1) for _ in range(n)] if "length" in case else [0] * n
    most = case.get("nodes", 0)
    counts = [most - r.randrange(most // 3 + 1) if most > 1 else most for _ in range(n)]
    counts[r.randrange(n)] = most
    parents, accepted = [], []
    for w in counts:
        # a node hangs under one of the four before it; the first is the root
        parents += [r.randrange(max(0, i - 4), i) if i else -1 for i in range(w)]
        accepted.append(r.randrange(w) if w else -1)
    return lengths, counts, parents, accepted


def _depths(counts, parents):
    """Nodes on the path of each node, itself included."""
    out, at = [], 0
    for w in counts:
        d = []
        for i in range(w):
            p = parents[at + i]
            d.append(1 + (d[p] if p >= 0 else 0))
        out.append(d)
        at += w
    return out


def work(case):
    lengths, counts, parents, accepted = _sizes(case)
    n, total = case["n"], sum(counts)
    depths = _depths(counts, parents)
    if case["op"] == "tree":
        h = case["heads"]
        keys = sum((x + w) for x, w in zip(lengths, counts))
        pairs = sum(h * (w * x + sum(d)) for x, w, d in zip(lengths, counts, depths))
        return {"bytes": keys * KEY * 2 + total * h * (KEY + LATENT) * 2 + total * 8, "flops": 2.0 * pairs * (KEY + LATENT)}
    if case["op"] == "pages":
        rows = sum((x % case["page"]) * case["children"] for x in lengths) * case["layers"]
        pages = sum(-(-x // case["page"]) for x in lengths) * case["children"]
        return {"bytes": rows * KEY * 2 * 2 + pages * 4 * 4, "flops": 0}
    if case["op"] == "cache":
        moved = sum(d[a] for d, a in zip(depths, accepted) if a >= 0)
        return {"bytes": (total + moved) * case["layers"] * KEY * 2 * 2, "flops": 0}
    h = case["heads"]
    state = n * h * HD * HD * 4
    if case["op"] == "verify":
        row = h * HD * (3 * 2 + 4 + 2 + 2) + h * 4
        return {"bytes": state + total * row + n * 3 * 3 * h * HD * 2 + 3 * h * HD * 4 * 2,
                "flops": 2.0 * 2 * total * h * HD * HD + 4.0 * h * HD * 2 * sum(sum(d) for d in depths)}
    steps = sum(d[a] for d, a in zip(depths, accepted))
    row = h * HD * (2 * 2 + 4) + h * 4       # k and v streams, retention, strength
    return {"bytes": 2 * state + steps * row + 2 * n * 3 * 3 * h * HD * 2, "flops": 6.0 * steps * h * HD * HD}


# ---- inputs ----------------------------------------------------------------------------------

class _Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(int(seed))

    def normal(self, *shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, generator=self.g, device=DEV, dtype=torch.float32).mul_(std).to(dtype)

    def uniform(self, *shape, low=0.0, high=1.0):
        return torch.rand(shape, generator=self.g, device=DEV, dtype=torch.float32).mul_(high - low).add_(low)

    def order(self, n):
        return torch.randperm(n, generator=self.g, device=DEV).to(torch.int32)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _table(d, needs, most, n_pages):
    """Page table rows with the given numbers of pages, placed at random, and the pages left over."""
    order = d.order(n_pages)
    need = _i32(needs)
    at = torch.cumsum(need, 0) - need
    j = torch.arange(most, device=DEV, dtype=torch.int32)
    used = j[None, :] < need[:, None]
    idx = (at[:, None] + j[None, :]).clamp_(max=n_pages - 1)
    return torch.where(used, order[idx.long()], torch.full_like(idx, -1)).to(torch.int32).contiguous()


def prepare(case, seed):
    d = _Draw(seed)
    lengths, counts, parents, accepted = _sizes(case)
    n, total = case["n"], sum(counts)
    s = {"case": case, "op": case["op"], "lengths": _i32(lengths), "most": max(counts) if counts else 0}
    cu = [0]
    for w in counts:
        cu.append(cu[-1] + w)
    s["cu"] = _i32(cu)
    s["parent"] = _i32(parents) if parents else torch.zeros(0, dtype=torch.int32, device=DEV)
    if case["op"] == "tree":
        h, page = case["heads"], case["page"]
        needs = [-(-(x + w) // page) for x, w in zip(lengths, counts)]
        n_pages = sum(needs) + 3
        s["pool"] = d.normal(n_pages, page, KEY)
        s["table"] = _table(d, needs, max(needs), n_pages)
        s["q"] = d.normal(total, h, KEY)
        s["mask"] = torch.tensor(_bits(counts, parents), dtype=torch.int64, device=DEV)
        s["z"] = torch.empty(total, h, LATENT, dtype=torch.bfloat16, device=DEV)
        if own:
            from hybrid_linear_attention_gb300 import kda
            s["ws"] = torch.empty(kda.mla_tree_workspace_size(n, total, h), dtype=torch.uint8, device=DEV)
    elif case["op"] == "pages":
        page, kids, layers = case["page"], case["children"], case["layers"]
        needs = [-(-x // page) for x in lengths]
        grown = [-(-(x + 8) // page) for x in lengths]
        n_pages = sum(needs) + kids * sum(g - x // page for g, x in zip(grown, lengths)) + 5
        most = max(grown)
        table = _table(d, needs, most, n_pages)
        s["refs"] = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        s["refs"][table[table >= 0].long()] = 1
        s["table"] = torch.cat([table, torch.full((n * kids, most), -1, dtype=torch.int32, device=DEV)]).contiguous()
        s["held"] = torch.cat([_i32(needs), torch.zeros(n * kids, dtype=torch.int32, device=DEV)])
        s["lengths"] = torch.cat([s["lengths"], torch.zeros(n * kids, dtype=torch.int32, device=DEV)])
        s["src"] = torch.arange(n, device=DEV, dtype=torch.int32).repeat_interleave(kids)
        s["dst"] = torch.arange(n, n + n * kids, device=DEV, dtype=torch.int32)
        s["extra"] = torch.full((n * kids,), 8, dtype=torch.int32, device=DEV)  # room for the next draft
        s["pool"] = d.normal(layers, n_pages, page, KEY)
        if own:
            from hybrid_linear_attention_gb300 import kda
            s["ws"] = torch.empty(kda.mla_pages_workspace_size(n * kids), dtype=torch.uint8, device=DEV)
    elif case["op"] == "cache":
        page, layers = case["page"], case["layers"]
        needs = [-(-(x + w) // page) for x, w in zip(lengths, counts)]
        n_pages = sum(needs) + 3
        s["pool"] = d.normal(layers, n_pages, page, KEY)
        s["table"] = _table(d, needs, max(needs), n_pages)
        s["rows"] = d.normal(layers, total, KEY)
        s["accepted"] = _i32(accepted)
        s["new_lengths"] = torch.empty(n, dtype=torch.int32, device=DEV)
    else:
        h = case["heads"]
        c = 3 * h * HD
        s["x"] = d.normal(total, c)
        s["conv_w"] = d.normal(c, 4, std=0.5)
        s["conv_state"] = d.normal(n, 3, c)
        s["g"] = d.uniform(total, h, HD, low=-5.0, high=0.0)
        s["beta"] = torch.sigmoid(d.normal(total, h, dtype=torch.float32))
        s["state"] = d.normal(n, h, HD, HD, std=0.02, dtype=torch.float32)
        s["slots"] = d.order(n)
        if case["op"] == "verify":
            s["gate"] = d.normal(total, h, HD)
            s["norm_w"] = d.uniform(HD, low=0.5, high=1.5)
            s["out"] = torch.empty(total, h, HD, dtype=torch.bfloat16, device=DEV)
        else:
            s["accepted"] = _i32(accepted)
        if own:
            from hybrid_linear_attention_gb300 import kda
            s["p"] = kda.params(H=h)
    return s


def _bits(counts, parents):
    """Each node's ancestors and itself, as bits."""
    out, at = [], 0
    for w in counts:
        b = []
        for i in range(w):
            p = parents[at + i]
            b.append((b[p] if p >= 0 else 0) | (1 << i))
        out += [x - (1 << 64) if x >> 63 else x for x in b]
        at += w
    return out


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    if own:
        return _library(s)
    return {"tree": _plain_tree, "pages": _plain_pages, "cache": _plain_cache, "verify": _plain_verify, "accept": _plain_accept}[s["op"]](s)


def _library(s):
    from hybrid_linear_attention_gb300 import kda
    op = s["op"]
    if op == "tree":
        kda.mla_tree_latent(s["q"], s["pool"], s["table"], s["lengths"], s["cu"], s["z"], mask=s["mask"], scale=SCALE, workspace=s["ws"])
        return s["z"]
    if op == "pages":
        kda.mla_pages_free(s["refs"], s["table"], s["held"], s["lengths"], s["dst"])
        kda.mla_pages_fork(s["pool"], s["refs"], s["table"], s["held"], s["lengths"], s["src"], s["dst"], workspace=s["ws"])
        kda.mla_pages_reserve(s["case"]["page"], s["refs"], s["table"], s["held"], s["lengths"], s["dst"], s["extra"], workspace=s["ws"])
        return {k: s[k] for k in ("pool", "refs", "table", "held", "lengths")}
    if op == "cache":
        kda.mla_cache_append(s["pool"], s["table"], s["lengths"], s["cu"], s["rows"])
        kda.mla_cache_accept(s["pool"], s["table"], s["lengths"], s["cu"], s["parent"], s["accepted"], s["new_lengths"])
        return {k: s[k] for k in ("pool", "new_lengths")}
    if op == "verify":
        kda.kda_tree_verify(s["p"], s["x"], s["conv_w"], s["conv_state"], s["g"], s["beta"], s["state"], s["cu"], s["parent"], s["out"],
                            max_nodes=s["most"], slot_idx=s["slots"], gate_logit=s["gate"], norm_w=s["norm_w"])
        return s["out"]
    kda.kda_tree_accept(s["p"], s["x"], s["conv_w"], s["conv_state"], s["g"], s["beta"], s["state"], s["cu"], s["parent"], s["accepted"],
                        slot_idx=s["slots"])
    return {"state": s["state"], "conv_state": s["conv_state"]}


def _padded(s):
    """For [sequence, node]: the packed row (clamped), and whether there is such a node."""
    cu = s["cu"].long()
    i = torch.arange(s["most"], device=DEV)
    rows = cu[:-1, None] + i[None, :]
    valid = rows < cu[1:, None]
    return rows.clamp(max=int(s["parent"].numel()) - 1), valid


def _plain_tree(s):
    rows, valid = _padded(s)
    n, w = rows.shape
    pool, table, lengths = s["pool"], s["table"], s["lengths"].long()
    page = pool.shape[1]
    keys = pool[table.clamp(min=0).long()].reshape(n, -1, KEY).float()          # [n, L, 576]
    h = s["q"].shape[1]
    q = s["q"][rows].float().reshape(n, w * h, KEY)
    score = torch.matmul(q, keys.transpose(1, 2)).mul_(SCALE).view(n, w, h, -1)
    t = torch.arange(keys.shape[1], device=DEV)
    back = t[None, :] - lengths[:, None]                                         # drafted node at a position
    drafted = (back >= 0) & (back < valid.sum(1)[:, None])
    bit = (s["mask"][rows][:, :, None] >> back.clamp(0, 63)[:, None, :]) & 1
    seen = (back < 0)[:, None, :] | (drafted[:, None, :] & (bit == 1))           # [n, w, L]
    score.masked_fill_(~seen[:, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    score = score.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    z = torch.matmul(score.view(n, w * h, -1), keys[:, :, :LATENT]).view(n, w, h, LATENT)
    total = score.sum(-1, keepdim=True)
    z = z / torch.where(total > 0, total, torch.ones_like(total))
    return z[valid].to(torch.bfloat16)


def _lowest_free(refs, k):
    """The k lowest pages that nobody holds."""
    return torch.argsort((refs > 0).to(torch.uint8), stable=True)[:k].to(torch.int32)


def _plain_pages(s):
    refs, table, held, lengths, pool = s["refs"], s["table"], s["held"], s["lengths"], s["pool"]
    src, dst = s["src"].long(), s["dst"].long()
    page, most = pool.shape[2], table.shape[1]
    j = torch.arange(most, device=DEV, dtype=torch.int32)[None, :]
    # free
    mine = j < held[dst][:, None]
    refs.index_add_(0, table[dst].clamp(min=0).long().reshape(-1), -mine.to(torch.int32).reshape(-1))
    table[dst] = torch.where(mine, torch.full_like(table[dst], -1), table[dst])
    held[dst], lengths[dst] = 0, 0
    # fork: full pages shared, the partly filled one copied
    length = lengths[src]
    full, part = length // page, (length % page > 0)
    shared = j < full[:, None]
    taken = table[src]
    refs.index_add_(0, taken.clamp(min=0).long().reshape(-1), shared.to(torch.int32).reshape(-1))
    free = _lowest_free(refs, dst.numel())
    rank = torch.cumsum(part.to(torch.int32), 0) - part.to(torch.int32)
    fresh = free[rank.long()]
    old = taken.gather(1, full.clamp(max=most - 1).long()[:, None])[:, 0].long()
    inside = (torch.arange(page, device=DEV)[None, :] < (length % page)[:, None])[part][None, :, :, None]
    pool[:, fresh[part].long()] = torch.where(inside, pool[:, old[part]], pool[:, fresh[part].long()])
    refs.index_add_(0, fresh.long(), part.to(torch.int32))
    row = torch.where(shared, taken, torch.full_like(taken, -1))
    table[dst] = torch.where((j == full[:, None]) & part[:, None], fresh[:, None], row)
    held[dst] = full + part.to(torch.int32)
    lengths[dst] = length
    # reserve
    need = (lengths[dst] + s["extra"] + page - 1) // page
    new = (j >= held[dst][:, None]) & (j < need[:, None])
    at = torch.cumsum(new.reshape(-1).to(torch.int32), 0).view_as(new) - 1
    free = _lowest_free(refs, min(refs.numel(), new.numel()))
    pick = free[at.clamp(min=0, max=free.numel() - 1).long()]
    table[dst] = torch.where(new, pick, table[dst])
    refs.index_add_(0, pick.long().reshape(-1), new.to(torch.int32).reshape(-1))
    held[dst] = need
    return {k: s[k] for k in ("pool", "refs", "table", "held", "lengths")}


def _plain_cache(s):
    rows, valid = _padded(s)
    pool, table, lengths = s["pool"], s["table"], s["lengths"].long()
    page, layers = pool.shape[2], pool.shape[0]
    flat = pool.view(layers, -1, KEY)

    def place(at):                                       # pool row of [sequence, position]
        return table.gather(1, (at // page).clamp(max=table.shape[1] - 1)).clamp(min=0).long() * page + at % page

    i = torch.arange(rows.shape[1], device=DEV)[None, :]
    where = place(lengths[:, None] + i)
    flat[:, where[valid]] = s["rows"]
    # the accepted path, root first: node i is on it where bit i of the accepted node's ancestors is set
    accepted = s["accepted"].long()
    on = _ancestors(s, rows, valid).gather(1, accepted.clamp(min=0)[:, None, None].expand(-1, 1, rows.shape[1]))[:, 0]
    on = on & (accepted >= 0)[:, None]
    step = torch.cumsum(on.long(), 1) - 1
    to = place(lengths[:, None] + step.clamp(min=0))
    flat[:, to[on]] = flat[:, where[on]]
    s["new_lengths"].copy_(lengths + on.sum(1))
    return {k: s[k] for k in ("pool", "new_lengths")}


def _ancestors(s, rows, valid):
    """[sequence, node, node]: whether the second is the first or one of its ancestors."""
    w = rows.shape[1]
    parent = torch.where(valid, s["parent"][rows].long(), torch.full_like(rows, -1))
    up = (parent[:, :, None] == torch.arange(w, device=DEV)).float()
    reach = torch.eye(w, device=DEV).expand(rows.shape[0], w, w) + up
    for _ in range(max(1, (w - 1).bit_length())):        # paths of twice the length each time
        reach = (torch.matmul(reach, reach) > 0).float()
    return reach > 0


def _streams(s, rows, valid):
    """q, k, v of every [sequence, node, head] after the convolution along its path (32 bits), q and k normalised."""
    n, w = rows.shape
    c = s["x"].shape[1]
    x = torch.cat([s["conv_state"][s["slots"].long()], s["x"][rows]], 1).float()  # tail first: position i + 3 is node i
    parent = torch.where(valid, s["parent"][rows].long(), torch.full_like(rows, -1))

    def up(a):                                            # the token before node a on its path; below 0: the tail
        return torch.where(a >= 0, parent.gather(1, a.clamp(min=0)), (a - 1).clamp(min=-3))

    a0 = torch.arange(w, device=DEV).expand(n, w)
    a1 = up(a0)
    a2 = up(a1)
    a3 = up(a2)
    cw = s["conv_w"].float()
    tap = lambda a: x.gather(1, (a + 3)[:, :, None].expand(-1, -1, c))  # noqa: E731
    y = cw[:, 0] * tap(a3) + cw[:, 1] * tap(a2) + cw[:, 2] * tap(a1) + cw[:, 3] * tap(a0)
    y = (y * torch.sigmoid(y)).view(n, w, 3, -1, HD)
    q, k, v = y.unbind(2)
    unit = lambda t: t * torch.rsqrt(t.square().sum(-1, keepdim=True) + 1e-6)  # noqa: E731
    return unit(q), unit(k), v, (a1, a2, x)


def _plain_verify(s):
    rows, valid = _padded(s)
    n, w = rows.shape
    q, k, v, _ = _streams(s, rows, valid)
    decay = s["g"][rows].clamp(min=-5.0).exp()
    beta = s["beta"][rows]
    h = q.shape[2]
    parent = torch.where(valid, s["parent"][rows].long(), torch.full_like(rows, -1))
    seq = torch.arange(n, device=DEV)
    state = torch.empty(n, w + 1, h, HD, HD, device=DEV)  # the pool state, then the state after each node
    state[:, 0] = s["state"][s["slots"].long()]
    o = torch.empty(n, w, h, HD, device=DEV)
    for i in range(w):                                    # a node needs its parent's state
        m = state[seq, parent[:, i] + 1] * decay[:, i, :, :, None]
        u = beta[:, i, :, None] * (v[:, i] - (m * k[:, i, :, :, None]).sum(2))
        m += k[:, i, :, :, None] * u[:, :, None, :]
        state[:, i + 1] = m
        o[:, i] = (m * q[:, i, :, :, None]).sum(2)
    o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-6) * s["norm_w"] * torch.sigmoid(s["gate"][rows].float())
    return o[valid].to(torch.bfloat16)


def _plain_accept(s):
    rows, valid = _padded(s)
    n, w = rows.shape
    _, k, v, (a1, a2, x) = _streams(s, rows, valid)
    decay = s["g"][rows].clamp(min=-5.0).exp()
    beta = s["beta"][rows]
    slots, accepted = s["slots"].long(), s["accepted"].long()
    on = _ancestors(s, rows, valid).gather(1, accepted[:, None, None].expand(-1, 1, w))[:, 0]
    m = s["state"][slots]
    for i in range(w):                                    # the path's tokens in order
        t = m * decay[:, i, :, :, None]
        u = beta[:, i, :, None] * (v[:, i] - (t * k[:, i, :, :, None]).sum(2))
        t += k[:, i, :, :, None] * u[:, :, None, :]
        m = torch.where(on[:, i, None, None, None], t, m)
    s["state"][slots] = m
    # the last three raw inputs of the path, oldest first
    pick = torch.stack([a2.gather(1, accepted[:, None])[:, 0], a1.gather(1, accepted[:, None])[:, 0], accepted], 1) + 3
    s["conv_state"][slots] = x.gather(1, pick[:, :, None].expand(-1, -1, x.shape[2])).to(torch.bfloat16)
    return {"state": s["state"], "conv_state": s["conv_state"]}


# ---- from the definitions, in 64 bits ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s, case)
    if case["op"] in ("pages", "cache"):
        return {"pool": _exact_pool(s, case)}
    return _exact_kda(s, case)


def _exact_tree(s, case):
    lengths, counts, parents, _ = _sizes(case)
    out, at = [], 0
    for b, (length, w) in enumerate(zip(lengths, counts)):
        pages = s["table"][b][: -(-(length + w) // case["page"])].long()
        keys = s["pool"][pages].reshape(-1, KEY)[: length + w].double()
        for i in range(w):
            path, j = [], i
            while j >= 0:
                path.append(length + j)
                j = parents[at + j]
            mine = torch.cat([keys[:length], keys[path]])
            p = torch.softmax(s["q"][at + i].double() @ mine.T * SCALE, -1)
            out.append(p @ mine[:, :LATENT])
        at += w
    return torch.stack(out)


def _exact_pool(s, case):
    """Copies alone: the values of the pages and rows after the pass, row by row."""
    lengths, counts, parents, accepted = _sizes(case)
    pool, table, page = s["pool"].clone(), s["table"].tolist(), case["page"]
    if case["op"] == "cache":
        at = 0
        for b, (length, w) in enumerate(zip(lengths, counts)):
            spot = lambda t: (table[b][t // page], t % page)  # noqa: B023, E731
            for i in range(w):
                pool[:, spot(length + i)[0], spot(length + i)[1]] = s["rows"][:, at + i]
            path, j = [], accepted[b]
            while j >= 0:
                path.insert(0, j)
                j = parents[at + j]
            for i, j in enumerate(path):
                pool[:, spot(length + i)[0], spot(length + i)[1]] = s["rows"][:, at + j]
            at += w
        return pool.double()
    refs = s["refs"].tolist()
    free = iter([i for i, r in enumerate(refs) if r == 0])
    for b, length in enumerate(lengths):
        for _ in range(case["children"]):
            if length % page:
                pool[:, next(free), : length % page] = s["pool"][:, table[b][length // page], : length % page]
    return pool.double()


def _exact_kda(s, case):
    _, counts, parents, accepted = _sizes(case)
    h = case["heads"]
    slots = s["slots"].tolist()
    cw = s["conv_w"].double()
    state, tails = s["state"].double(), s["conv_state"].double()
    out, at = [], 0
    for b, w in enumerate(counts):
        mine = parents[at:at + w]
        paths = []
        for i in range(w):
            paths.append((paths[mine[i]] if mine[i] >= 0 else []) + [i])
        x, tail = s["x"][at:at + w].double(), s["conv_state"][slots[b]].double()
        y = []
        for path in paths:
            taps = torch.cat([tail, x[path]])[-4:]
            y.append((taps * cw.T).sum(0))
        y = torch.stack(y)
        y = (y / (1 + torch.exp(-y))).view(w, 3, h, HD)
        q, k = (t / torch.sqrt(t.square().sum(-1, keepdim=True) + 1e-6) for t in (y[:, 0], y[:, 1]))
        v = y[:, 2]
        g = s["g"][at:at + w].double().clamp(min=-5.0)
        beta = s["beta"][at:at + w].double()
        m0 = state[slots[b]]
        if case["op"] == "verify":
            # each node's state unrolled as a sum of decayed writes: the writes by forward substitution
            on = torch.zeros(w, w, device=DEV, dtype=torch.float64)
            for i, path in enumerate(paths):
                on[i, path] = 1
            total = torch.einsum("ij,jhc->ihc", on, g)
            span = torch.where(on[:, :, None, None] > 0, total[:, None] - total[None], torch.full((), -math.inf, device=DEV, dtype=torch.float64)).exp()
            kk = torch.einsum("ihc,jhc,ijhc->hij", k, k, span)
            qk = torch.einsum("ihc,jhc,ijhc->hij", q, k, span)
            lower = torch.tril(kk, -1) * beta.T[:, :, None] + torch.eye(w, device=DEV, dtype=torch.float64)
            right = beta[:, :, None] * (v - torch.einsum("ihc,hcd->ihd", k * total.exp(), m0))
            u = torch.linalg.solve_triangular(lower, right.transpose(0, 1), upper=False)
            o = torch.einsum("ihc,hcd->ihd", q * total.exp(), m0) + torch.einsum("hij,hjd->ihd", qk, u)
            o = o / torch.sqrt(o.square().mean(-1, keepdim=True) + 1e-6) * s["norm_w"].double() / (1 + torch.exp(-s["gate"][at:at + w].double()))
            out.append(o)
        else:
            m, path = m0, paths[accepted[b]]
            for i in path:
                m = g[i].exp()[:, :, None] * m
                m = m + k[i][:, :, None] * (beta[i][:, None] * (v[i] - torch.einsum("hc,hcd->hd", k[i], m)))[:, None, :]
            state[slots[b]] = m
            tails[slots[b]] = torch.cat([tail, x[path]])[-3:]
        at += w
    return torch.cat(out) if case["op"] == "verify" else {"state": state, "conv_state": tails}
