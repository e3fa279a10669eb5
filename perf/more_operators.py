"""The long-context operators of the paged latent cache as a serving step uses them: what is timed, on which inputs.

Four operators, each with its plain form in elementary torch operations and, where `own` is set, the
library's call:

  weights  the attention that each cached position received in a step, added to its running sum
  evict    a sequence cut to a budget of positions, the heaviest kept, its rows compacted in every layer
  keys     the mean row of every page that filled up, the key of that page as a block
  sparse   blocks scored by their keys, the best chosen, and attention over those alone

A case's "shape" number fixes its ragged sizes, so that the work of a case does not depend on the
seed; the seed fixes every value and the placement of the pages.
"""
import math
import random

import torch

own = False

DEV = "cuda"
LATENT, KEY = 512, 576
SCALE = 192 ** -0.5


def listed():
    return [
        # one user on one of four tensor-parallel ranks: 16 heads, one token, a short prompt
        dict(name="weights_1x1_h16", op="weights", n=1, nodes=1, heads=16, length=700, page=16, shape=1),
        # every decode step of a full batch
        dict(name="weights_256x1", op="weights", n=256, nodes=1, heads=64, length=4096, page=64, shape=2),
        # the last tokens of long prompts, whose attention decides what is kept of them
        dict(name="weights_8x32_window", op="weights", n=8, nodes=32, heads=64, length=16384, page=64, shape=3),
        # one conversation past its budget
        dict(name="evict_1", op="evict", n=1, length=1500, budget=1024, layers=9, page=16, shape=4),
        # a batch cut to half of its cache in all latent layers
        dict(name="evict_64", op="evict", n=64, length=4096, budget=2048, layers=9, page=64, shape=5),
        # a few long contexts
        dict(name="evict_4_long", op="evict", n=4, length=65536, budget=16384, layers=9, page=64, shape=6),
        # a decode step of a full batch: few pages fill up
        dict(name="keys_256_step", op="keys", n=256, length=4096, added=1, layers=9, page=64, shape=7),
        # prompts just written
        dict(name="keys_16_prompt", op="keys", n=16, length=8192, added=8192, layers=9, page=64, shape=8),
        # one user on one of four tensor-parallel ranks, small pages
        dict(name="sparse_1x1_h16", op="sparse", n=1, nodes=1, heads=16, length=5000, page=16, blocks=32, shape=9),
        # decode of a full batch, a quarter of each context read
        dict(name="sparse_256x1", op="sparse", n=256, nodes=1, heads=64, length=4096, page=64, blocks=16, shape=10),
        # drafted chains over longer contexts
        dict(name="sparse_16x4", op="sparse", n=16, nodes=4, heads=64, length=32768, page=64, blocks=32, shape=11),
        # long contexts, a sixty-fourth of them read
        dict(name="sparse_4x1_long", op="sparse", n=4, nodes=1, heads=64, length=262144, page=64, blocks=64, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["weights", "weights", "evict", "keys", "sparse", "sparse"])
    shape = rng.randrange(1, 1 << 30)
    page = rng.choice([16, 32, 64, 128])
    if op == "weights":
        heads, n, nodes = rng.choice([16, 32, 64]), _log(rng, 1, 256), _log(rng, 1, 33)
        most = min(65536, (1 << 28) // (n * nodes * heads), (1 << 20) // n)
        return dict(op=op, n=n, nodes=nodes, heads=heads, length=_log(rng, 1, max(2, most)), page=page, shape=shape)
    if op == "evict":
        n, layers = _log(rng, 1, 64), rng.choice([1, 3, 9])
        length = _log(rng, 40, min(65536, (9 << 18) // (n * layers)))
        return dict(op=op, n=n, length=length, budget=max(16, int(length * rng.uniform(0.1, 1.0))), layers=layers, page=page, shape=shape)
    if op == "keys":
        n, layers = _log(rng, 1, 256), rng.choice([1, 9])
        length = _log(rng, 100, min(65536, (9 << 17) // (n * layers)))
        return dict(op=op, n=n, length=length, added=_log(rng, 1, length), layers=layers, page=page, shape=shape)
    heads, n, nodes = rng.choice([16, 32, 64]), _log(rng, 1, 256), rng.randint(1, 4)
    blocks = _log(rng, 4, 64 if heads == 64 else 32)
    most = min(262144, (1 << 20) // n, (1 << 24) // (n * nodes))
    return dict(op=op, n=n, nodes=nodes, heads=heads, length=_log(rng, 60, most), page=page, blocks=blocks, shape=shape)


# ---- the sizes that a case's shape number stands for ----------------------------------------

FIRST, RECENT = 4, 32           # positions that eviction always keeps
FIRST_BLOCKS, RECENT_BLOCKS = 1, 2  # blocks that the selection always takes


def _sizes(case):
    """(lengths, drafted nodes of each sequence, accepted ones among them)"""
    r = random.Random(case["shape"])
    n, most = case["n"], case.get("nodes", 0)
    lengths = [case["length"] - r.randrange(case["length"] // 2 + 1) for _ in range(n)]
    lengths[r.randrange(n)] = case["length"]
    counts = [most - r.randrange(most // 3 + 1) if most > 1 else most for _ in range(n)]
    if most:
        counts[r.randrange(n)] = most
    accepted = [1 + r.randrange(w) if w else 0 for w in counts]
    return lengths, counts, accepted


def _kept(case):
    """(budget, first, recent) of an eviction: what is always kept fits the budget."""
    first = min(FIRST, case["budget"])
    return case["budget"], first, min(RECENT, case["budget"] - first)


def _selected_pages(case):
    """Room of a selection's table row: the blocks, then the page in use and those of the drafted rows."""
    return case["blocks"] + (2 * (case["page"] - 1) + case["nodes"]) // case["page"]


def work(case):
    lengths, counts, _ = _sizes(case)
    total, page = sum(counts), case["page"]
    if case["op"] == "weights":
        h = case["heads"]
        keys = sum(x + w for x, w in zip(lengths, counts))
        pairs = sum(h * w * (x + (w + 1) / 2) for x, w in zip(lengths, counts))
        return {"bytes": keys * (KEY * 2 + 8) + total * h * (KEY * 2 + 4), "flops": 2.0 * pairs * KEY}
    if case["op"] == "evict":
        budget, _, _ = _kept(case)
        cut = [x for x in lengths if x > budget]
        # of the kept rows, those behind the first gap move: about all of them
        return {"bytes": 2 * len(cut) * budget * KEY * 2 * case["layers"] + sum(8 * x for x in lengths) + 4 * case["n"] * budget, "flops": 0}
    if case["op"] == "keys":
        filled = sum(x // page - max(0, x - case["added"]) // page for x in lengths)
        return {"bytes": filled * case["layers"] * (page + 1) * KEY * 2 + 8 * case["n"], "flops": float(filled * case["layers"] * page * KEY)}
    h = case["heads"]
    full = [x // page for x in lengths]
    read = [min(f, case["blocks"]) * page + x % page for f, x in zip(full, lengths)]
    pairs = sum(h * w * (r + (w + 1) / 2) for r, w in zip(read, counts))
    return {"bytes": sum(full) * (KEY * 2 + 4) + sum(r + w for r, w in zip(read, counts)) * KEY * 2 + total * h * (KEY + LATENT) * 2,
            "flops": 2.0 * KEY * sum(h * w * f for f, w in zip(full, counts)) + 2.0 * pairs * (KEY + LATENT)}


# ---- inputs ----------------------------------------------------------------------------------

class _Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(int(seed))

    def normal(self, *shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, generator=self.g, device=DEV, dtype=torch.float32).mul_(std).to(dtype)

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.g, device=DEV, dtype=torch.float32)

    def order(self, n):
        return torch.randperm(n, generator=self.g, device=DEV).to(torch.int32)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _table(d, needs, most, n_pages):
    """Page table rows with the given numbers of pages, placed at random."""
    order = d.order(n_pages)
    need = _i32(needs)
    at = torch.cumsum(need, 0) - need
    j = torch.arange(most, device=DEV, dtype=torch.int32)
    used = j[None, :] < need[:, None]
    idx = (at[:, None] + j[None, :]).clamp_(max=n_pages - 1)
    return torch.where(used, order[idx.long()], torch.full_like(idx, -1)).to(torch.int32).contiguous()


def prepare(case, seed):
    d = _Draw(seed)
    lengths, counts, accepted = _sizes(case)
    n, total, page, op = case["n"], sum(counts), case["page"], case["op"]
    layers = case.get("layers", 1)
    needs = [-(-(x + w) // page) for x, w in zip(lengths, counts)]
    n_pages, most = sum(needs) + 3, max(needs)
    s = {"case": case, "op": op, "lengths": _i32(lengths), "most": max(counts)}
    s["table"] = _table(d, needs, most, n_pages)
    cu = [0]
    for w in counts:
        cu.append(cu[-1] + w)
    s["cu"], s["total"] = _i32(cu), total
    if op == "weights":
        h = case["heads"]
        s["pool"], s["q"] = d.normal(n_pages, page, KEY), d.normal(total, h, KEY)
        s["lse"] = torch.empty(total, h, device=DEV)  # as the step's attention left it
        for b in range(n):
            lo, w, x = cu[b], counts[b], lengths[b]
            keys = s["pool"][s["table"][b, : needs[b]].long()].view(-1, KEY)[: x + w].float()
            score = torch.matmul(s["q"][lo:lo + w].float(), keys.T).mul_(SCALE)
            t = torch.arange(x + w, device=DEV)
            behind = t[None, None, :] > x + torch.arange(w, device=DEV)[:, None, None]
            s["lse"][lo:lo + w] = torch.logsumexp(score.masked_fill_(behind, -math.inf).double(), -1).float()
        # the accepted drafts count, the others do not
        s["node_weight"] = torch.cat([(torch.arange(w, device=DEV) < a).float() for w, a in zip(counts, accepted)]) if case["nodes"] > 1 else None
        s["weights"] = d.uniform(n, most * page)
    elif op == "evict":
        s["pool"] = d.normal(layers, n_pages, page, KEY)
        s["refs"] = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        s["refs"][s["table"][s["table"] >= 0].long()] = 1
        # a few positions hold most of the attention, some have had none yet
        w = d.normal(n, most * page, std=2.0, dtype=torch.float32).exp_()
        s["weights"] = torch.where(d.uniform(n, most * page) < 0.1, torch.zeros_like(w), w)
        s["kept"] = torch.empty(n, case["budget"], dtype=torch.int32, device=DEV)
        s["new_lengths"] = torch.empty(n, dtype=torch.int32, device=DEV)
        s["new_weights"] = torch.zeros_like(s["weights"])
    elif op == "keys":
        s["pool"] = d.normal(layers, n_pages, page, KEY)
        s["before"] = _i32([max(0, x - case["added"]) for x in lengths])
        s["keys"] = d.normal(layers, n_pages, KEY)
    else:
        _prepare_sparse(s, d, case, lengths, n_pages)
        if own:
            from hybrid_linear_attention_gb300 import kda
            s["ws"] = torch.empty(kda.mla_sparse_workspace_size(n, total, case["heads"], most), dtype=torch.uint8, device=DEV)
    return s


def _prepare_sparse(s, d, case, lengths, n_pages):
    """A step whose queries look for one topic: each sequence has a direction, its blocks hold the topic
    to a degree that falls off with their rank, and the heads' queries share the direction."""
    n, page, h, total = case["n"], case["page"], case["heads"], s["total"]
    table = s["table"]
    ranked = (3 * case["blocks"] + 1) // 2
    topic = d.normal(n + 1, KEY, dtype=torch.float32)
    topic /= topic.square().sum(-1, keepdim=True).sqrt()
    rank = torch.argsort(d.uniform(n, table.shape[1]) + (table < 0), 1).argsort(1)   # of each of a sequence's pages
    logit = 6.0 - 12.0 * rank.clamp(max=ranked).float() / ranked - (rank >= ranked).float()
    owner = torch.full((n_pages,), n, dtype=torch.long, device=DEV)
    level = torch.zeros(n_pages, device=DEV)
    at = table.clamp(min=0).long()[table >= 0]
    owner[at] = torch.arange(n, device=DEV)[:, None].expand_as(table)[table >= 0]
    level[at] = logit[table >= 0] / (24.0 * SCALE)
    pool = d.normal(n_pages, page, KEY, dtype=torch.float32)
    g = topic[owner][:, None, :]
    within = 0.5 * d.normal(n_pages, page, dtype=torch.float32)
    along = level[:, None] + within - within.mean(1, keepdim=True)
    pool += g * (along - (pool * g).sum(-1))[:, :, None]
    s["pool"] = pool.to(torch.bfloat16)
    s["keys"] = s["pool"].float().mean(1).to(torch.bfloat16)
    of = torch.repeat_interleave(torch.arange(n, device=DEV), s["cu"].diff().long())
    s["q"] = (24.0 * topic[of][:, None, :] + d.normal(total, h, KEY, std=0.5, dtype=torch.float32)).to(torch.bfloat16)
    s["scores"] = torch.zeros(n, table.shape[1], device=DEV)
    s["sel_table"] = torch.empty(n, _selected_pages(case), dtype=torch.int32, device=DEV)
    s["sel_lengths"] = torch.empty(n, dtype=torch.int32, device=DEV)
    s["z"] = torch.empty(total, h, LATENT, dtype=torch.bfloat16, device=DEV)


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    if own:
        return _library(s)
    return {"weights": _plain_weights, "evict": _plain_evict, "keys": _plain_keys, "sparse": _plain_sparse}[s["op"]](s)


def _library(s):
    from hybrid_linear_attention_gb300 import kda
    op = s["op"]
    if op == "weights":
        kda.mla_cache_weights(s["q"], s["pool"], s["table"], s["lengths"], s["cu"], s["lse"], s["weights"], node_weight=s["node_weight"],
                              scale=SCALE)
        return s["weights"]
    if op == "evict":
        budget, first, recent = _kept(s["case"])
        kda.mla_cache_evict(s["pool"], s["table"], s["lengths"], s["weights"], s["kept"], s["new_lengths"], s["new_weights"], first=first,
                            recent=recent, refcount=s["refs"])
        return {k: s[k] for k in ("pool", "kept", "new_lengths", "new_weights")}
    if op == "keys":
        kda.mla_block_keys(s["pool"], s["table"], s["before"], s["lengths"], s["keys"])
        return s["keys"]
    kda.mla_sparse_latent(s["q"], s["pool"], s["keys"], s["table"], s["lengths"], s["cu"], s["scores"], s["sel_table"], s["sel_lengths"],
                          s["z"], blocks=s["case"]["blocks"], first=FIRST_BLOCKS, recent=RECENT_BLOCKS, scale=SCALE, workspace=s["ws"])
    return {k: s[k] for k in ("z", "scores", "sel_table", "sel_lengths")}


def _padded(s):
    """For [sequence, node]: the packed row (clamped), and whether there is such a node."""
    cu = s["cu"].long()
    i = torch.arange(s["most"], device=DEV)
    rows = cu[:-1, None] + i[None, :]
    valid = rows < cu[1:, None]
    return rows.clamp(max=s["total"] - 1), valid


def _scores(s, table, lengths):
    """Scores [n, node, head, position] of a drafted chain over the pages of `table`, -inf where a position is not visible."""
    rows, valid = _padded(s)
    n, w = rows.shape
    keys = s["pool"][table.clamp(min=0).long()].reshape(n, -1, KEY).float()
    h = s["q"].shape[1]
    q = s["q"][rows].float().reshape(n, w * h, KEY)
    score = torch.matmul(q, keys.transpose(1, 2)).mul_(SCALE).view(n, w, h, -1)
    t = torch.arange(keys.shape[1], device=DEV)
    i = torch.arange(w, device=DEV)
    seen = (t[None, None, :] <= lengths[:, None, None] + i[None, :, None]) & valid[:, :, None]
    return score.masked_fill_(~seen[:, :, None, :], -math.inf), keys, rows, valid


def _plain_weights(s):
    score, _, rows, valid = _scores(s, s["table"], s["lengths"].long())
    part = score.sub_(s["lse"][rows][..., None]).exp_()
    if s["node_weight"] is not None:
        part = part * s["node_weight"][rows][:, :, None, None]
    s["weights"] += part.sum((1, 2))
    return s["weights"]


def _best(value, first, recent, count, most):
    """Which entries of each row [n, entries] of `count` valid ones are taken: the first, the most recent, and the
    largest others to `most` in all, the lower index first among equals."""
    j = torch.arange(value.shape[1], device=DEV)
    inside = j[None, :] < count[:, None]
    always = inside & ((j < first)[None, :] | (j[None, :] >= count[:, None] - recent))
    key = torch.where(always, torch.full_like(value, math.inf), torch.where(inside, value, torch.full_like(value, -math.inf)))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    place = torch.empty_like(order).scatter_(1, order, j.expand_as(order).contiguous())
    return (place < most) & inside


def _plain_evict(s):
    pool, table, lengths, weights = s["pool"], s["table"], s["lengths"], s["weights"]
    budget, first, recent = _kept(s["case"])
    page, layers = pool.shape[2], pool.shape[0]
    keep = _best(weights, first, recent, lengths, budget)
    place = torch.cumsum(keep.long(), 1) - 1
    seq, old = keep.nonzero(as_tuple=True)
    new = place[seq, old]
    s["kept"].fill_(-1)
    s["kept"][seq, new] = old.to(torch.int32)
    s["new_lengths"].copy_(lengths.clamp(max=budget))
    inside = torch.arange(weights.shape[1], device=DEV)[None, :] < lengths[:, None]
    s["new_weights"].masked_fill_(inside, 0.0)
    s["new_weights"][seq, new] = weights[seq, old]
    moved = old != new
    seq, old, new = seq[moved], old[moved], new[moved]
    flat = pool.view(layers, -1, KEY)
    spot = lambda t: table[seq, t // page].long() * page + t % page  # noqa: E731
    flat[:, spot(new)] = flat[:, spot(old)]
    return {k: s[k] for k in ("pool", "kept", "new_lengths", "new_weights")}


def _plain_keys(s):
    pool, table, keys = s["pool"], s["table"], s["keys"]
    page = pool.shape[2]
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    filled = (j >= (s["before"] // page)[:, None]) & (j < (s["lengths"] // page)[:, None])
    which = table[filled].long()
    keys[:, which] = pool[:, which].float().mean(2).to(torch.bfloat16)
    return keys


def _plain_sparse(s):
    case, table, lengths = s["case"], s["table"], s["lengths"].long()
    page, blocks, most = case["page"], case["blocks"], s["table"].shape[1]
    rows, valid = _padded(s)
    n, w = rows.shape
    full = lengths // page
    j = torch.arange(most, device=DEV)
    candidate = j[None, :] < full[:, None]
    # each row's softmax over the blocks, summed over the rows
    keys = s["keys"][table.clamp(min=0).long()].float()
    q = s["q"][rows].float().reshape(n, -1, KEY)
    score = torch.matmul(q, keys.transpose(1, 2)).mul_(SCALE).masked_fill_(~candidate[:, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    part = score.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    part = part / part.sum(-1, keepdim=True).clamp(min=1e-30)
    part = part.view(n, w, -1, most) * valid[:, :, None, None]
    s["scores"].copy_(torch.where(candidate, part.sum((1, 2)), s["scores"]))
    # the chosen blocks in order, then the pages of the last positions and of the drafted rows
    take = _best(s["scores"], FIRST_BLOCKS, RECENT_BLOCKS, full, blocks)
    last = (lengths + valid.sum(1) + page - 1) // page
    take = take | ((j[None, :] >= full[:, None]) & (j[None, :] < last[:, None]))
    place = torch.cumsum(take.long(), 1) - 1
    seq, at = take.nonzero(as_tuple=True)
    s["sel_table"].fill_(-1)
    s["sel_table"][seq, place[seq, at]] = table[seq, at]
    s["sel_lengths"].copy_(full.clamp(max=blocks) * page + lengths % page)
    score, keys, _, valid = _scores(s, s["sel_table"], s["sel_lengths"].long())
    top = score.amax(-1, keepdim=True)
    score = score.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    z = torch.matmul(score.view(n, -1, score.shape[-1]), keys[:, :, :LATENT]).view(n, w, -1, LATENT)
    z = z / score.sum(-1, keepdim=True).clamp(min=1e-30)
    s["z"].copy_(z[valid])
    return {k: s[k] for k in ("z", "scores", "sel_table", "sel_lengths")}


# ---- from the definitions, in 64 bits ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"weights": _exact_weights, "evict": _exact_evict, "keys": _exact_keys, "sparse": _exact_sparse}[case["op"]](s, case)


def _exact_weights(s, case):
    lengths, counts, _ = _sizes(case)
    out, at = s["weights"].double(), 0
    for b, (x, w) in enumerate(zip(lengths, counts)):
        rows = s["pool"][s["table"][b, : -(-(x + w) // case["page"])].long()].reshape(-1, KEY)[: x + w].double()
        for i in range(w):
            u = 1.0 if s["node_weight"] is None else float(s["node_weight"][at + i])
            p = torch.exp(rows[: x + i + 1] @ s["q"][at + i].double().T * SCALE - s["lse"][at + i].double())
            out[b, : x + i + 1] += u * p.sum(1)
        at += w
    return out


def _choose(values, count, first, recent, most):
    """Indices that are taken of `count` values in a list, ascending."""
    if count <= most:
        return list(range(count))
    middle = sorted(range(first, count - recent), key=lambda j: (-values[j], j))[: most - first - recent]
    return list(range(first)) + sorted(middle) + list(range(count - recent, count))


def _exact_evict(s, case):
    lengths, _, _ = _sizes(case)
    budget, first, recent = _kept(case)
    pool, table, page = s["pool"].clone(), s["table"].long(), case["page"]
    kept, weights = torch.full_like(s["kept"], -1), s["new_weights"].double()
    values = s["weights"].tolist()
    for b, x in enumerate(lengths):
        chosen = torch.tensor(_choose(values[b], x, first, recent, budget), device=DEV)
        m = chosen.numel()
        kept[b, :m] = chosen.to(torch.int32)
        weights[b, :x] = 0
        weights[b, :m] = s["weights"][b, chosen].double()
        to = torch.arange(m, device=DEV)
        pool[:, table[b, to // page], to % page] = s["pool"][:, table[b, chosen // page], chosen % page]
    return {"pool": pool.double(), "kept": kept, "new_lengths": _i32([min(x, budget) for x in lengths]), "new_weights": weights}


def _exact_keys(s, case):
    lengths, _, _ = _sizes(case)
    out, page = s["keys"].double(), case["page"]
    for b, x in enumerate(lengths):
        which = s["table"][b, max(0, x - case["added"]) // page: x // page].long()
        for layer in range(case["layers"]):
            out[layer, which] = s["pool"][layer, which].double().sum(1) / page
    return out


def _exact_sparse(s, case):
    lengths, counts, _ = _sizes(case)
    page, at, z = case["page"], 0, []
    scores, sel, cut = s["scores"].double(), torch.full_like(s["sel_table"], -1), []
    for b, (x, w) in enumerate(zip(lengths, counts)):
        full = x // page
        mine = s["table"][b].tolist()
        if full:
            k = s["keys"][s["table"][b, :full].long()].double()
            scores[b, :full] = torch.softmax(s["q"][at:at + w].double() @ k.T * SCALE, -1).sum((0, 1))
        chosen = _choose(scores[b].tolist(), full, FIRST_BLOCKS, RECENT_BLOCKS, case["blocks"])
        pages = [mine[j] for j in chosen] + mine[full: -(-(x + w) // page)]
        sel[b, : len(pages)] = _i32(pages)
        cut.append(len(chosen) * page + x % page)
        rows = s["pool"][sel[b, : len(pages)].long()].reshape(-1, KEY).double()
        for i in range(w):
            seen = rows[: cut[-1] + i + 1]
            z.append(torch.softmax(s["q"][at + i].double() @ seen.T * SCALE, -1) @ seen[:, :LATENT])
        at += w
    return {"z": torch.stack(z), "scores": scores, "sel_table": sel, "sel_lengths": _i32(cut)}
