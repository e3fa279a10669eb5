"""GPU: steps of a serving loop that uses the long-context calls together, eager and captured, and
calls that run at the same time on two streams."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from hybrid_linear_attention_gb300 import kda
from tests import _gpu
from tests import _long_ref as long
from tests import _tree_ref as ref

pytestmark = pytest.mark.gpu
COUNTS, H, PAGE, LAYERS, N_PAGES, MOST, BUDGET = [5, 1, 7, 3], 64, 32, 2, 60, 16, 150
TOTAL, N = sum(COUNTS), len(COUNTS)


class Step:
    """Four sequences whose drafts are verified over chosen blocks, accepted, weighed and, where they have
    outgrown their budget, cut."""

    def __init__(self):
        z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        bf, i32 = torch.bfloat16, torch.int32
        self.pool, self.keys = z(LAYERS, N_PAGES, PAGE, 576, dtype=bf), z(LAYERS, N_PAGES, 576, dtype=bf)
        self.refs, self.held, self.lengths = z(N_PAGES, dtype=i32), z(N, dtype=i32), z(N, dtype=i32)
        self.before, self.table = z(N, dtype=i32), torch.full((N, MOST), -1, dtype=i32, device="cuda")
        self.cu, self.extra = ref.i32([0] + [int(x) for x in np.cumsum(COUNTS)]), ref.i32(COUNTS)
        self.parent, self.accept, self.slots = z(TOTAL, dtype=i32), z(N, dtype=i32), ref.i32([0, 1, 2, 3])
        self.rows, self.q = z(LAYERS, TOTAL, 576, dtype=bf), z(LAYERS, TOTAL, H, 576, dtype=bf)
        self.mask, self.count = z(TOTAL, dtype=torch.int64), z(TOTAL)
        self.z, self.whole = z(LAYERS, TOTAL, H, 512), z(LAYERS, TOTAL, H, 512, dtype=bf)
        self.lse, self.scores, self.weights = z(LAYERS, TOTAL, H), z(LAYERS, N, MOST), z(N, MOST * PAGE)
        self.sel, self.cut = z(LAYERS, N, 7, dtype=i32), z(LAYERS, N, dtype=i32)
        self.kept = z(N, BUDGET, dtype=i32)
        size = max(kda.mla_sparse_workspace_size(N, TOTAL, H, MOST), kda.mla_tree_workspace_size(N, TOTAL, H))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.pages = torch.empty(kda.mla_pages_workspace_size(N), dtype=torch.uint8, device="cuda")

    def fill(self, seed):
        rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        for t in (self.rows, self.q, self.pool):
            t.copy_(torch.randn(t.shape, generator=g))
        lengths = [int(x) for x in rng.integers(0, 300, N)]
        pages = [-(-n // PAGE) for n in lengths]
        order = [int(x) for x in rng.permutation(N_PAGES)]
        table, refs = [], [0] * N_PAGES
        for k in pages:
            table.append([order.pop() for _ in range(k)])
            for page in table[-1]:
                refs[page] = 1
        self.table.copy_(ref.i32([r + [-1] * (MOST - len(r)) for r in table]))
        self.refs.copy_(ref.i32(refs)), self.held.copy_(ref.i32(pages)), self.lengths.copy_(ref.i32(lengths))
        self.parents = [ref.random_parents(rng, w, root_share=0.0) for w in COUNTS]
        self.accepted = [int(rng.integers(-1, c)) for c in COUNTS]
        self.parent.copy_(ref.i32([p for q in self.parents for p in q])), self.accept.copy_(ref.i32(self.accepted))
        on = [[float(i in ref.path_to(p, a)) for i in range(len(p))] for p, a in zip(self.parents, self.accepted)]
        self.count.copy_(torch.tensor([x for q in on for x in q]))
        for t in (self.weights, self.keys, self.before, self.z, self.whole, self.lse, self.scores, self.kept, self.ws):
            t.zero_()
        self.start = [t.clone() for t in (self.pool, self.table, self.lengths)]

    def run(self):
        kda.mla_block_keys(self.pool, self.table, self.before, self.lengths, self.keys)
        kda.mla_pages_reserve(PAGE, self.refs, self.table, self.held, self.lengths, self.slots, self.extra, workspace=self.pages)
        kda.mla_cache_append(self.pool, self.table, self.lengths, self.cu, self.rows)
        kda.mla_tree_mask(self.parent, self.cu, self.mask)
        for y in range(LAYERS):
            kda.mla_sparse_latent(self.q[y], self.pool[y], self.keys[y], self.table, self.lengths, self.cu, self.scores[y],
                                  self.sel[y], self.cut[y], self.z[y], blocks=4, first=1, recent=1, mask=self.mask,
                                  workspace=self.ws)
            kda.mla_tree_latent_lse(self.q[y], self.pool[y], self.table, self.lengths, self.cu, self.whole[y], self.lse[y],
                                    mask=self.mask, workspace=self.ws)
            kda.mla_cache_weights(self.q[y], self.pool[y], self.table, self.lengths, self.cu, self.lse[y], self.weights,
                                  mask=self.mask, node_weight=self.count)
        kda.mla_weights_accept(self.weights, self.lengths, self.cu, self.parent, self.accept)
        self.before.copy_(self.lengths)
        kda.mla_cache_accept(self.pool, self.table, self.lengths, self.cu, self.parent, self.accept, self.lengths)
        kda.mla_block_keys(self.pool, self.table, self.before, self.lengths, self.keys)
        kda.mla_cache_evict(self.pool, self.table, self.lengths, self.weights, self.kept, self.lengths, self.weights, first=4,
                            recent=16, refcount=self.refs)
        kda.mla_pages_trim(PAGE, self.refs, self.table, self.held, self.lengths, self.slots)
        self.before.zero_()
        kda.mla_block_keys(self.pool, self.table, self.before, self.lengths, self.keys)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.pool, self.keys, self.refs, self.table, self.held, self.lengths, self.weights, self.z,
                                    self.whole, self.lse, self.scores, self.sel, self.cut, self.kept)]


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_a_step_is_what_its_parts_say(seed):
    """The state behind a step, followed with lists and 64-bit sums."""
    _gpu.lib()
    s = Step()
    s.fill(seed)
    s.run()
    kda.kda_check_device_error()
    s.results()
    pool, table0, lengths = s.start[0].cpu(), s.start[1].tolist(), s.start[2].tolist()
    cu, rows, q = s.cu.tolist(), s.rows.cpu(), s.q.cpu()
    weights, tol = np.zeros((N, MOST * PAGE)), np.zeros((N, MOST * PAGE))
    caches = []
    for n in range(N):  # each sequence's rows as one tensor
        x = lengths[n]
        old = pool[:, table0[n][:-(-x // PAGE)]].reshape(LAYERS, -1, 576)[:, :x]
        caches.append(torch.cat([old, rows[:, cu[n]:cu[n + 1]]], 1))
    mask = [m for p in s.parents for m in ref.masks(p)]
    top = max(len(c[0]) for c in caches)
    for y in range(LAYERS):
        flat = torch.zeros(N, top, 576, dtype=torch.bfloat16)
        for n, c in enumerate(caches):
            flat[n, :c.shape[1]] = c[y]
        paged = flat.view(N, top, 576)
        lse, size = long.lse(q[y], paged, [[n] for n in range(N)], lengths, cu, mask, kda.MLA_SCALE)
        assert (np.abs(s.lse[y].double().cpu().numpy() - lse) <= 1e-4).all()
        w, t = long.weights(q[y], paged, [[n] for n in range(N)], lengths, cu, mask, s.count.tolist(), lse, kda.MLA_SCALE,
                            MOST * PAGE)
        weights += w
        tol += t + 2e-4 * w  # the lse that the call was given: within 1e-4 (as asserted), twice its exponent's slope
    for n in range(N):
        x, path = lengths[n], ref.path_to(s.parents[n], s.accepted[n])
        keep = list(range(x)) + [x + j for j in path]
        cache, w = caches[n][:, keep], weights[n, keep]
        count = len(keep)
        assert int(s.lengths[n]) == min(count, BUDGET)
        assert int(s.held[n]) == -(-min(count, BUDGET) // PAGE)
        kept = s.kept[n].tolist()[:min(count, BUDGET)]
        if count <= BUDGET:
            assert kept == list(range(count))
        else:  # what was kept weighs more than what was not, as far as the weights are known
            assert kept[:4] == [0, 1, 2, 3] and kept[-16:] == list(range(count - 16, count)) and kept == sorted(set(kept))
            out = sorted(set(range(count)) - set(kept))
            inner = kept[4:-16]
            slack = tol[n, keep][out].max() + tol[n, keep][inner].max()
            assert w[inner].min() >= w[out].max() - slack
        got_w = s.weights[n].double().cpu().numpy()
        assert (np.abs(got_w[:len(kept)] - w[kept]) <= tol[n, keep][kept] + 1e-6).all() and not got_w[len(kept):].any()
        pages = s.table[n].tolist()
        assert all(p >= 0 for p in pages[:int(s.held[n])]) and set(pages[int(s.held[n]):]) == {-1}
        now = s.pool[:, pages[:int(s.held[n])]].reshape(LAYERS, -1, 576)[:, :len(kept)].cpu()
        assert torch.equal(now, cache[:, kept])
        for j in range(len(kept) // PAGE):  # the keys of the pages as they are now
            mean = now[:, j * PAGE:(j + 1) * PAGE].double().mean(1)
            got = s.keys[:, pages[j]].double().cpu()
            assert ((got - mean).abs() <= 2.0**-8 * mean.abs() + 1e-5).all()
    named = [p for row in s.table.tolist() for p in row if p >= 0]
    assert sorted(named) == [p for p, r in enumerate(s.refs.tolist()) if r == 1] and set(s.refs.tolist()) <= {0, 1}


def test_a_captured_step_gives_the_eager_bits():
    _gpu.lib()
    s, want = Step(), []
    for seed in (1, 2, 3):
        s.fill(seed)
        torch.cuda.synchronize()
        s.run()
        kda.kda_check_device_error()
        want.append(s.results())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (3, 1, 2):
        s.fill(seed)
        torch.cuda.synchronize()
        graph.replay()
        kda.kda_check_device_error()
        for a, b in zip(s.results(), want[seed - 1]):
            assert torch.equal(a, b)


def test_the_first_calls_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import torch\n"
            "from tests.test_gpu_long_step import Step, kda\n"
            "s = Step(); s.fill(4); torch.cuda.synchronize()\n"
            "graph = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(graph): s.run()\n"
            "graph.replay(); kda.kda_check_device_error(); a = s.results()\n"
            "s.fill(4); torch.cuda.synchronize(); s.run(); kda.kda_check_device_error()\n"
            "assert all(torch.equal(x, y) for x, y in zip(a, s.results()))\n")
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_two_steps_at_once_on_two_streams():
    """Each with its own buffers and workspace; the same bits as one after another."""
    _gpu.lib()
    steps = [Step(), Step()]
    want = []
    for s, seed in zip(steps, (5, 6)):
        s.fill(seed)
        torch.cuda.synchronize()
        s.run()
        want.append(s.results())
        s.fill(seed)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, stream in zip(steps, streams):
        with torch.cuda.stream(stream):
            s.run()
    kda.kda_check_device_error()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.results(), w))


def test_calls_in_a_row_share_their_buffers():
    """Layer after layer with one selection, one score buffer and one workspace, and eviction after eviction
    with one list of kept positions: each launch overlaps the end of the one before, and sees what it wrote."""
    _gpu.lib()
    g = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n, page, blocks, layers = 24, 32, 5, 6
    lengths = [int(x) for x in np.random.default_rng(1).integers(200, 900, n)]
    most = 30
    table = torch.arange(n * most, dtype=torch.int32, device="cuda").view(n, most)
    pool, q = r(layers, n * most, page, 576).to(torch.bfloat16), r(layers, n, 16, 576).to(torch.bfloat16)
    keys = pool.float().mean(2).to(torch.bfloat16)
    size = kda.mla_sparse_workspace_size(n, n, 16, most)
    new = lambda: (torch.zeros(n, most, device="cuda"), torch.zeros(n, blocks + 3, dtype=torch.int32, device="cuda"),  # noqa: E731
                   torch.zeros(n, dtype=torch.int32, device="cuda"), torch.empty(size, dtype=torch.uint8, device="cuda"))
    cu, lens = ref.i32(list(range(n + 1))), ref.i32(lengths)

    def step(y, z, scores, sel, cut, ws):
        kda.mla_sparse_latent(q[y], pool[y], keys[y], table, lens, cu, scores, sel, cut, z, blocks=blocks, workspace=ws)

    want = [torch.zeros(n, 16, 512, device="cuda") for _ in range(layers)]
    for y in range(layers):
        step(y, want[y], *new())
        torch.cuda.synchronize()
    shared = new()
    for _ in range(20):
        got = [torch.zeros(n, 16, 512, device="cuda") for _ in range(layers)]
        torch.cuda.synchronize()
        for y in range(layers):
            step(y, got[y], *shared)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    weights = [torch.rand(n, most * page, generator=g, device="cuda") for _ in range(layers)]
    pools = [r(1, n * most, page, 576).to(torch.bfloat16) for _ in range(layers)]
    first = [p.clone() for p in pools]
    kept, cut, moved = torch.zeros(n, 150, dtype=torch.int32, device="cuda"), torch.zeros_like(lens), torch.zeros_like(weights[0])
    for y in range(layers):
        kda.mla_cache_evict(pools[y], table, lens, weights[y], kept, cut, moved, recent=8)
        torch.cuda.synchronize()
    for _ in range(20):
        again = [p.clone() for p in first]
        torch.cuda.synchronize()
        for y in range(layers):
            kda.mla_cache_evict(again[y], table, lens, weights[y], kept, cut, moved, recent=8)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, pools))
    kda.kda_check_device_error()


def test_wrong_shapes_types_and_devices_are_refused():
    _gpu.lib()
    s = Step()
    s.fill(7)
    q, args = s.q[0], (s.table, s.lengths, s.cu)
    with pytest.raises((TypeError, ValueError)):
        kda.mla_cache_weights(q, s.pool[0], *args, s.lse[0].double(), s.weights)
    with pytest.raises(ValueError):
        kda.mla_cache_weights(q, s.pool[0], *args, s.lse[0, :-1], s.weights)
    with pytest.raises(ValueError):
        kda.mla_cache_weights(q, s.pool[0], *args, s.lse[0], s.weights[:2])
    with pytest.raises((TypeError, ValueError)):
        kda.mla_cache_weights(q, s.pool[0], *args, s.lse[0], s.weights.cpu())
    with pytest.raises(ValueError):
        kda.mla_cache_evict(s.pool, s.table, s.lengths, s.weights, s.kept, s.lengths, s.weights[:, :-1].contiguous())
    with pytest.raises(ValueError):
        kda.mla_cache_evict(s.pool, s.table, s.lengths, s.weights, s.kept, s.lengths, refcount=s.refs[:-1].clone())
    with pytest.raises(kda.KdaError):
        kda.mla_cache_evict(s.pool, s.table, s.lengths, s.weights, s.kept, s.lengths, first=BUDGET, recent=1)
    with pytest.raises(ValueError):
        kda.mla_block_keys(s.pool, s.table, s.before, s.lengths, s.keys[:1])
    with pytest.raises(kda.KdaError):
        kda.mla_block_scores(q, s.keys[0], PAGE, *args, s.scores[0], workspace=None)
    with pytest.raises(ValueError):
        kda.mla_sparse_latent(q, s.pool[0], s.keys[0, :-1], *args, s.scores[0], s.sel[0], s.cut[0], s.z[0], blocks=4,
                              workspace=s.ws)
    with pytest.raises((TypeError, ValueError)):
        kda.mla_sparse_latent(q[:, ::2], s.pool[0], s.keys[0], *args, s.scores[0], s.sel[0], s.cut[0], s.z[0], blocks=4,
                              workspace=s.ws)
