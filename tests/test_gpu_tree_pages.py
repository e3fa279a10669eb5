"""GPU: the paged latent cache's row and page calls against lists in Python (bit-exact)."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_gb300 import kda
from tests import _gpu
from tests import _tree_ref as ref
from tests.test_gpu_tree_attention import Case
from tests.test_gpu_tree_kda import make, out_error, plain

pytestmark = pytest.mark.gpu


def status():
    try:
        kda.kda_check_device_error()
    except kda.KdaError as e:
        return e.status
    return kda.KDA_OK


class Both:
    """The device's pool and tables, and the model beside them."""

    def __init__(self, n_pages, n_slots, max_pages, page, layers=2, seed=0):
        _gpu.lib()
        g = torch.Generator().manual_seed(seed)
        self.model = ref.Pages(n_pages, n_slots, max_pages, page)
        self.pool = torch.randn(layers, n_pages, page, 576, generator=g).to(torch.bfloat16)
        self.d_pool = self.pool.cuda()
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((n_slots, max_pages), -1, dtype=torch.int32, device="cuda")
        self.held = torch.zeros(n_slots, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(n_slots, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(kda.mla_pages_workspace_size(2048), dtype=torch.uint8, device="cuda")

    def free(self, slots):
        kda.mla_pages_free(self.refs, self.table, self.held, self.lengths, ref.i32(slots))
        self.model.free(slots)

    def fork(self, src, dst):
        kda.mla_pages_fork(self.d_pool, self.refs, self.table, self.held, self.lengths, ref.i32(src), ref.i32(dst),
                           workspace=self.ws)

        def copied(old, new, rows):
            self.pool[:, new, :rows] = self.pool[:, old, :rows]
        return self.model.fork(src, dst, copied)

    def reserve(self, slots, extra):
        kda.mla_pages_reserve(self.model.page, self.refs, self.table, self.held, self.lengths, ref.i32(slots),
                              ref.i32(extra), workspace=self.ws)
        return self.model.reserve(slots, extra)

    def set_length(self, slot, n):
        self.lengths[slot] = n
        self.model.lengths[slot] = n

    def same(self):
        torch.cuda.synchronize()
        assert self.refs.tolist() == self.model.refs
        assert self.table.tolist() == self.model.table
        assert self.held.tolist() == self.model.held
        assert self.lengths.tolist() == self.model.lengths
        assert torch.equal(self.d_pool.cpu(), self.pool)


@pytest.mark.parametrize("page", [16, 64])
def test_random_life_of_a_pool(page):
    """Reserve, grow, fork and free in random order, until pages run out and after."""
    rng = np.random.default_rng(page)
    b = Both(24, 12, 9, page, seed=page)
    ran_out = 0
    for _ in range(60):
        kind = rng.integers(3)
        slots = [int(x) for x in rng.permutation(12)[:rng.integers(1, 5)]]
        if kind == 0:
            extra = [int(rng.integers(0, 3 * page)) for _ in slots]
            extra = [min(e, 9 * page - b.model.lengths[s]) for s, e in zip(slots, extra)]
            out = b.reserve(slots, extra)
            ran_out += out
            assert status() == (kda.KDA_ERR_NO_PAGES if out else kda.KDA_OK)
            for s in slots:
                b.set_length(s, min(b.model.held[s] * page, b.model.lengths[s] + int(rng.integers(0, 2 * page))))
        elif kind == 1:
            src = [s for s in range(12) if b.model.held[s]]
            dst = [s for s in slots if not b.model.held[s]]
            if src and dst:
                bad, out = b.fork([int(rng.choice(src)) for _ in dst], dst)
                ran_out += out
                assert not bad and status() == (kda.KDA_ERR_NO_PAGES if out else kda.KDA_OK)
        else:
            b.free(slots[:2])
            assert status() == kda.KDA_OK
        b.same()
    assert ran_out


def test_fork_refuses_and_reports():
    b = Both(30, 8, 4, 16)
    b.reserve([0, 1], [40, 16])
    b.set_length(0, 40)
    b.set_length(1, 16)
    bad, _ = b.fork([0, 0, 1, 0], [2, 1, 2, 3])  # 1 holds pages; 2 is taken by the first entry
    assert bad and status() == kda.KDA_ERR_BAD_INDEX
    b.same()
    bad, _ = b.fork([4, 0, 5], [4, 5, 6])  # a child of the same call cannot be a parent
    assert bad and status() == kda.KDA_ERR_BAD_INDEX
    b.same()
    kda.mla_pages_fork(b.d_pool, b.refs, b.table, b.held, b.lengths, ref.i32([0, 99]), ref.i32([-1, 7]), workspace=b.ws)
    assert status() == kda.KDA_ERR_BAD_INDEX
    b.same()


def test_reserve_and_free_refuse_and_report():
    b = Both(30, 8, 4, 16)
    b.reserve([0], [20])
    for slots, extra in (([1, 9], [16, 16]), ([2, 2], [16, 16]), ([3, 0], [16, 65]), ([4, 5], [3, -1])):
        kda.mla_pages_reserve(16, b.refs, b.table, b.held, b.lengths, ref.i32(slots), ref.i32(extra), workspace=b.ws)
        assert status() == kda.KDA_ERR_BAD_INDEX
        b.model.reserve(slots[:1], extra[:1])
        b.same()
    b.free([0, 0, 1])
    assert status() == kda.KDA_OK
    b.same()
    kda.mla_pages_free(b.refs, b.table, b.held, b.lengths, ref.i32([8, -1]))
    assert status() == kda.KDA_ERR_BAD_INDEX
    b.same()
    b.held[5] = 2  # a row that claims pages it does not name
    kda.mla_pages_free(b.refs, b.table, b.held, b.lengths, ref.i32([5]))
    assert status() == kda.KDA_ERR_BAD_INDEX
    b.same()


def test_a_large_pool_is_searched_to_its_end():
    """Free pages only at the far end; more entries than one pass of the bookkeeping takes."""
    n_pages, n = 50021, 1500
    _gpu.lib()
    refs = torch.full((n_pages,), 1, dtype=torch.int32, device="cuda")
    free = [3, 17, 16384] + list(range(n_pages - 2 * n, n_pages))
    refs[torch.tensor(free, device="cuda")] = 0
    table = torch.full((n, 2), -1, dtype=torch.int32, device="cuda")
    held, lengths = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
    slots, extra = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).contiguous(), ref.i32([17] * n)
    ws = torch.empty(kda.mla_pages_workspace_size(n), dtype=torch.uint8, device="cuda")
    kda.mla_pages_reserve(16, refs, table, held, lengths, slots, extra, workspace=ws)
    assert status() == kda.KDA_OK
    assert table.flip(0).reshape(-1).tolist() == free[:2 * n] and held.tolist() == [2] * n
    assert int((refs == 0).sum()) == len(free) - 2 * n


def test_pages_copy():
    b = Both(20, 1, 1, 32, layers=3)
    kda.mla_pages_copy(b.d_pool, ref.i32([1, 1, 2, 5]), ref.i32([7, 8, 9, 5]))
    assert status() == kda.KDA_OK
    b.pool[:, 7], b.pool[:, 8], b.pool[:, 9] = b.pool[:, 1].clone(), b.pool[:, 1].clone(), b.pool[:, 2].clone()
    b.same()
    # a target twice (the first has it), a target that is a source, indices out of range
    kda.mla_pages_copy(b.d_pool, ref.i32([1, 2, 3, 10, 20, 4]), ref.i32([11, 11, 10, 12, 13, -1]))
    assert status() == kda.KDA_ERR_BAD_INDEX
    b.pool[:, 11], b.pool[:, 12] = b.pool[:, 1].clone(), b.pool[:, 10].clone()
    b.same()


@pytest.mark.parametrize("layers", [1, 9, 11])
def test_append_and_accept(layers):
    """Rows across page edges; paths that skip nodes; nothing accepted; a tree of 64."""
    _gpu.lib()
    case = Case([0, 15, 16, 130, 7], [3, 20, 1, 64, 0], H=1, page=16, seed=12)
    g = torch.Generator().manual_seed(13)
    rows = torch.randn(layers, case.cu[-1] + 3, 576, generator=g).to(torch.bfloat16)  # three rows of no sequence
    pool = torch.randn(layers, case.pool.shape[0], 16, 576, generator=g).to(torch.bfloat16)
    d_pool, lengths = pool.cuda(), ref.i32(case.lengths)
    spot = lambda b, t: (case.table[b][t // 16], t % 16)  # noqa: E731
    kda.mla_cache_append(d_pool, ref.i32(case.table), lengths, ref.i32(case.cu), rows.cuda())
    assert status() == kda.KDA_OK
    for b in range(5):
        for i in range(case.counts[b]):
            p, r = spot(b, case.lengths[b] + i)
            pool[:, p, r] = rows[:, case.cu[b] + i]
    assert torch.equal(d_pool.cpu(), pool) and lengths.tolist() == case.lengths
    accept = [2, 19, 0, 63, -1]
    parents = [p for q in case.parents for p in q]
    kda.mla_cache_accept(d_pool, ref.i32(case.table), lengths, ref.i32(case.cu), ref.i32(parents), ref.i32(accept), lengths)
    assert status() == kda.KDA_OK
    want = []
    for b in range(5):
        path = ref.path_to(case.parents[b], accept[b])
        for d, i in enumerate(path):
            (p, r), (p0, r0) = spot(b, case.lengths[b] + d), spot(b, case.lengths[b] + i)
            pool[:, p, r] = rows[:, case.cu[b] + i]
        want.append(case.lengths[b] + len(path))
    assert torch.equal(d_pool.cpu(), pool) and lengths.tolist() == want


def test_rows_without_a_page_are_reported():
    _gpu.lib()
    pool = torch.zeros(1, 4, 16, 576, dtype=torch.bfloat16, device="cuda")
    rows = torch.ones(1, 6, 576, dtype=torch.bfloat16, device="cuda")
    table = ref.i32([[0, -1], [1, 99], [2, 3]])
    kda.mla_cache_append(pool, table, ref.i32([15, 15, 31]), ref.i32([0, 2, 4, 6]), rows)
    assert status() == kda.KDA_ERR_BAD_INDEX
    on = pool[0, :, :, 0].cpu()
    assert on.sum() == 3 and on[0, 15] == 1 and on[1, 15] == 1 and on[3, 15] == 1
    kda.mla_cache_append(pool, table, ref.i32([0, 0, 0]), ref.i32([0, 2, 9, 6]), rows)
    assert status() == kda.KDA_ERR_BAD_SEQLENS
    lengths = ref.i32([3, 4, -1])
    kda.mla_cache_accept(pool, table, lengths, ref.i32([0, 2, 4, 6]), ref.i32([-1, 0] * 3), ref.i32([2, -2, 1]), lengths)
    assert status() == kda.KDA_ERR_BAD_INDEX and lengths.tolist() == [3, 4, -1]


def test_accept_at_the_largest_length():
    """A length whose sum with the path would pass 32 bits keeps its value and is reported."""
    _gpu.lib()
    pool = torch.zeros(1, 4, 16, 576, dtype=torch.bfloat16, device="cuda")
    lengths = ref.i32([2**31 - 1, 3])
    kda.mla_cache_accept(pool, ref.i32([[0], [1]]), lengths, ref.i32([0, 1, 2]), ref.i32([-1, -1]), ref.i32([0, 0]), lengths)
    assert status() == kda.KDA_ERR_BAD_INDEX and lengths.tolist() == [2**31 - 1, 4]


def test_reserve_more_entries_than_fit_on_chip():
    """2500 entries: the notes are kept in the workspace; pages run out at the last ones."""
    n = 2500
    b = Both(n + 700, n, 2, 16, layers=1)
    b.ws = torch.empty(kda.mla_pages_workspace_size(n), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(31)
    slots = [int(x) for x in rng.permutation(n)]
    assert b.reserve(slots, [int(x) for x in rng.integers(0, 33, n)])
    assert status() == kda.KDA_ERR_NO_PAGES
    b.same()


def test_tensors_of_another_device_are_refused(monkeypatch):
    b = Both(4, 2, 2, 16)
    monkeypatch.setattr(kda, "_device", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        b.reserve([0], [3])
    monkeypatch.undo()
    b.same()


def test_a_verification_step_as_a_server_runs_it():
    """Two turns of: reserve, append the drafted rows, tree masks, latent attention and the KDA
    verify call, accept into both caches; a fork in between; everything against the plain forms."""
    _gpu.lib()
    H, page, layers = 2, 16, 2
    rng = np.random.default_rng(21)
    g = torch.Generator().manual_seed(21)
    b = Both(64, 3, 12, page, layers=layers, seed=22)
    p = kda.params(H=H)
    state = torch.randn(3, H, 128, 128, generator=g) * 0.1
    tail = torch.randn(3, 3, 3 * H * 128, generator=g).to(torch.bfloat16)
    d_state, d_tail = state.cuda(), tail.cuda()
    # a prompt for sequences 0 and 1
    prompt = [20, 33]
    rows = torch.randn(layers, 53, 576, generator=g).to(torch.bfloat16)
    b.reserve([0, 1], prompt)
    kda.mla_cache_append(b.d_pool, b.table, b.lengths, ref.i32([0, 20, 53]), rows.cuda())
    for n in range(2):
        for t in range(prompt[n]):
            b.pool[:, b.model.table[n][t // page], t % page] = rows[:, 20 * n + t]
        b.set_length(n, prompt[n])
    b.same()
    for turn in range(2):
        n = 2 + turn
        if turn == 1:  # a second sample of sequence 1
            assert b.fork([1], [2]) == (False, False)
            d_state[2], d_tail[2] = d_state[1], d_tail[1]
            state[2], tail[2] = state[1], tail[1]
        m = make([5, 4, 7][:n], H, 128, seed=23 + turn, slots=list(range(n)), n_slots=3)
        m["state"], m["conv_state"] = state, tail
        cu, parent = ref.i32(m["cu"]), ref.i32(m["parent"])
        counts = [m["cu"][i + 1] - m["cu"][i] for i in range(n)]
        assert not b.reserve(list(range(n)), counts)
        rows = torch.randn(layers, m["cu"][-1], 576, generator=g).to(torch.bfloat16)
        kda.mla_cache_append(b.d_pool, b.table, b.lengths, cu, rows.cuda())
        for i in range(n):
            for j in range(counts[i]):
                t = b.model.lengths[i] + j
                b.pool[:, b.model.table[i][t // page], t % page] = rows[:, m["cu"][i] + j]
        b.same()
        mask = torch.empty(m["cu"][-1], dtype=torch.int64, device="cuda")
        kda.mla_tree_mask(parent, cu, mask)
        q = torch.randn(m["cu"][-1], H, 576, generator=g).to(torch.bfloat16)
        z = torch.empty((m["cu"][-1], H, 512), device="cuda")
        ws = torch.empty(kda.mla_tree_workspace_size(n, m["cu"][-1], H), dtype=torch.uint8, device="cuda")
        for layer in range(layers):
            kda.mla_tree_latent(q.cuda(), b.d_pool[layer], b.table, b.lengths, cu, z, mask=mask, workspace=ws)
            want, unit, _ = ref.tree_attention(q, b.pool[layer], b.model.table, b.model.lengths[:n], m["cu"],
                                               mask.tolist(), kda.MLA_SCALE)
            assert (np.abs(z.double().cpu().numpy() - want) <= 1.1 * 2.0**-8 * (unit + np.abs(want))).all()
        out = torch.empty((m["cu"][-1], H, 128), dtype=torch.bfloat16, device="cuda")
        args = (p, m["x"].cuda(), m["conv_w"].cuda(), d_tail, m["g"].cuda(), m["beta"].cuda(), d_state, cu, parent)
        kda.kda_tree_verify(*args, out, max_nodes=7)
        accept = [int(rng.integers(-1, c)) for c in counts]
        kda.kda_tree_accept(*args, ref.i32(accept))
        kda.mla_cache_accept(b.d_pool, b.table, b.lengths, cu, parent, ref.i32(accept), b.lengths)
        assert status() == kda.KDA_OK
        o, new_state, new_tail = plain(m, p, gated=False, accept=accept)
        assert out_error(out, o) <= 1e-2
        assert np.abs(d_state.double().cpu().numpy() - new_state).max() <= 1e-4 * np.sqrt((new_state ** 2).mean())
        assert np.array_equal(d_tail.double().cpu().numpy(), new_tail)
        state, tail = d_state.cpu(), d_tail.cpu()
        for i in range(n):
            path = ref.path_to(m["parent"][m["cu"][i]:m["cu"][i + 1]], accept[i])
            for d, j in enumerate(path):
                t = b.model.lengths[i] + d
                b.pool[:, b.model.table[i][t // page], t % page] = rows[:, m["cu"][i] + j]
            b.model.lengths[i] += len(path)
        b.same()


@pytest.mark.parametrize("layers", [1, 11])
def test_accept_over_a_missing_page_keeps_rows_and_length(layers):
    """Pages of 16, lengths 14: nodes 0 and 1 on the sequence's first page, the others on its second.
    Sequence 0 a chain over a page that is not there, 1 a path whose source page alone is missing,
    2 a path that moves rows onto a missing page, 3 and 4 as they should be, 5 no path at all."""
    _gpu.lib()
    g = torch.Generator().manual_seed(61)
    pool = torch.randn(layers, 16, 16, 576, generator=g).to(torch.bfloat16)
    table = [[0, -1, 1], [2, 99, 3], [-1, 4, 5], [6, 7, 8], [9, 10, 11], [12, -1, -1]]
    parents = [[-1, 0, 1, 2], [-1, 0, 1, 0], [-1, -1, 1, 2], [-1, 0, 0, 2], [-1, 0, 1, 2], [-1, 0, 1, 2]]
    accept, lengths = [3, 3, 3, 3, 3, -1], [14] * 6
    want, new = pool.clone(), list(lengths)
    for b in (3, 4):
        path = ref.path_to(parents[b], accept[b])
        for d, i in enumerate(path):
            (p, r), (p0, r0) = ((table[b][(14 + x) // 16], (14 + x) % 16) for x in (d, i))
            want[:, p, r] = pool[:, p0, r0]
        new[b] += len(path)
    d_pool, out = pool.cuda(), ref.i32([-7] * 6)
    kda.mla_cache_accept(d_pool, ref.i32(table), ref.i32(lengths), ref.i32([0, 4, 8, 12, 16, 20, 24]),
                         ref.i32([p for q in parents for p in q]), ref.i32(accept), out)
    assert status() == kda.KDA_ERR_BAD_INDEX
    assert out.tolist() == new and torch.equal(d_pool.cpu(), want)
    # a plain chain over a missing page alone is told of too
    kda.mla_cache_accept(d_pool, ref.i32(table[:1]), ref.i32([14]), ref.i32([0, 4]), ref.i32(parents[0]), ref.i32([2]), out)
    assert status() == kda.KDA_ERR_BAD_INDEX
    assert out.tolist()[0] == 14 and torch.equal(d_pool.cpu(), want)


@pytest.mark.parametrize("n", [3, 33, 100])
def test_append_beside_bad_offsets(n):
    """Offsets below 0, past the rows or running backwards lose their own sequences' rows alone."""
    _gpu.lib()
    g = torch.Generator().manual_seed(62 + n)
    counts = [2 + i % 2 for i in range(n)]
    cu = [0] + [int(x) for x in np.cumsum(counts)]
    total = cu[-1]
    for at, value in ((n // 2, -5), (n - 1, -1), (n // 2, total + 7), (1, 0), (n // 3, -2**31)):
        bad = list(cu)
        bad[at] = value
        rows = torch.randn(2, total, 576, generator=g).to(torch.bfloat16)
        want = torch.zeros(2, n, 16, 576, dtype=torch.bfloat16)
        told = False
        for b in range(n):
            lo, hi = bad[b], bad[b + 1]
            if lo < 0 or hi < lo or hi > total:
                told = True
                continue
            want[:, b, 5:5 + hi - lo] = rows[:, lo:hi]
        pool = torch.zeros(2, n, 16, 576, dtype=torch.bfloat16, device="cuda")
        kda.mla_cache_append(pool, ref.i32([[b] for b in range(n)]), ref.i32([5] * n), ref.i32(bad), rows.cuda())
        assert status() == (kda.KDA_ERR_BAD_SEQLENS if told else kda.KDA_OK), (at, value)
        assert torch.equal(pool.cpu(), want), (at, value)


def test_free_of_a_sequence_without_pages_clears_its_length():
    b = Both(8, 3, 4, 16)
    b.reserve([0], [20])
    b.set_length(0, 20)
    b.lengths[1] = 9  # set before any page was reserved
    b.free([1, 0, 1])
    assert status() == kda.KDA_OK
    b.same()
