"""GPU: block keys, scores and selection, and attention over the selection, against the plain
64-bit forms.  Keys: an fp32 sum over the page (2^-24 of sum|x| per row) and a bf16 rounding (2^-8 of
the mean); scores: derived in _long_ref.py; selections from given scores are exact."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_gb300 import kda
from tests import _gpu
from tests import _long_ref as long
from tests import _tree_ref as ref
from tests.test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layers", [1, 3])
def test_block_keys(page, layers):
    _gpu.lib()
    g, rng = torch.Generator().manual_seed(page), np.random.default_rng(page)
    lengths = [0, 1, page - 1, page, page + 1, 3 * page, 5 * page + 7, 2 * page]
    before = [0, 0, page - 2, page - 1, page, page - 1, 0, 3 * page]
    n_pages = 20
    table = [[int(x) for x in rng.permutation(n_pages)[:6]] for _ in lengths]
    pool = torch.randn(layers, n_pages, page, 576, generator=g).to(torch.bfloat16)
    keys = torch.full((layers, n_pages, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.mla_block_keys(pool.cuda(), ref.i32(table), ref.i32(before), ref.i32(lengths), keys)
    kda.kda_check_device_error()
    done = {table[n][j] for n in range(len(lengths)) for j in range(before[n] // page, lengths[n] // page)}
    got, x = keys.double().cpu(), pool.double()
    for p in range(n_pages):
        if p not in done:
            assert (got[:, p] == 7.0).all()
            continue
        mean, size = x[:, p].mean(1), x[:, p].abs().mean(1)
        assert ((got[:, p] - mean).abs() <= 1.01 * (2.0**-8 * mean.abs() + page * 2.0**-24 * size)).all()


def test_block_keys_of_many_sequences_and_bad_ones():
    _gpu.lib()
    n, page, n_pages = 700, 16, 1500
    g, rng = torch.Generator().manual_seed(1), np.random.default_rng(1)
    lengths = [int(x) for x in rng.integers(0, 33, n)]
    order, table = iter(int(x) for x in rng.permutation(n_pages)), []
    for _ in range(n):
        table.append([next(order), next(order), -1])
    pool = torch.randn(1, n_pages, page, 576, generator=g).to(torch.bfloat16)
    want = pool.double().mean(2)
    lengths[5], lengths[6], lengths[7], table[7][0] = -1, 10**6, 20, n_pages
    keys = torch.full((1, n_pages, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.mla_block_keys(pool.cuda(), ref.i32(table), ref.i32([0] * n), ref.i32(lengths), keys)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX
    done = {table[i][j] for i in range(n) if i not in (5, 6, 7) for j in range(lengths[i] // page)}
    got = keys.double().cpu()
    for p in range(n_pages):
        if p in done:
            assert ((got[0, p] - want[0, p]).abs() <= 2.0**-7 * want[0, p].abs() + 2.0**-18).all()
        else:
            assert (got[0, p] == 7.0).all()


def block_batch(lengths, counts, *, H=64, page=64, seed=0, q_std=1.0, extra=2):
    """q, keys, table, cu of a batch of which only the keys exist."""
    g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    cu = [0] + [int(x) for x in np.cumsum(counts)]
    needs = [-(-(n + w) // page) for n, w in zip(lengths, counts)]
    n_pages = sum(needs) + 3
    order = [int(x) for x in rng.permutation(n_pages)]
    most = max(max(needs), 1) + extra
    table, at = [], 0
    for k in needs:
        table.append(order[at:at + k] + [-1] * (most - k))
        at += k
    q = (torch.randn(cu[-1], H, 576, generator=g) * q_std).to(torch.bfloat16)
    keys = torch.randn(n_pages, 576, generator=g).to(torch.bfloat16)
    return q, keys, table, cu


def run_scores(q, keys, page, table, lengths, cu, width=None):
    _gpu.lib()
    total, H = q.shape[:2]
    s = torch.full((len(lengths), width or len(table[0])), 7.0, device="cuda")
    ws = torch.empty(kda.mla_block_scores_workspace_size(total, H, len(table[0])), dtype=torch.uint8, device="cuda")
    ws.fill_(255)  # NaN: nothing of it is read before it is written
    kda.mla_block_scores(q.cuda(), keys.cuda(), page, ref.i32(table), ref.i32(lengths), ref.i32(cu), s, workspace=ws)
    torch.cuda.synchronize()
    return s


def check_scores(s, q, keys, page, table, lengths, cu):
    for n, (want, tol) in enumerate(long.block_scores(q, keys, table, lengths, cu, page, kda.MLA_SCALE)):
        got = s[n].double().cpu().numpy()
        assert (got[len(want):] == 7.0).all()
        off = np.abs(got[:len(want)] - want)
        assert (off <= tol).all(), f"sequence {n}: {(off - tol).max()}"


@pytest.mark.parametrize("H", [1, 16, 64, 96, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_scores_of_ragged_batches(H, page):
    lengths = [0, 1, page - 1, page, 2 * page + 3, 31 * page, 128 * page, 129 * page - 1, 257 * page, 600 * page]
    counts = [1, 2, 1, 3, 1, 4, 2, 1, 3, 0]
    b = block_batch(lengths, counts, H=H, page=page, seed=H)
    check_scores(run_scores(b[0], b[1], page, b[2], lengths, b[3]), b[0], b[1], page, b[2], lengths, b[3])
    kda.kda_check_device_error()


@pytest.mark.parametrize("q_std", [0.01, 6.0, 20.0])
def test_scores_flat_and_peaked(q_std):
    lengths, counts = [5000, 40000], [1, 5]
    b = block_batch(lengths, counts, seed=3, q_std=q_std)
    check_scores(run_scores(b[0], b[1], 64, b[2], lengths, b[3], width=700), b[0], b[1], 64, b[2], lengths, b[3])


def test_scores_of_wide_trees_and_many_sequences():
    rng = np.random.default_rng(4)
    lengths = [int(x) for x in rng.integers(0, 3000, 400)]
    counts = [int(x) for x in rng.choice([0, 1, 2, 64], 400, p=[0.1, 0.7, 0.17, 0.03])]
    b = block_batch(lengths, counts, H=8, page=16, seed=4)
    check_scores(run_scores(b[0], b[1], 16, b[2], lengths, b[3]), b[0], b[1], 16, b[2], lengths, b[3])


def test_scores_of_one_row_and_of_a_thousand_sequences():
    b = block_batch([700], [1], H=1, page=16, seed=5)
    check_scores(run_scores(b[0], b[1], 16, b[2], [700], b[3]), b[0], b[1], 16, b[2], [700], b[3])
    rng = np.random.default_rng(5)
    lengths = [int(x) for x in rng.integers(0, 200, 1000)]
    b = block_batch(lengths, [1] * 1000, H=3, page=16, seed=5)
    check_scores(run_scores(b[0], b[1], 16, b[2], lengths, b[3]), b[0], b[1], 16, b[2], lengths, b[3])


def test_scores_report_what_is_bad():
    lengths, counts = [640, 640, 640], [1, 1, 1]
    q, keys, table, cu = block_batch(lengths, counts, seed=6)
    want = run_scores(q, keys, 64, table, lengths, cu)
    table[1][3] = -1
    got = run_scores(q, keys, 64, table, [640, 640, -2], cu)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX
    assert torch.equal(got[0], want[0]) and got[1, 3] == 0 and (got[2] == 7.0).all()
    left = [j for j in range(10) if j != 3]
    p = torch.softmax(q[1].double() @ keys[[table[1][j] for j in left]].double().T * kda.MLA_SCALE, -1).sum(0)
    assert ((got[1, left].double().cpu() - p).abs() <= 1e-4 * p).all()
    got = run_scores(q, keys, 64, table, lengths, [0, 1, 2, 9])
    with pytest.raises(kda.KdaError):
        kda.kda_check_device_error()
    assert torch.equal(got[0], want[0]) and (got[2] == 7.0).all()


def run_select(scores, page, table, lengths, cu, *, blocks, first=0, recent=0, width=None):
    _gpu.lib()
    most = max(b - a for a, b in zip(cu, cu[1:])) if len(cu) > 1 else 0
    width = width or blocks + (2 * (page - 1) + most) // page + 1
    sel = torch.full((len(lengths), width), 77, dtype=torch.int32, device="cuda")
    cut = torch.full((len(lengths),), 77, dtype=torch.int32, device="cuda")
    kda.mla_block_select(scores.cuda(), page, ref.i32(table), ref.i32(lengths), ref.i32(cu), sel, cut, blocks=blocks,
                         total_nodes=cu[-1], first=first, recent=recent)
    torch.cuda.synchronize()
    return sel, cut


def want_select(scores, page, table, lengths, cu, n, blocks, first, recent):
    full, w = lengths[n] // page, cu[n + 1] - cu[n]
    if w == 0:
        return [], 0
    taken = long.choose(scores[n].tolist(), full, first, recent, blocks)
    tail = table[n][full:-(-(lengths[n] + w) // page)]
    return [table[n][j] for j in taken] + tail, len(taken) * page + lengths[n] % page


@pytest.mark.parametrize("kind", ["random", "ties"])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_select(page, kind):
    lengths = [0, 1, page - 1, page, 3 * page, 9 * page, 9 * page + 5, 10 * page, 11 * page + 1, 300 * page, 2000 * page - 1, 40 * page]
    counts = [1, 2, 3, 1, 2, 64, 1, 1, 5, 1, 4, 0]
    _, _, table, cu = block_batch(lengths, counts, H=1, page=page, seed=7)
    g = torch.Generator().manual_seed(8)
    s = torch.rand(len(lengths), len(table[0]) + 3, generator=g)
    if kind == "ties":
        s = (s * 3).floor()
    for blocks, first, recent in ((1, 0, 0), (9, 0, 0), (9, 1, 2), (9, 9, 0), (9, 0, 9), (64, 2, 8), (5000, 1, 1)):
        sel, cut = run_select(s, page, table, lengths, cu, blocks=blocks, first=first, recent=recent)
        for n in range(len(lengths)):
            want, length = want_select(s, page, table, lengths, cu, n, blocks, first, recent)
            assert sel[n].tolist() == want + [-1] * (sel.shape[1] - len(want)), (n, blocks)
            assert int(cut[n]) == length
    kda.kda_check_device_error()


def test_select_of_long_contexts_by_clusters():
    lengths, counts = [16 * 100000, 16 * 70001 + 3], [1, 2]
    table = [[int(x) for x in np.random.default_rng(n).permutation(1 << 20)[:100003]] for n in range(2)]
    s = torch.randint(0, 1000, (2, 100003), generator=torch.Generator().manual_seed(9)).float()
    sel, cut = run_select(s, 16, table, lengths, [0, 1, 3], blocks=3000, first=1, recent=4)
    for n in range(2):
        want, length = want_select(s, 16, table, lengths, [0, 1, 3], n, 3000, 1, 4)
        assert sel[n].tolist() == want + [-1] * (sel.shape[1] - len(want)) and int(cut[n]) == length


def test_select_reports_what_is_bad():
    lengths = [1000, -1, 1000, 10**7, 1000]
    _, _, table, cu = block_batch([1000] * 5, [1] * 5, H=1, page=16, seed=7)
    s = torch.rand(5, len(table[0]))
    cu = [0, 1, 2, 3, 4, 90]
    sel, cut = run_select(s, 16, table, lengths, cu, blocks=4, width=5)
    with pytest.raises(kda.KdaError):
        kda.kda_check_device_error()
    assert cut.tolist() == [4 * 16 + 8, 0, 4 * 16 + 8, 0, 0]
    for n in (1, 3, 4):
        assert sel[n].tolist() == [-1] * 5
    lengths = [1000, 1008]
    sel, cut = run_select(s[:2], 16, table, [1000, 1007], [0, 1, 3], blocks=4, width=5)  # the second needs six entries
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX
    assert cut.tolist() == [4 * 16 + 8, 0] and sel[1].tolist() == [-1] * 5


class Sparse(Case):
    """A paged batch with its pages' keys."""

    def step(self, blocks, first=0, recent=0, z_dtype=torch.float32):
        _gpu.lib()
        n, total = len(self.counts), self.cu[-1]
        pool = torch.nan_to_num(self.pool, nan=0.0).cuda()
        d = dict(keys=torch.full((pool.shape[0], 576), float("nan"), dtype=torch.bfloat16, device="cuda"))
        kda.mla_block_keys(pool[None], ref.i32(self.table), ref.i32([0] * n), ref.i32(self.lengths), d["keys"][None])
        d["scores"] = torch.zeros(n, len(self.table[0]), device="cuda")
        width = blocks + (2 * (self.page - 1) + max(self.counts)) // self.page
        d["sel"] = torch.full((n, width), 77, dtype=torch.int32, device="cuda")
        d["cut"] = torch.full((n,), 77, dtype=torch.int32, device="cuda")
        d["z"] = torch.full((total, self.H, 512), 7.0, dtype=z_dtype, device="cuda")
        d["ws"] = torch.empty(kda.mla_sparse_workspace_size(n, total, self.H, len(self.table[0])), dtype=torch.uint8,
                              device="cuda")
        d["mask"] = None if self.mask is None else torch.tensor(self.mask, dtype=torch.int64, device="cuda")
        kda.mla_sparse_latent(self.q.cuda(), pool, d["keys"], ref.i32(self.table), ref.i32(self.lengths), ref.i32(self.cu),
                              d["scores"], d["sel"], d["cut"], d["z"], blocks=blocks, first=first, recent=recent,
                              mask=d["mask"], workspace=d["ws"])
        torch.cuda.synchronize()
        return d


@pytest.mark.parametrize("H,page", [(16, 16), (64, 64), (128, 32)])
def test_a_sparse_step(H, page):
    """The call's parts one by one: scores of the keys, the selection from those scores, the attention
    over the selected pages as over a shorter cache."""
    case = Sparse([0, 5, page, 700, 1500, 90], [2, 1, 3, 5, 1, 4], H=H, page=page, seed=H)
    d = case.step(6, first=1, recent=2)
    kda.kda_check_device_error()
    scores = d["scores"].cpu()
    full = [x // page for x in case.lengths]
    padded = d["scores"].clone()
    for n, f in enumerate(full):
        padded[n, f:] = 7.0
    check_scores(padded, case.q, d["keys"].cpu(), page, case.table, case.lengths, case.cu)
    for n in range(len(full)):
        want, length = want_select(scores, page, case.table, case.lengths, case.cu, n, 6, 1, 2)
        assert d["sel"][n].tolist() == want + [-1] * (d["sel"].shape[1] - len(want)) and int(d["cut"][n]) == length
    short = Case([1], [1], seed=1)
    short.q, short.pool, short.mask, short.H = case.q, case.pool, case.mask, H
    short.cu, short.counts, short.page = case.cu, case.counts, page
    short.table, short.lengths = d["sel"].tolist(), d["cut"].tolist()
    short.check(d["z"].double().cpu().numpy(), torch.float32)


def test_all_blocks_is_the_whole_attention():
    case = Sparse([0, 700, 3000, 64], [2, 1, 3, 1], seed=21)
    d = case.step(60)
    assert torch.equal(d["z"].cpu().double(), torch.tensor(case.run(torch.float32)))


def test_sparse_decode_is_its_parts():
    _gpu.lib()
    case = Sparse([1000, 3000, 130], [2, 1, 3], page=32, seed=22, mask=None)
    g = torch.Generator().manual_seed(5)
    bf = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    total, n = 6, 3
    m = (bf(total, 64, 128), bf(total, 64, 64), bf(64, 128, 512, std=0.05), bf(64, 128, 512, std=0.05))
    gate = bf(total, 64)
    pool = torch.nan_to_num(case.pool, nan=0.0).cuda()
    keys = torch.zeros(pool.shape[0], 576, dtype=torch.bfloat16, device="cuda")
    table, lengths, cu = ref.i32(case.table), ref.i32(case.lengths), ref.i32(case.cu)
    kda.mla_block_keys(pool[None], table, ref.i32([0] * n), lengths, keys[None])
    scores = torch.zeros(n, table.shape[1], device="cuda")
    sel, cut = torch.zeros(n, 12, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    ws = torch.empty(kda.mla_sparse_workspace_size(n, total, 64, table.shape[1]), dtype=torch.uint8, device="cuda")
    q = [torch.empty((total, 64, 576), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    z = [torch.empty((total, 64, 512), device="cuda") for _ in range(2)]
    out = [torch.empty((total, 64, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kda.mla_sparse_decode(*m, pool, keys, table, lengths, cu, gate, scores, sel, cut, q[0], z[0], out[0], blocks=9, recent=1,
                          workspace=ws)
    kda.mla_tree_decode(*m, pool, sel, cut, cu, gate, q[1], z[1], out[1], workspace=ws)
    kda.kda_check_device_error()
    assert torch.equal(q[0], q[1]) and torch.equal(z[0], z[1]) and torch.equal(out[0], out[1])
    s2 = torch.zeros_like(scores)
    kda.mla_block_scores(q[0], keys, 32, table, lengths, cu, s2, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(scores, s2)
