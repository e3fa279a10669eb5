"""GPU: latent attention of drafted trees over the paged cache against the plain 64-bit form.

Tolerance, element by element: a softmax weight is rounded to bf16 (half a step, 2^-8 of its
value) and the normaliser sums the rounded weights, so z moves by at most 2^-8 (sum p|c| + |z|);
the score, an fp32 sum of 576 products, scaled and shifted (eight more roundings), is good to
584 * 2^-24 * scale * sum|q c|, a relative change of its weight that enters the sum and the
normaliser; a bf16 z adds its own 2^-8 |z|.  Second-order terms are covered by the factor 1.02."""
import numpy as np
import pytest
import torch

import oracle
from hybrid_linear_attention_gb300 import kda
from tests import _gpu
from tests import _tree_ref as ref

pytestmark = pytest.mark.gpu


class Case:
    """A paged batch; rows behind the drafted nodes and unused pages hold NaN."""

    def __init__(self, lengths, counts, *, H=64, page=64, seed=0, q_std=1.0, mask="tree", spare=2):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lengths, self.counts, self.H, self.page = lengths, counts, H, page
        self.cu = [0] + [int(x) for x in np.cumsum(counts)]
        total = self.cu[-1]
        self.q = (torch.randn(total, H, 576, generator=g) * q_std).to(torch.bfloat16)
        needs = [-(-(n + w) // page) for n, w in zip(lengths, counts)]
        n_pages = sum(needs) + spare
        order = [int(x) for x in rng.permutation(n_pages)]
        most = max(max(needs), 1) + 1
        self.table, at = [], 0
        for k in needs:
            self.table.append(order[at:at + k] + [-1] * (most - k))
            at += k
        self.pool = torch.full((n_pages, page, 576), float("nan"), dtype=torch.bfloat16)
        for b, (n, w) in enumerate(zip(lengths, counts)):
            rows = torch.randn(n + w, 576, generator=g).to(torch.bfloat16)
            for t0 in range(0, n + w, page):
                m = min(page, n + w - t0)
                self.pool[self.table[b][t0 // page], :m] = rows[t0:t0 + m]
        self.parents = [ref.random_parents(rng, w) for w in counts]
        if mask == "tree":
            self.mask = [m for p in self.parents for m in ref.masks(p)]
        elif mask == "random":
            self.mask = [int(x) for x in rng.integers(-2**63, 2**63, total, dtype=np.int64)]
        elif mask == "none":
            self.mask = [0] * total
        else:
            self.mask = None

    def run(self, z_dtype=torch.bfloat16, fill=7.0, stream=None):
        _gpu.lib()
        total, n = self.cu[-1], len(self.counts)
        z = torch.full((total, self.H, 512), fill, dtype=z_dtype, device="cuda")
        ws = torch.empty(kda.mla_tree_workspace_size(n, total, self.H), dtype=torch.uint8, device="cuda")
        mask = None if self.mask is None else torch.tensor(self.mask, dtype=torch.int64, device="cuda")
        kda.mla_tree_latent(self.q.cuda(), self.pool.cuda(), ref.i32(self.table), ref.i32(self.lengths),
                            ref.i32(self.cu), z, mask=mask, workspace=ws, stream=stream)
        torch.cuda.synchronize()
        return z.double().cpu().numpy()

    def expect(self):
        return ref.tree_attention(self.q, torch.nan_to_num(self.pool, nan=0.0), self.table, self.lengths, self.cu,
                                  self.mask, kda.MLA_SCALE)

    def check(self, z, z_dtype=torch.bfloat16):
        want, unit, size = self.expect()
        e = 2.0**-8 + 584 * 2.0**-24 * size
        tol = 1.02 * (e * (unit + np.abs(want)) + (2.0**-8 * np.abs(want) if z_dtype == torch.bfloat16 else 0))
        off = np.abs(z - want)
        assert np.isfinite(z).all()
        worst = np.unravel_index(np.argmax(off - tol), off.shape)
        assert (off <= tol + 1e-30).all(), f"at {worst}: {z[worst]} for {want[worst]}, allowed {tol[worst]:.3g}"


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H", [1, 16, 64, 96, 128])
def test_ragged_trees(page, H):
    """Lengths around tile and page edges, from no cached position on; one to nine nodes."""
    case = Case([0, 1, 15, 63, 120, 127, 128, 255, 300], [3, 1, 2, 9, 8, 1, 5, 4, 2], H=H, page=page, seed=page + H)
    case.check(case.run())
    kda.kda_check_device_error()


@pytest.mark.parametrize("z_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("length", [0, 1, 191, 192, 193, 247, 248, 249, 255, 256, 257, 511, 513])
def test_tile_edges(length, z_dtype):
    """The drafted nodes end before, on and behind a tile's edge."""
    case = Case([length], [8], seed=900 + length)
    case.check(case.run(z_dtype), z_dtype)


@pytest.mark.parametrize("w", [1, 2, 3, 33, 63, 64])
def test_node_counts(w):
    """One node (the decode step over pages) up to 64 (bit 63 of the mask)."""
    case = Case([130, 70], [w, 64], seed=1000 + w, H=16)
    case.check(case.run())


@pytest.mark.parametrize("q_std", [0.01, 4.0, 12.0])
def test_flat_and_peaked_scores(q_std):
    """Running maxima that jump between tiles: the largest score is in a different place per row."""
    case = Case([1500, 700], [4, 2], seed=77, q_std=q_std)
    case.check(case.run())


def test_rising_scores_rescale():
    """Scores that grow along the cache by hundreds, so the reference point has to move often."""
    case = Case([1400], [2], seed=78)
    for t in range(1400):
        case.pool[case.table[0][t // 64], t % 64, 575] = t / 4.0
    case.q[:, :, 575] = 8.0
    case.check(case.run())


@pytest.mark.parametrize("mask", ["random", "none", None])
def test_other_masks(mask):
    """Any bit pattern (bits past the last node are ignored), no drafted node visible, a chain."""
    case = Case([0, 40, 0, 300], [5, 7, 64, 3], H=16, mask=mask, seed=88)
    case.check(case.run())
    if mask == "none":
        z = case.run()
        assert not z[0:5].any() and not z[12:76].any()  # nothing visible: zero


def test_split_long_contexts():
    """Few sequences, long caches: the positions are spread over the device and merged."""
    case = Case([9000, 3, 5000], [1, 2, 6], seed=91)
    case.check(case.run())
    case.check(case.run(torch.float32), torch.float32)


@pytest.mark.parametrize("w", [2, 11])
@pytest.mark.parametrize("length", [500, 760, 1100, 1900, 4300, 21000])
def test_merges_of_few_and_many_parts(length, w):
    """A sequence alone is cut into as many parts as it has tiles, up to one a worker."""
    case = Case([length], [w], H=16, seed=150 + w)
    case.check(case.run())


def test_many_short_sequences():
    rng = np.random.default_rng(5)
    case = Case([int(x) for x in rng.integers(0, 90, 300)], [int(x) for x in rng.integers(0, 4, 300)], H=16, page=16,
                seed=92)
    case.check(case.run())


def test_many_sequences_with_odd_node_counts():
    """Row tiles of one CTA's rows between full ones, several sequences in every cluster's run."""
    rng = np.random.default_rng(6)
    case = Case([int(x) for x in rng.integers(0, 700, 240)], [int(x) for x in rng.integers(1, 5, 240)], seed=192)
    for _ in range(3):
        case.check(case.run())
    kda.kda_check_device_error()


def test_same_bits_every_time():
    case = Case([3000, 200], [4, 9], seed=93)
    a, b = case.run(), case.run()
    assert np.array_equal(a, b)


def test_nonfinite_drafted_rows_reach_only_the_nodes_that_see_them():
    case = Case([100, 250], [6, 6], seed=94)
    for b in range(2):
        for j, bad in ((4, float("nan")), (5, float("inf"))):
            t = case.lengths[b] + j
            case.pool[case.table[b][t // 64], t % 64, 10:300] = bad
            case.q[:, :, 10:300] = case.q[:, :, 10:300].abs()  # inf scores, not inf - inf alone
    case.mask = [0b1, 0b11, 0b101, 0b1001, 0b10001, 0b100001] * 2
    want = case.expect()[0]
    z = case.run()
    for b in range(2):
        assert np.isfinite(z[6 * b:6 * b + 4]).all() and not np.isfinite(z[6 * b + 4:6 * b + 6]).all(-1).any()
    good = np.array([0, 1, 2, 3, 6, 7, 8, 9])
    assert np.abs(z[good] - want[good]).max() <= 2.0**-6 * np.abs(want[good]).max()


def test_bad_lengths_pages_and_offsets_are_reported():
    case = Case([100, 100, 70, 100], [2, 2, 2, 2], seed=95)
    want = case.expect()[0]
    case.lengths[1] = -5
    case.lengths[3] = 10**6
    case.table[2][1] = 10**6  # positions 64.. of sequence 2 cannot be seen
    z = case.run()
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX
    assert not z[2:4].any() and not z[6:8].any()
    assert np.abs(z[:2] - want[:2]).max() <= 2.0**-6 * np.abs(want[:2]).max()
    case.table[2][1] = -1
    short = Case([64], [1], seed=1)
    short.q, short.pool, short.table, short.mask = case.q[4:6], case.pool, [case.table[2]], [0, 0]
    short.cu, short.counts, short.lengths = [0, 2], [2], [64]
    want = short.expect()[0]
    assert np.abs(z[4:6] - want).max() <= 2.0**-6 * np.abs(want).max()
    case = Case([10, 10], [2, 2], seed=96)
    case.cu = [0, 2, 9]
    case.cu[-1] = 4
    good = case.run()
    _gpu.lib()
    z = torch.full((4, 64, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kda.mla_tree_workspace_size(2, 4, 64), dtype=torch.uint8, device="cuda")
    kda.mla_tree_latent(case.q.cuda(), case.pool.cuda(), ref.i32(case.table), ref.i32(case.lengths), ref.i32([0, 2, 9]),
                        z, workspace=ws, mask=torch.tensor(case.mask, dtype=torch.int64, device="cuda"))
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_SEQLENS
    z = z.double().cpu().numpy()
    assert np.array_equal(z[:2], good[:2]) and (z[2:] == 7.0).all()


def test_rows_of_no_sequence_stay():
    """Padding rows in front of nothing: the batch's buffers are longer than its sequences."""
    case = Case([50, 20], [3, 2], seed=97)
    case.q = torch.cat([case.q, case.q[:4]])
    _gpu.lib()
    z = torch.full((9, 64, 512), 7.0, device="cuda")
    ws = torch.empty(kda.mla_tree_workspace_size(2, 9, 64), dtype=torch.uint8, device="cuda")
    mask = torch.tensor(case.mask + [0] * 4, dtype=torch.int64, device="cuda")
    kda.mla_tree_latent(case.q.cuda(), case.pool.cuda(), ref.i32(case.table), ref.i32(case.lengths), ref.i32(case.cu), z,
                        mask=mask, workspace=ws)
    kda.kda_check_device_error()
    z = z.double().cpu().numpy()
    assert (z[5:] == 7.0).all()
    case.q = case.q[:5]
    case.check(z[:5], torch.float32)


def test_captured_and_replayed_with_new_lengths_beside_another_stream():
    """A graph replayed after its inputs changed, while another call runs on a second stream with
    a workspace of its own."""
    _gpu.lib()
    a, b = Case([700, 90], [4, 3], seed=98), Case([300, 1200], [4, 3], seed=99)
    most = max(len(r) for r in a.table + b.table)
    pages = max(a.pool.shape[0], b.pool.shape[0])
    pad = lambda c: [r + [-1] * (most - len(r)) for r in c.table]  # noqa: E731
    pool = torch.full((pages, 64, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    q, z = a.q.cuda(), torch.full((7, 64, 512), 7.0, device="cuda")
    table, lengths, cu = ref.i32(pad(a)), ref.i32(a.lengths), ref.i32(a.cu)
    mask = torch.tensor(a.mask, dtype=torch.int64, device="cuda")
    size = kda.mla_tree_workspace_size(2, 7, 64)
    ws, ws2 = (torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    pool[:a.pool.shape[0]] = a.pool.cuda()
    call = lambda out, w: kda.mla_tree_latent(q, pool, table, lengths, cu, out, mask=mask, workspace=w)  # noqa: E731
    call(z, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(z, ws)
    for case in (b, a):
        pool[:case.pool.shape[0]] = case.pool.cuda()
        q.copy_(case.q)
        table.copy_(ref.i32(pad(case)))
        lengths.copy_(ref.i32(case.lengths))
        mask.copy_(torch.tensor(case.mask, dtype=torch.int64))
        other = torch.full((7, 64, 512), 7.0, device="cuda")
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            call(other, ws2)
        graph.replay()
        torch.cuda.synchronize()
        case.check(z.double().cpu().numpy(), torch.float32)
        assert torch.equal(z, other)


@pytest.mark.parametrize("nodes", [1, 5])
def test_tree_decode_matches_the_one_token_step(nodes):
    """The whole step: a chain's node i equals mla_decode over the cache that ends with it (the
    same operands, roundings and normaliser; both are within the bound of the 64-bit form)."""
    _gpu.lib()
    lengths, L = [65, 130, 7], 192
    g = torch.Generator().manual_seed(31 + nodes)
    bf = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    n, total = len(lengths), nodes * len(lengths)
    cache = bf(n, L, 576)
    pool = cache.view(n * L // 64, 64, 576).clone()
    table = torch.arange(n * L // 64, dtype=torch.int32, device="cuda").view(n, -1).contiguous()
    m = dict(q_nope=bf(total, 64, 128), q_rope=bf(total, 64, 64), w_uk=bf(64, 128, 512, std=0.05),
             w_uv=bf(64, 128, 512, std=0.05), gate=bf(total, 64))
    q_cat = torch.empty((total, 64, 576), dtype=torch.bfloat16, device="cuda")
    z = torch.empty((total, 64, 512), device="cuda")
    out = torch.empty((total, 64, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kda.mla_tree_workspace_size(n, total), dtype=torch.uint8, device="cuda")
    kda.mla_tree_decode(m["q_nope"], m["q_rope"], m["w_uk"], m["w_uv"], pool, table, ref.i32(lengths),
                        ref.i32([nodes * i for i in range(n + 1)]), m["gate"], q_cat, z, out, workspace=ws)
    kda.kda_check_device_error()
    for i in range(nodes):
        pick = torch.arange(n, device="cuda") * nodes + i
        one = {k: v[pick].contiguous() if k in ("q_nope", "q_rope", "gate") else v for k, v in m.items()}
        qc = torch.empty((n, 64, 576), dtype=torch.bfloat16, device="cuda")
        z1 = torch.empty((n, 64, 512), device="cuda")
        o1 = torch.empty((n, 64, 128), dtype=torch.bfloat16, device="cuda")
        kda.mla_decode(one["q_nope"], one["q_rope"], one["w_uk"], one["w_uv"], cache, ref.i32([x + i + 1 for x in lengths]),
                       one["gate"], qc, z1, o1)
        assert torch.equal(qc, q_cat[pick])
        rms = float(o1.double().square().mean().sqrt())
        # each within 1e-2 of the RMS of the same function, and half a bf16 step (2^-8) of its value
        off = (out[pick].double() - o1.double()).abs() - 2.0**-8 * (out[pick].double().abs() + o1.double().abs())
        assert float(off.max()) <= 2e-2 * rms
    qa = oracle.mla_absorb(m["q_nope"].cpu(), m["q_rope"].cpu(), m["w_uk"].cpu())
    assert np.abs(q_cat.double().cpu().numpy() - qa).max() <= 2.0**-7 * np.abs(qa).max()


def test_masks_from_parents():
    _gpu.lib()
    rng = np.random.default_rng(3)
    counts = [1, 0, 64, 7, 33]
    parents = [ref.random_parents(rng, w) for w in counts]
    parents[2] = list(range(-1, 63))  # a chain of 64: all bits of the last word
    cu = [0] + [int(x) for x in np.cumsum(counts)]
    mask = torch.full((cu[-1],), 5, dtype=torch.int64, device="cuda")
    kda.mla_tree_mask(ref.i32([p for q in parents for p in q]), ref.i32(cu), mask)
    kda.kda_check_device_error()
    assert mask.tolist() == [m for p in parents for m in ref.masks(p)]
    bad = [p for q in parents for p in q]
    bad[1 + 3] = 60  # node 3 of the chain names a later node: a root
    kda.mla_tree_mask(ref.i32(bad), ref.i32(cu), mask)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX and mask.tolist()[4] == 8


@pytest.mark.parametrize("bad", [-2, -1, -2**31, 10**6])
@pytest.mark.parametrize("page,where", [(16, 3), (64, 0), (64, 1), (256, 0)])
def test_every_table_entry_that_names_no_page_is_reported(bad, page, where):
    """Whatever the value: its positions are invisible and the call says so."""
    case = Case([200, 130], [2, 3], H=4, page=page, seed=110)
    want = case.expect()[0]
    case.table[1][where] = bad
    z = case.run(torch.float32)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX
    assert np.abs(z[:2] - want[:2]).max() <= 2.0**-6 * np.abs(want[:2]).max()
    # sequence 1 without the page: its other positions as a shorter cache
    hidden = range(where * page, (where + 1) * page)
    keys = {t: torch.nan_to_num(case.pool[case.table[1][t // page], t % page], nan=0.0).double().numpy()
            for t in range(133) if t not in hidden}
    for i in range(3):
        seen = [t for t in keys if t < 130 or (case.mask[2 + i] >> (t - 130)) & 1]
        if not seen:
            assert not z[2 + i].any()
            continue
        k = np.stack([keys[t] for t in seen])
        s = case.q[2 + i].double().numpy() @ k.T * kda.MLA_SCALE
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        unit, one = p @ np.abs(k[:, :512]), p @ k[:, :512]
        size = (np.abs(case.q[2 + i].double().numpy()) @ np.abs(k).T).max(-1, keepdims=True) * kda.MLA_SCALE
        assert (np.abs(z[2 + i] - one) <= 1.02 * (2.0**-8 + 584 * 2.0**-24 * size) * (unit + np.abs(one))).all()


def test_entries_behind_the_last_position_are_not_read():
    """The table past the pages in use may hold anything, and nothing is reported."""
    case = Case([200, 130, 0], [2, 3, 1], H=4, page=16, seed=111)
    for row in case.table:
        row[:] = [p if p >= 0 else (-2, 10**6, -1)[i % 3] for i, p in enumerate(row)]
    case.check(case.run())
    kda.kda_check_device_error()
