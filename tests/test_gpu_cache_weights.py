"""GPU: the log-sums of the tree attention and the attention that cached positions receive, against
the plain 64-bit forms.  Tolerances: an fp32 score is a sum of 576 products, scaled and shifted
(584 * 2^-24 of scale * sum|q c|); the rest is derived beside the forms in _long_ref.py."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_gb300 import kda
from tests import _gpu
from tests import _long_ref as long
from tests import _tree_ref as ref
from tests.test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu


def clean(case):
    return torch.nan_to_num(case.pool, nan=0.0)


def run_lse(case, z_dtype=torch.float32):
    _gpu.lib()
    total, n = case.cu[-1], len(case.counts)
    z = torch.full((total, case.H, 512), 7.0, dtype=z_dtype, device="cuda")
    lse = torch.full((total, case.H), 7.0, device="cuda")
    ws = torch.empty(kda.mla_tree_workspace_size(n, total, case.H), dtype=torch.uint8, device="cuda")
    mask = None if case.mask is None else torch.tensor(case.mask, dtype=torch.int64, device="cuda")
    kda.mla_tree_latent_lse(case.q.cuda(), case.pool.cuda(), ref.i32(case.table), ref.i32(case.lengths), ref.i32(case.cu),
                            z, lse, mask=mask, workspace=ws)
    torch.cuda.synchronize()
    return z, lse


def check_lse(case, lse):
    want, size = long.lse(case.q, clean(case), case.table, case.lengths, case.cu, case.mask, kda.MLA_SCALE)
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isinf(want), np.isinf(got)) and not np.isnan(got).any()
    assert (got[np.isinf(want)] < 0).all()
    there = np.isfinite(want)
    most = max(n + w for n, w in zip(case.lengths, case.counts))
    # relative error of the sum (each weight's, 2^-21 for the powers, the additions), and of the logarithm
    tol = 1.02 * (584 * 2.0**-24 * size + (most + 16) * 2.0**-24 + 2.0**-21 * (1 + np.abs(np.where(there, want, 0))))
    assert (np.abs(got[there] - want[there]) <= tol[there]).all()


def run_weights(case, lse, *, node_weight=None, start=None, width=None, mask="own", stream=None):
    _gpu.lib()
    n = len(case.counts)
    width = width or len(case.table[0]) * case.page
    w = torch.full((n, width), 0.5, device="cuda") if start is None else start
    m = case.mask if mask == "own" else mask
    kda.mla_cache_weights(case.q.cuda(), case.pool.cuda(), ref.i32(case.table), ref.i32(case.lengths), ref.i32(case.cu),
                          lse.cuda(), w, mask=None if m is None else torch.tensor(m, dtype=torch.int64, device="cuda"),
                          node_weight=None if node_weight is None else torch.tensor(node_weight, device="cuda"),
                          stream=stream)
    torch.cuda.synchronize()
    return w


def true_lse(case):
    return torch.tensor(long.lse(case.q, clean(case), case.table, case.lengths, case.cu, case.mask, kda.MLA_SCALE)[0]).float()


def check_weights(case, got, lse, *, node_weight=None, before=0.5):
    want, tol = long.weights(case.q, clean(case), case.table, case.lengths, case.cu, case.mask, node_weight,
                             lse.double().numpy(), kda.MLA_SCALE, got.shape[1])
    got = got.double().cpu().numpy()
    off = np.abs(got - before - want)
    allowed = tol + 2.0**-24 * (np.abs(want) + 2 * abs(before))
    for n, (x, w) in enumerate(zip(case.lengths, case.counts)):
        end = x + w if w else 0
        assert (got[n, end:] == before).all()
    worst = np.unravel_index(np.argmax(off - allowed), off.shape)
    assert (off <= allowed).all(), f"at {worst}: {got[worst]} for {want[worst] + before}, allowed {allowed[worst]:.3g}"


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H", [1, 16, 64, 96, 128])
def test_ragged_trees(page, H):
    case = Case([0, 1, 15, 63, 120, 127, 128, 255, 300], [3, 1, 2, 9, 8, 1, 5, 4, 2], H=H, page=page, seed=page + H)
    z, lse = run_lse(case)
    check_lse(case, lse)
    assert np.array_equal(z.double().cpu().numpy(), case.run(torch.float32))  # the attention's bits stay
    given = true_lse(case)
    check_weights(case, run_weights(case, given), given)
    kda.kda_check_device_error()


@pytest.mark.parametrize("length", [0, 1, 127, 128, 129, 255, 256, 257, 511, 513])
def test_tile_edges(length):
    case = Case([length], [1], seed=900 + length)
    _, lse = run_lse(case, torch.bfloat16)
    check_lse(case, lse)
    given = true_lse(case)
    check_weights(case, run_weights(case, given), given)


@pytest.mark.parametrize("w,H", [(1, 64), (2, 64), (3, 64), (4, 64), (5, 64), (64, 1), (64, 2), (33, 64), (64, 128)])
def test_row_counts(w, H):
    """Resident rows up to 128, then chunks of 256, whole and odd."""
    case = Case([300, 40], [w, 1], H=H, seed=1000 + w)
    given = true_lse(case)
    check_weights(case, run_weights(case, given), given)


def test_resident_and_streamed_sequences_take_turns():
    rng = np.random.default_rng(8)
    counts = [int(x) for x in rng.choice([0, 1, 2, 3, 5, 9], 120)]
    case = Case([int(x) for x in rng.integers(0, 700, 120)], counts, seed=11)
    given = true_lse(case)
    for _ in range(3):
        check_weights(case, run_weights(case, given), given)
    kda.kda_check_device_error()


def test_more_sequences_than_threads():
    rng = np.random.default_rng(9)
    case = Case([int(x) for x in rng.integers(0, 60, 900)], [int(x) for x in rng.integers(0, 3, 900)], H=4, page=16, seed=12)
    given = true_lse(case)
    check_weights(case, run_weights(case, given), given)


@pytest.mark.parametrize("mask", ["random", "none", None])
def test_other_masks(mask):
    case = Case([0, 40, 0, 300], [5, 7, 64, 3], H=16, mask=mask, seed=88)
    _, lse = run_lse(case)
    check_lse(case, lse)
    given = true_lse(case)
    check_weights(case, run_weights(case, given), given)


def test_long_contexts_merge_their_parts():
    case = Case([9000, 3, 5000], [1, 2, 6], seed=91, H=16)
    _, lse = run_lse(case)
    check_lse(case, lse)
    given = true_lse(case)
    check_weights(case, run_weights(case, given), given)


@pytest.mark.parametrize("q_std", [0.01, 4.0, 12.0])
def test_flat_and_peaked_scores(q_std):
    case = Case([1500, 700], [4, 2], seed=77, q_std=q_std, H=16)
    _, lse = run_lse(case)
    check_lse(case, lse)
    given = true_lse(case)
    check_weights(case, run_weights(case, given), given)


def test_node_weights_and_rejected_nodes_of_any_content():
    """A node of weight 0 adds nothing though its query holds NaN; others by their weight."""
    case = Case([500, 90], [6, 3], H=64, seed=31)
    u = [1.0, 0.5, 0.0, -2.0, 0.0, 1.0, 0.0, 0.0, 0.25]
    given = true_lse(case)
    want = run_weights(case, given, node_weight=u)
    check_weights(case, want, given, node_weight=u)
    for i, x in enumerate(u):
        if x == 0:
            case.q[i] = float("nan")
            given[i] = float("nan")
    assert torch.equal(run_weights(case, given, node_weight=u), want)


def test_nonfinite_drafted_rows_reach_only_their_own_position():
    case = Case([100, 250], [6, 6], seed=94)
    case.mask = [0b1, 0b11, 0b101, 0b1001, 0b10001, 0b100001] * 2
    given = true_lse(case)
    want = run_weights(case, given)
    for b in range(2):
        for j, bad in ((4, float("nan")), (5, float("inf"))):
            t = case.lengths[b] + j
            case.pool[case.table[b][t // 64], t % 64, 10:300] = bad
    got = run_weights(case, given)
    for b in range(2):
        end = case.lengths[b] + 4
        assert torch.equal(got[b, :end], want[b, :end]) and torch.equal(got[b, end + 2:], want[b, end + 2:])


def test_bad_lengths_pages_and_offsets_are_reported():
    case = Case([100, 100, 70, 100], [2, 2, 2, 2], seed=95)
    given = true_lse(case)
    want = run_weights(case, given)
    case.lengths[1], case.lengths[3] = -5, 10**6
    case.table[2][1] = 10**6
    got = run_weights(case, given)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX
    assert torch.equal(got[0], want[0]) and (got[1] == 0.5).all() and (got[3] == 0.5).all()
    assert torch.equal(got[2, :64], want[2, :64]) and (got[2, 64:] == 0.5).all()
    case = Case([100, 100], [2, 2], seed=96)
    given = true_lse(case)
    want = run_weights(case, given)
    case.cu = [0, 2, 9]
    got = run_weights(case, given)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_SEQLENS
    assert torch.equal(got[0], want[0]) and (got[1] == 0.5).all()
    case.cu = [0, 2, 4]
    got = run_weights(case, given, width=101)  # sequence 0 and 1 have 102 positions
    with pytest.raises(kda.KdaError):
        kda.kda_check_device_error()
    assert (got == 0.5).all()


def test_it_adds_up_and_gives_the_same_bits():
    case = Case([3000, 200], [1, 1], seed=93)
    given = true_lse(case)
    a, b = run_weights(case, given), run_weights(case, given)
    assert torch.equal(a, b)
    run_weights(case, given, start=a)
    want, tol = long.weights(case.q, clean(case), case.table, case.lengths, case.cu, case.mask, None, given.double().numpy(),
                             kda.MLA_SCALE, a.shape[1])
    assert (np.abs(a.double().cpu().numpy() - 0.5 - 2 * want) <= 2 * tol + 2.0**-22).all()


def test_decode_with_lse_gives_the_same_bits():
    _gpu.lib()
    lengths, nodes = [65, 130, 7], 2
    g = torch.Generator().manual_seed(31)
    bf = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    n, total = 3, 6
    pool = bf(9, 64, 576)
    table = torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)
    m = (bf(total, 64, 128), bf(total, 64, 64), bf(64, 128, 512, std=0.05), bf(64, 128, 512, std=0.05))
    gate, cu = bf(total, 64), ref.i32([0, 2, 4, 6])
    q = [torch.empty((total, 64, 576), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    z = [torch.empty((total, 64, 512), device="cuda") for _ in range(3)]
    out = [torch.empty((total, 64, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lse = [torch.empty((total, 64), device="cuda") for _ in range(2)]
    ws = torch.empty(kda.mla_tree_workspace_size(n, total), dtype=torch.uint8, device="cuda")
    kda.mla_tree_decode(*m, pool, table, ref.i32(lengths), cu, gate, q[0], z[0], out[0], workspace=ws)
    kda.mla_tree_decode_lse(*m, pool, table, ref.i32(lengths), cu, gate, q[1], z[1], out[1], lse[0], workspace=ws)
    kda.mla_tree_latent_lse(q[1], pool, table, ref.i32(lengths), cu, z[2], lse[1], workspace=ws)
    kda.kda_check_device_error()
    assert torch.equal(q[0], q[1]) and torch.equal(z[0], z[1]) and torch.equal(out[0], out[1])
    assert torch.equal(lse[0], lse[1]) and torch.equal(z[1], z[2])


def test_all_nodes_rejected_is_no_work():
    case = Case([500, 90], [6, 3], H=64, seed=31)
    got = run_weights(case, true_lse(case), node_weight=[0.0, -0.0] * 4 + [0.0])
    kda.kda_check_device_error()
    assert (got == 0.5).all()


@pytest.mark.parametrize("H", [1, 5, 64, 100])
def test_chunks_without_a_node_that_counts(H):
    """Any pattern of weights over 64 nodes: chunks of 256 rows begin and end inside nodes."""
    case = Case([300], [64], H=H, seed=32)
    given = true_lse(case)
    for pattern in (0x1, 1 << 63, 0x00F0000000000F00, 0xAAAAAAAAAAAAAAAA):
        u = [float((pattern >> i) & 1) for i in range(64)]
        check_weights(case, run_weights(case, given, node_weight=u), given, node_weight=u)


def test_accepted_weights_follow_their_rows():
    _gpu.lib()
    rng = np.random.default_rng(40)
    counts = [64, 1, 9, 0, 33, 5, 4, 7]
    cu = [0] + [int(x) for x in np.cumsum(counts)]
    parents = [ref.random_parents(rng, w) for w in counts]
    accept = [63, -1, 5, -1, 20, 0, 3, 6]
    lengths = [100, 7, 0, 50, 190, 30, -1, 219]
    w = torch.rand(8, 224, generator=torch.Generator().manual_seed(2))
    want = w.clone()
    for n, (x, k) in enumerate(zip(lengths, counts)):
        if n in (6, 7):  # a length below 0, nodes past the row's end
            continue
        path = ref.path_to(parents[n], accept[n])
        want[n, x:x + k] = 0
        want[n, x:x + len(path)] = w[n, [x + j for j in path]]
    got = w.cuda()
    kda.mla_weights_accept(got, ref.i32(lengths), ref.i32(cu), ref.i32([p for q in parents for p in q]), ref.i32(accept))
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX
    assert torch.equal(got.cpu(), want)
    got = w.cuda()
    bad = list(accept)
    bad[0], bad[2] = 64, -2
    kda.mla_weights_accept(got[:3], ref.i32(lengths[:3]), ref.i32(cu[:3] + [1000]), ref.i32([-1] * cu[3]), ref.i32(bad[:3]))
    with pytest.raises(kda.KdaError):
        kda.kda_check_device_error()
    want = w.clone()
    want[1, 7] = 0
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("length", [0, 5, 300])
def test_one_row(length):
    """One head of one node in the whole batch."""
    case = Case([length], [1], H=1, page=16, seed=7)
    given = true_lse(case)
    check_weights(case, run_weights(case, given), given)
    _, lse = run_lse(case)
    check_lse(case, lse)


def test_rows_of_any_width_and_padding_behind_the_last_sequence():
    """weights rows that are no multiple of 16 bytes; query rows of no sequence behind the last."""
    case = Case([100, 61], [2, 1], H=16, page=16, seed=8)
    given = true_lse(case)
    check_weights(case, run_weights(case, given, width=103), given)
    case.q = torch.cat([case.q, torch.full_like(case.q, float("nan"))])
    padded = torch.cat([given, torch.full_like(given, float("nan"))])
    case.mask = case.mask + [0, 0, 0]
    got = run_weights(case, padded, width=103)
    kda.kda_check_device_error()
    case.q, case.mask = case.q[:3], case.mask[:3]
    check_weights(case, got, given)


def test_a_pool_beyond_four_gigabytes():
    _gpu.lib()
    n_pages, page, H, length = 70000, 64, 16, 200
    g = torch.Generator().manual_seed(3)
    rows = torch.randn(4 * page, 576, generator=g).to(torch.bfloat16)
    table = [n_pages - 1, 2, n_pages - 3, 5]
    pool = torch.zeros(n_pages, page, 576, dtype=torch.bfloat16, device="cuda")
    pool[table] = rows.view(4, page, 576).cuda()
    q = torch.randn(1, H, 576, generator=g).to(torch.bfloat16)
    paged = rows[None, :length + 1].contiguous()
    given = torch.tensor(long.lse(q, paged, [[0]], [length], [0, 1], None, kda.MLA_SCALE)[0]).float()
    want, tol = long.weights(q, paged, [[0]], [length], [0, 1], None, None, given.double().numpy(), kda.MLA_SCALE, 256)
    w = torch.zeros(1, 256, device="cuda")
    args = (pool, ref.i32([table]), ref.i32([length]))
    kda.mla_cache_weights(q.cuda(), *args, ref.i32([0, 1]), given.cuda(), w)
    assert (np.abs(w.double().cpu().numpy() - want) <= tol + 2.0**-24 * want).all()
    keys = torch.zeros(1, n_pages, 576, dtype=torch.bfloat16, device="cuda")
    kda.mla_block_keys(pool[None], args[1], ref.i32([256]), ref.i32([256]), keys)  # nothing filled up since
    assert not keys.any()
    kda.mla_block_keys(pool[None], args[1], ref.i32([0]), ref.i32([256]), keys)
    mean = rows.double().view(4, page, 576).mean(1)
    assert ((keys[0, table].double().cpu() - mean).abs() <= 2.0**-8 * mean.abs() + 1e-5).all()
    kept, cut = torch.zeros(1, 90, dtype=torch.int32, device="cuda"), ref.i32([0])
    kda.mla_cache_evict(pool[None], *args[1:], w, kept, cut, recent=9)
    kda.kda_check_device_error()
    chosen = long.choose(w[0].tolist(), length, 0, 9, 90)
    assert kept[0].tolist() == chosen
    assert torch.equal(pool[table[:2]].view(-1, 576)[:90].cpu(), rows[chosen])
