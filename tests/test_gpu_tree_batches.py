"""GPU: the tree calls over batches as large as a server's: more sequences, entries and units of work
than one pass of a kernel's bookkeeping or one wave of its blocks takes."""
import numpy as np
import pytest
import torch

import oracle
from hybrid_linear_attention_gb300 import kda
from tests import _gpu
from tests import _tree_ref as ref
from tests.test_gpu_tree_attention import Case
from tests.test_gpu_tree_kda import make
from tests.test_gpu_tree_pages import Both, status

pytestmark = pytest.mark.gpu


# ---- attention: the plan of a batch is made 448 sequences at a time --------------------------------

@pytest.mark.parametrize("n,long_at", [(448, 447), (449, 448), (900, 500), (900, 899), (2000, 1300)])
def test_attention_of_many_sequences(n, long_at):
    """Short ragged sequences, empty ones among them, and one long context that several workers share,
    planned in a later pass than the first."""
    rng = np.random.default_rng(n + long_at)
    lengths = [int(x) for x in rng.integers(0, 60, n)]
    counts = [int(x) for x in rng.choice([0, 1, 1, 2, 3], n)]
    lengths[long_at], counts[long_at] = 6000, 9
    case = Case(lengths, counts, H=16, page=16, seed=n)
    for z_dtype in (torch.bfloat16, torch.float32):
        case.check(case.run(z_dtype), z_dtype)
    kda.kda_check_device_error()


def test_attention_of_many_long_sequences_in_groups():
    """More sequences than a pass and several row tiles each, so that clusters work in groups."""
    rng = np.random.default_rng(17)
    case = Case([int(x) for x in rng.integers(200, 700, 460)], [int(x) for x in rng.integers(6, 9, 460)], H=48, page=32,
                seed=171)
    z = case.run(torch.float32)
    kda.kda_check_device_error()
    pick = [0, 1, 200, 446, 447, 448, 449, 450, 458, 459]
    rows = np.concatenate([np.arange(case.cu[b], case.cu[b + 1]) for b in pick])
    part = Case([1], [1], H=48, page=32)
    part.lengths, part.counts = [case.lengths[b] for b in pick], [case.counts[b] for b in pick]
    part.cu = [0] + [int(x) for x in np.cumsum(part.counts)]
    part.table, part.pool, part.q = [case.table[b] for b in pick], case.pool, case.q[rows]
    part.mask = [case.mask[r] for r in rows]
    part.check(z[rows], torch.float32)
    assert np.isfinite(z).all() and not (z == 7.0).any()  # no row was left out


# ---- the whole latent-attention step ---------------------------------------------------------------

def test_tree_decode_against_the_64_bit_form():
    """Three blocks of 128 rows in the projections.  Stage by stage, each from what the one before
    left: q~ is an fp32 sum of 128 products rounded to bf16; z as mla_tree_latent's; o an fp32 sum of
    2 x 512 products of z in two bf16 parts (2^-17 of it) and W_V, times the gate, rounded to bf16.
    Each addition may be off by a whole fp32 step, 2^-23 of the sum of the sizes."""
    _gpu.lib()
    rng = np.random.default_rng(41)
    n = 131
    case = Case([int(x) for x in rng.integers(0, 300, n)], [int(x) for x in rng.choice([0, 1, 2, 3, 4], n)], seed=41)
    total = case.cu[-1]
    assert 256 < total < 384
    g = torch.Generator().manual_seed(42)
    bf = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(torch.bfloat16)  # noqa: E731
    qn, qr, gate = bf(total, 64, 128), bf(total, 64, 64), bf(total, 64)
    uk, uv = bf(64, 128, 512, std=0.05), bf(64, 128, 512, std=0.05)
    q_cat = torch.full((total, 64, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    z = torch.full((total, 64, 512), 7.0, device="cuda")
    out = torch.full((total, 64, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kda.mla_tree_workspace_size(n, total), dtype=torch.uint8, device="cuda")
    kda.mla_tree_decode(qn.cuda(), qr.cuda(), uk.cuda(), uv.cuda(), case.pool.cuda(), ref.i32(case.table),
                        ref.i32(case.lengths), ref.i32(case.cu), gate.cuda(), q_cat, z, out,
                        mask=torch.tensor(case.mask, dtype=torch.int64, device="cuda"), workspace=ws)
    kda.kda_check_device_error()
    want = oracle.mla_absorb(qn, qr, uk)
    size = np.einsum("bhn,hnl->bhl", np.abs(qn.double().numpy()), np.abs(uk.double().numpy()))
    off = np.abs(q_cat.double().cpu().numpy() - want)
    assert (off[..., 512:] == 0).all()
    assert (off[..., :512] <= 1.02 * (2.0**-8 * np.abs(want[..., :512]) + 128 * 2.0**-23 * size)).all()
    case.q = q_cat.cpu()
    case.check(z.double().cpu().numpy(), torch.float32)
    zz, w = z.double().cpu().numpy(), uv.double().numpy()
    s = 1 / (1 + np.exp(-gate.double().numpy()))[..., None]
    want, size = (np.einsum("bhl,hvl->bhv", f(zz), f(w)) * s for f in (lambda x: x, np.abs))
    off = np.abs(out.double().cpu().numpy() - want)
    assert (off <= 1.02 * (2.0**-8 * np.abs(want) + (2.0**-17 + 1024 * 2.0**-23) * size)).all()


# ---- KDA accept: more (sequence, head) groups than blocks ------------------------------------------

def pick_heads(m, heads, H, d=128):
    """The same batch with some of its heads (heads do not meet in a KDA layer)."""
    split = lambda t: t.view(*t.shape[:-1], 3, H, d)[..., heads, :].reshape(*t.shape[:-1], -1)  # noqa: E731
    w = m["conv_w"].view(3, H, d, 4)[:, heads].reshape(-1, 4)
    return dict(m, x=split(m["x"]), conv_w=w, conv_state=split(m["conv_state"]), g=m["g"][:, heads],
                beta=m["beta"][:, heads], state=m["state"][:, heads])


@pytest.mark.parametrize("st", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,H", [(40, 16), (61, 15), (24, 128), (48, 64)])
def test_accept_of_many_groups(n, H, st):
    """Blocks that walk several groups of one head (the first two sizes) and of two (the others; 24 x 128 and
    48 x 64 heads give each block at least four).  Rejected drafts, empty trees, slots out of range and
    accepted nodes out of range lie between sequences with short and with long paths."""
    _gpu.lib()
    rng = np.random.default_rng(n * H)
    counts = [int(x) for x in rng.choice([0, 1, 3, 6, 8, 14], n)]
    counts[0], counts[-1] = 14, 14
    p = kda.params(H=H, state_dtype=st)
    m = make(counts, H, 128, seed=500 + n, st=st)
    for b in range(0, n, 3):  # long paths: more than eight tokens
        m["parent"][m["cu"][b]:m["cu"][b + 1]] = list(range(-1, counts[b] - 1))
    accept = [-1 if w == 0 or rng.random() < 0.3 else int(rng.integers(0, w)) for w in counts]
    accept[0], accept[-1] = 13, 13
    accept[1], accept[2] = -1, -1
    slots = list(m["slots"])
    slots[4], slots[5], slots[17] = -1, n + 2, 2**31 - 1
    accept[7], accept[8] = counts[7], -2
    c = lambda t: t.cuda().contiguous()  # noqa: E731
    args = [c(m[k]) for k in ("x", "conv_w", "conv_state", "g", "beta", "state")]
    cu, parent = ref.i32(m["cu"]), ref.i32(m["parent"])
    kda.kda_tree_accept(p, *args, cu, parent, ref.i32(accept), slot_idx=ref.i32(slots))
    assert status() == kda.KDA_ERR_BAD_INDEX
    got_state, got_tail = args[5].cpu(), args[2].cpu()
    good = [b for b in range(n) if 0 <= accept[b] < counts[b] and 0 <= slots[b] < n + 2]
    assert len(good) > n // 3
    # a sequence at a time, a group a block: the same bits
    one_state, one_tail = c(m["state"]), c(m["conv_state"])
    for b in good:
        lo, hi = m["cu"][b], m["cu"][b + 1]
        x, g, beta, par = (t[lo:hi].clone() for t in (args[0], args[3], args[4], parent))
        kda.kda_tree_accept(p, x, args[1], one_tail, g, beta, one_state, ref.i32([0, hi - lo]), par,
                            ref.i32([accept[b]]), slot_idx=ref.i32([slots[b]]))
    kda.kda_check_device_error()
    assert torch.equal(got_state, one_state.cpu()) and torch.equal(got_tail, one_tail.cpu())
    # and some heads against the 64-bit form
    heads = [0, 1, H // 2, H - 1]
    few = pick_heads(m, heads, H)
    ok = [accept[b] if b in good else -1 for b in range(n)]
    _, state, tail = ref.kda_tree(few["x"], few["conv_w"], few["conv_state"], few["g"], few["beta"], few["state"],
                                  m["slots"], m["cu"], m["parent"], H=4, d=128, accept=ok)
    got = got_state[:, heads].double().numpy()
    step = 2.0**-8 * np.abs(state) if st == torch.bfloat16 else 0
    assert (np.abs(got - state) - step).max() <= (1e-3 if st == torch.bfloat16 else 1e-4) * np.sqrt((state ** 2).mean())
    got = pick_heads(dict(m, conv_state=got_tail), heads, H)["conv_state"]
    assert np.array_equal(got.double().numpy(), tail)


# ---- rows and pages --------------------------------------------------------------------------------

@pytest.mark.parametrize("n", [32, 33, 65, 500, 1100])
def test_append_of_many_sequences(n):
    """Empty sequences in runs, at the front and at the end; one prompt of 3000 rows among them."""
    _gpu.lib()
    rng = np.random.default_rng(n)
    counts = [int(x) for x in rng.choice([0, 0, 1, 2, 9], n)]
    counts[:3] = counts[-3:] = [0, 0, 0]
    counts[n // 2] = 3000
    lengths = [int(x) for x in rng.integers(0, 40, n)]
    cu = [0] + [int(x) for x in np.cumsum(counts)]
    needs = [-(-(a + b) // 16) for a, b in zip(lengths, counts)]
    order, at, most = rng.permutation(sum(needs) + 3), 0, max(needs)
    table = np.full((n, most), -1)
    for b, k in enumerate(needs):
        table[b, :k] = order[at:at + k]
        at += k
    rows = torch.randn(2, cu[-1] + 5, 576, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16)
    want = torch.zeros(2, sum(needs) + 3, 16, 576, dtype=torch.bfloat16)
    for b in range(n):
        t = lengths[b] + np.arange(counts[b])
        want[:, table[b, t // 16], t % 16] = rows[:, cu[b]:cu[b + 1]]
    pool = torch.zeros_like(want).cuda()
    kda.mla_cache_append(pool, ref.i32(table.tolist()), ref.i32(lengths), ref.i32(cu), rows.cuda())
    assert status() == kda.KDA_OK
    assert torch.equal(pool.cpu(), want)


@pytest.mark.parametrize("room", [2000, 900, 0])
def test_fork_of_more_entries_than_a_pass(room):
    """1500 children of 60 parents, some named twice; pages enough, too few for the later entries, none."""
    rng = np.random.default_rng(room)
    parents, children = 60, 1500
    needs = [int(x) for x in rng.integers(0, 49, parents)]
    pages = sum(-(-x // 16) for x in needs)
    b = Both(pages + room, parents + children, 4, 16, layers=1, seed=room)
    assert not b.reserve(list(range(parents)), needs)
    for s, x in enumerate(needs):
        b.set_length(s, x)
    src = [int(x) for x in rng.integers(0, parents, children)]
    dst = [parents + int(x) for x in rng.permutation(children)]
    if room == 2000:
        dst[1400], dst[1030] = dst[3], dst[1029]  # an earlier entry has the child
    bad, out = b.fork(src, dst)
    assert bad == (room == 2000) and out == (room < 2000)
    want = kda.KDA_ERR_BAD_INDEX if bad else kda.KDA_ERR_NO_PAGES
    assert status() == want
    b.same()
