"""GPU: the KDA layer over drafted trees against the plain 64-bit form.

Tolerances are the layer's own: fp32 arithmetic throughout, so outputs within 1e-4 of the output's
RMS (fp32 I/O) or 1e-2 beyond half a bf16 step (bf16 I/O), states within 1e-4 of the state's RMS
(1e-3 where the state is stored in bf16, beyond half a step); the conv tail bit for bit."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_gb300 import kda
from tests import _gpu
from tests import _tree_ref as ref
from tests import _parity

pytestmark = pytest.mark.gpu


def make(counts, H, d, seed, io=torch.bfloat16, st=torch.float32, slots=None, n_slots=None, chain=False):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    n, total = len(counts), sum(counts)
    n_slots = n_slots or n + 2
    slots = slots if slots is not None else [int(x) for x in rng.permutation(n_slots)[:n]]
    r = lambda *s, std=1.0: torch.randn(*s, generator=g) * std  # noqa: E731
    parents = [list(range(-1, w - 1)) if chain else ref.random_parents(rng, w) for w in counts]
    return dict(x=r(total, 3 * H * d).to(io), conv_w=r(3 * H * d, 4, std=0.5).to(io),
                conv_state=r(n_slots, 3, 3 * H * d).to(io), g=-5.5 * torch.rand(total, H, d, generator=g),
                beta=torch.sigmoid(r(total, H)), state=r(n_slots, H, d, d, std=0.1).to(st), slots=slots,
                cu=[0] + [int(v) for v in np.cumsum(counts)], parent=[p for q in parents for p in q],
                gate=r(total, H, d).to(io), norm_w=torch.rand(d, generator=g) + 0.5)


def device(m, p):
    _gpu.lib()
    c = _gpu.cuda
    keep = dict(state=c(m["state"]).clone(), conv_state=c(m["conv_state"]).clone())
    args = (p, c(m["x"]), c(m["conv_w"]), keep["conv_state"], c(m["g"]), c(m["beta"]), keep["state"], ref.i32(m["cu"]),
            ref.i32(m["parent"]) if m["parent"] else torch.zeros(0, dtype=torch.int32, device="cuda"))
    return args, keep


def verify(m, p, *, gated=True, max_nodes=64, fill=0.0):
    args, keep = device(m, p)
    out = torch.full(tuple(m["g"].shape), fill, dtype=p.io_torch, device="cuda")
    kda.kda_tree_verify(*args, out, max_nodes=max_nodes, slot_idx=ref.i32(m["slots"]),
                        gate_logit=_gpu.cuda(m["gate"]) if gated else None,
                        norm_w=_gpu.cuda(m["norm_w"]) if gated else None)
    torch.cuda.synchronize()
    assert torch.equal(keep["state"].cpu(), m["state"]) and torch.equal(keep["conv_state"].cpu(), m["conv_state"])
    return out


def plain(m, p, *, gated=True, accept=None):
    return ref.kda_tree(m["x"], m["conv_w"], m["conv_state"], m["g"], m["beta"], m["state"], m["slots"], m["cu"],
                        m["parent"], H=p.H, d=p.d_k, scale=p.scale, gate=m["gate"] if gated else None,
                        norm_w=m["norm_w"] if gated else None, accept=accept, l2norm=bool(p.qk_l2norm))


def out_error(got, want):
    return _parity.out_error(got, want, got.dtype)


def tol(p):
    return 1e-2 if p.io_torch == torch.bfloat16 else 1e-4


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [16, 128])
def test_verify_ragged_trees(d, io, gated):
    """One to eleven nodes, several roots, an empty sequence; retentions past the clamp."""
    p = kda.params(H=3, d=d, io_dtype=io)
    m = make([1, 5, 0, 11, 2, 3], 3, d, seed=d, io=io)
    out = verify(m, p, gated=gated, max_nodes=11)
    kda.kda_check_device_error()
    assert out_error(out, plain(m, p, gated=gated)[0]) <= tol(p)


@pytest.mark.parametrize("w,chain", [(1, True), (8, False), (9, True), (16, False), (17, False), (31, True), (40, False),
                                     (64, True), (64, False)])
def test_verify_node_counts(w, chain):
    """Up to 64 nodes; a chain of 64 has a path whose retentions add up past fp32's exponents."""
    p = kda.params(H=2)
    m = make([w, max(1, w // 2)], 2, 128, seed=200 + w, chain=chain)
    assert out_error(verify(m, p, max_nodes=w), plain(m, p)[0]) <= tol(p)
    kda.kda_check_device_error()


def test_verify_bf16_state_and_no_l2norm():
    p = kda.params(H=2, state_dtype=torch.bfloat16, qk_l2norm=False, scale=0.25)
    m = make([6, 4], 2, 128, seed=300, st=torch.bfloat16)
    m["conv_w"] = (m["conv_w"].float() * 0.2).to(torch.bfloat16)  # unnormalised keys: keep the writes contracting
    assert out_error(verify(m, p), plain(m, p)[0]) <= tol(p)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("chain", [True, False])
def test_verify_retentions_of_zero(chain, io):
    """Without a lower bound: a node that forgets its past, in some channels or in all.  One such node a
    path: its sums stay under 2^8, whose half step 2^-17 enters at most 11 times, 6e-5 of a term."""
    p = kda.params(H=2, g_min=-float("inf"), io_dtype=io)
    m = make([11, 6], 2, 128, seed=305, chain=chain, io=io)
    m["g"][2] = -float("inf")
    m["g"][13] = torch.tensor([-0.1, -300.0, -1e6, -3e38, -88.0, -100.0, -0.5, -float("inf")]).repeat(16)
    want = ref.kda_tree(m["x"], m["conv_w"], m["conv_state"], m["g"], m["beta"], m["state"], m["slots"], m["cu"],
                        m["parent"], H=2, d=128, gate=m["gate"], norm_w=m["norm_w"], g_min=-float("inf"))[0]
    assert out_error(verify(m, p, max_nodes=11), want) <= tol(p)
    kda.kda_check_device_error()


def test_verify_shared_slot():
    """Two drafts of one sequence: the pool state is only read."""
    p = kda.params(H=2)
    m = make([4, 5], 2, 128, seed=301, slots=[1, 1])
    assert out_error(verify(m, p), plain(m, p)[0]) <= tol(p)


def test_verify_large_batch_many_units():
    """More (sequence, head) units than CTAs fit: each CTA walks several trees of different sizes."""
    rng = np.random.default_rng(8)
    counts = [int(x) for x in rng.integers(0, 13, 60)]
    p = kda.params(H=16)
    m = make(counts, 16, 128, seed=302)
    assert out_error(verify(m, p, max_nodes=12), plain(m, p)[0]) <= tol(p)


def test_verify_equals_the_chain_call():
    """A chain's outputs are those of the fused one-token step run token by token."""
    p = kda.params(H=4)
    m = make([5, 5], 4, 128, seed=303, chain=True)
    out = verify(m, p)
    args, keep = device(m, p)
    for i in range(5):
        rows = torch.tensor([i, 5 + i], device="cuda")
        o = torch.empty((2, 4, 128), dtype=torch.bfloat16, device="cuda")
        kda.kda_decode_step_fused(p, args[1][rows].contiguous(), args[2], keep["conv_state"], args[4][rows].contiguous(),
                                  args[5][rows].contiguous(), keep["state"], o, slot_idx=ref.i32(m["slots"]),
                                  gate_logit=_gpu.cuda(m["gate"])[rows].contiguous(), norm_w=_gpu.cuda(m["norm_w"]))
        rms = float(o.double().square().mean().sqrt())
        # both within 1e-4 RMS of the same fp32 function, then each rounded to bf16 (2^-8 of the value)
        assert float((out[rows].double() - o.double()).abs().sub(2.0**-7 * o.double().abs()).max()) <= 2e-4 * rms
    # and accepting the last node leaves the state of that chain
    again, kept = device(m, p)
    kda.kda_tree_accept(*again, ref.i32([4, 4]), slot_idx=ref.i32(m["slots"]))
    kda.kda_check_device_error()
    rms = float(keep["state"].double().square().mean().sqrt())
    assert float((kept["state"].double() - keep["state"].double()).abs().max()) <= 1e-4 * rms
    assert torch.equal(kept["conv_state"], keep["conv_state"])


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [16, 128])
def test_accept_paths(d, io):
    """Paths of one to many tokens, nothing accepted, an empty tree; unnamed slots stay as they were."""
    p = kda.params(H=3, d=d, io_dtype=io)
    m = make([1, 6, 4, 0, 12, 3, 30], 3, d, seed=400 + d, io=io)
    accept = [0, 5, -1, -1, 11, 1, 29]
    args, keep = device(m, p)
    kda.kda_tree_accept(*args, ref.i32(accept), slot_idx=ref.i32(m["slots"]))
    kda.kda_check_device_error()
    _, state, tail = plain(m, p, accept=accept)
    got = keep["state"].double().cpu().numpy()
    assert np.abs(got - state).max() <= 1e-4 * np.sqrt((state ** 2).mean())
    assert np.array_equal(keep["conv_state"].double().cpu().numpy(), tail)
    named = {m["slots"][i] for i, a in enumerate(accept) if a >= 0}
    for s in set(range(m["state"].shape[0])) - named:
        assert torch.equal(keep["state"][s].cpu(), m["state"][s])


def test_accept_a_chain_of_64_and_bf16_state():
    p = kda.params(H=2, state_dtype=torch.bfloat16)
    m = make([64, 9], 2, 128, seed=410, st=torch.bfloat16, chain=True)
    args, keep = device(m, p)
    kda.kda_tree_accept(*args, ref.i32([63, 8]), slot_idx=ref.i32(m["slots"]))
    _, state, tail = plain(m, p, accept=[63, 8])
    got = keep["state"].double().cpu().numpy()
    off = np.maximum(np.abs(got - state) - 2.0**-8 * np.abs(state), 0)
    assert off.max() <= 1e-3 * np.sqrt((state ** 2).mean())
    assert np.array_equal(keep["conv_state"].double().cpu().numpy(), tail)


def test_bad_indices_are_reported_and_skipped():
    p = kda.params(H=2)
    m = make([3, 4, 2], 2, 128, seed=420)
    good = verify(m, p)
    # a parent that is not an earlier node counts as a root
    bad = dict(m, parent=list(m["parent"]))
    bad["parent"][1] = 2
    root = dict(m, parent=list(m["parent"]))
    root["parent"][1] = -1
    out = verify(bad, p)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX
    assert torch.equal(out, verify(root, p))
    # a slot outside the pool, a tree larger than max_nodes, offsets past the rows
    for change, status in ((dict(slots=[m["slots"][0], 99, m["slots"][2]]), kda.KDA_ERR_BAD_INDEX),
                           (dict(), kda.KDA_ERR_BAD_SEQLENS)):
        out = verify(dict(m, **change), p, max_nodes=64 if change else 3, fill=7.0)
        with pytest.raises(kda.KdaError) as e:
            kda.kda_check_device_error()
        assert e.value.status == status
        assert torch.equal(out[:3], good[:3]) and torch.equal(out[7:], good[7:]) and bool((out[3:7] == 7.0).all())
    args, keep = device(m, p)
    kda.kda_tree_accept(*args, ref.i32([3, -2, 1]), slot_idx=ref.i32(m["slots"]))
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX
    for s in (0, 1):
        assert torch.equal(keep["state"][m["slots"][s]].cpu(), m["state"][m["slots"][s]])
    _, state, _ = plain(m, p, accept=[-1, -1, 1])
    got = keep["state"].double().cpu().numpy()
    assert np.abs(got - state).max() <= 1e-4 * np.sqrt((state ** 2).mean())


def test_captured_verify_and_accept_replay():
    """Captured once, replayed on new inputs and trees."""
    p = kda.params(H=2)
    a, b = (make([5, 3], 2, 128, seed=s) for s in (430, 431))
    args, keep = device(a, p)
    out = torch.full((8, 2, 128), 0.0, dtype=torch.bfloat16, device="cuda")
    slots, accept = ref.i32(a["slots"]), ref.i32([3, 2])
    gate, nw = _gpu.cuda(a["gate"]), _gpu.cuda(a["norm_w"])

    def step():
        kda.kda_tree_verify(*args, out, max_nodes=5, slot_idx=slots, gate_logit=gate, norm_w=nw)
        kda.kda_tree_accept(*args, accept, slot_idx=slots)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    b["norm_w"] = a["norm_w"]
    for t, k in ((args[1], "x"), (args[2], "conv_w"), (keep["conv_state"], "conv_state"), (args[4], "g"),
                 (args[5], "beta"), (keep["state"], "state"), (gate, "gate")):
        t.copy_(b[k])
    slots.copy_(ref.i32(b["slots"]))
    args[8].copy_(ref.i32(b["parent"]))
    graph.replay()
    kda.kda_check_device_error()
    want, state, tail = plain(b, p, accept=[3, 2])
    assert out_error(out, want) <= tol(p)
    assert np.abs(keep["state"].double().cpu().numpy() - state).max() <= 1e-4 * np.sqrt((state ** 2).mean())
    assert np.array_equal(keep["conv_state"].double().cpu().numpy(), tail)


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("forget,nodes", [(-5.0, 8), (-5.0, 40), (-88.0, 11), (-88.0, 40)])
@pytest.mark.parametrize("d", [16, 128])
def test_verify_retains_after_forgetting(d, forget, nodes, io, gated):
    """A chain of 64 that forgets strongly for some nodes and then hardly at all.  The log-retentions'
    sum is held to 2^-21 a step (half a step of fp32 below 2^4), so a decay over 56 steps is off by at
    most 56 * 2^-21 * ln 2 = 1.9e-5 of itself, wherever on the path the steps are."""
    p = kda.params(H=2, d=d, io_dtype=io, g_min=forget)
    m = make([64, 50], 2, d, seed=306, chain=True, io=io)
    for lo in (0, 64):
        m["g"][lo:lo + nodes] = forget
        m["g"][lo + nodes:] = -0.013
    want = ref.kda_tree(m["x"], m["conv_w"], m["conv_state"], m["g"], m["beta"], m["state"], m["slots"], m["cu"],
                        m["parent"], H=2, d=d, gate=m["gate"] if gated else None,
                        norm_w=m["norm_w"] if gated else None, g_min=forget)[0]
    assert out_error(verify(m, p, gated=gated), want) <= tol(p)
    kda.kda_check_device_error()


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
def test_verify_deep_trees_of_mixed_retentions(io):
    """Channels that forget at different nodes of a branching tree, some at every other node."""
    p = kda.params(H=3, io_dtype=io, g_min=-float("inf"))
    m = make([64, 33, 5], 3, 128, seed=307, io=io)
    g = torch.Generator().manual_seed(308)
    kind = torch.randint(0, 6, m["g"].shape, generator=g)
    kind[:, :, ::3] = 5
    m["g"] = torch.tensor([-0.01, -0.3, -7.0, -40.0, -88.0, -0.02])[kind].contiguous()
    want = ref.kda_tree(m["x"], m["conv_w"], m["conv_state"], m["g"], m["beta"], m["state"], m["slots"], m["cu"],
                        m["parent"], H=3, d=128, gate=m["gate"], norm_w=m["norm_w"], g_min=-float("inf"))[0]
    assert out_error(verify(m, p), want) <= tol(p)
    kda.kda_check_device_error()


@pytest.mark.parametrize("io,st", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("most", [1, 3, 8, 11, 12, 20])
@pytest.mark.parametrize("d,n,H", [(128, 40, 16), (16, 90, 64)])
def test_verify_of_many_units_in_every_form(d, n, H, most, io, st):
    """More units than fit at a time, trees that are not a multiple of eight nodes, with the sums of the
    log-retentions short enough for one fp32 number (the clamp at -5) and not (none, or strong forgetting)."""
    rng = np.random.default_rng(most + d)
    counts = [int(x) for x in rng.integers(0, most + 1, n)]
    counts[3] = most
    for g_min, strong in ((-5.0, -5.0), (-float("inf"), -80.0)):
        p = kda.params(H=H, d=d, io_dtype=io, state_dtype=st, g_min=g_min)
        m = make(counts, H, d, seed=600 + most, io=io, st=st, chain=most > 9)
        kind = torch.rand(m["g"].shape, generator=torch.Generator().manual_seed(most))
        m["g"] = torch.where(kind < 0.4, torch.tensor(strong), -0.05 * kind).contiguous()
        want = ref.kda_tree(m["x"], m["conv_w"], m["conv_state"], m["g"], m["beta"], m["state"], m["slots"], m["cu"],
                            m["parent"], H=H, d=d, g_min=g_min)[0]
        assert out_error(verify(m, p, gated=False, max_nodes=most), want) <= tol(p)
    kda.kda_check_device_error()


@pytest.mark.parametrize("nodes,forget", [(17, 8), (17, 13), (12, 9), (11, 4), (8, 4), (8, 3)])
def test_verify_shallow_trees_retain_after_forgetting(nodes, forget):
    """Paths around the longest that one fp32 sum serves (8 nodes at the clamp -5): 7 steps off by 2^-20 each
    (half a step of fp32 below 2^5) are 4.6e-6 of a decay, 16 steps of 2^-21 behind it 5.3e-6."""
    for d, n, H in ((128, 40, 16), (16, 90, 64)):
        p = kda.params(H=H, d=d, io_dtype=torch.float32)
        m = make([nodes] * n, H, d, seed=610, chain=True, io=torch.float32)
        g = m["g"].view(n, nodes, H, d)
        g[:, :forget], g[:, forget:] = -5.0, -0.013
        want = ref.kda_tree(m["x"], m["conv_w"], m["conv_state"], m["g"], m["beta"], m["state"], m["slots"], m["cu"],
                            m["parent"], H=H, d=d)[0]
        assert out_error(verify(m, p, gated=False, max_nodes=nodes), want) <= tol(p)
    kda.kda_check_device_error()
