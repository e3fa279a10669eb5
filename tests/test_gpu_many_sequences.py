"""GPU: key sums of batches with more sequences than the kernels have threads (448 for positions, 480
for blocks), whose work is summed up in several passes: just behind a pass, and several passes long."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_gb300 import kda
from tests import _gpu
from tests import _tree_ref as ref
from tests.test_gpu_sparse import block_batch, check_scores, run_scores

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [447, 448, 449, 480, 481, 896, 897, 1345, 3000])
def test_weights_are_those_of_small_calls(n):
    """A position's sum does not depend on the other sequences of the call: the bits of calls of 64."""
    _gpu.lib()
    H, page, most = 4, 16, 9
    g, rng = torch.Generator().manual_seed(n), np.random.default_rng(n)
    lengths = [int(x) for x in rng.integers(0, page * most - 3, n)]
    counts = [int(x) for x in rng.integers(0, 4, n)]
    counts[-1] = 1
    cu = [0] + [int(x) for x in np.cumsum(counts)]
    table = torch.randint(0, 500, (n, most), generator=g, dtype=torch.int32).cuda()
    pool = torch.randn(500, page, 576, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(cu[-1], H, 576, generator=g).to(torch.bfloat16).cuda()
    lse = (3.0 + torch.rand(cu[-1], H, generator=g)).cuda()
    start = torch.rand(n, page * most, generator=g).cuda()
    got, want = start.clone(), start.clone()
    for _ in range(4):
        kda.mla_cache_weights(q, pool, table, ref.i32(lengths), ref.i32(cu), lse, got)
    for lo in range(0, n, 64):
        hi = min(lo + 64, n)
        a, b = cu[lo], cu[hi]
        if a == b:
            continue
        for _ in range(4):
            kda.mla_cache_weights(q[a:b], pool, table[lo:hi].contiguous(), ref.i32(lengths[lo:hi]),
                                  ref.i32([x - a for x in cu[lo:hi + 1]]), lse[a:b], want[lo:hi])
    kda.kda_check_device_error()
    assert torch.equal(got, want) and not torch.equal(got, start)


@pytest.mark.parametrize("n", [479, 480, 481, 961, 1500])
def test_scores_behind_a_pass(n):
    rng = np.random.default_rng(n)
    lengths = [int(x) for x in rng.integers(0, 260, n)]
    counts = [int(x) for x in rng.integers(0, 3, n)]
    b = block_batch(lengths, counts, H=2, page=16, seed=n)
    for _ in range(3):
        check_scores(run_scores(b[0], b[1], 16, b[2], lengths, b[3]), b[0], b[1], 16, b[2], lengths, b[3])
    kda.kda_check_device_error()
