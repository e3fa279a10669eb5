"""GPU: tree attention with log-sums inside a workspace of exactly the size asked for, with guards around it."""
import pytest
import torch

from hybrid_linear_attention_gb300 import kda
from tests import _gpu
from tests import _tree_ref as ref
from tests.test_gpu_cache_weights import check_lse
from tests.test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu
GUARD = 4096


@pytest.mark.parametrize("lengths,counts,H", [([20000], [1], 64), ([9000, 300], [9, 64], 16), ([700] * 90, [2] * 90, 64)])
def test_partial_sums_stay_inside(lengths, counts, H):
    _gpu.lib()
    case = Case(lengths, counts, H=H, seed=len(lengths))
    total, n = case.cu[-1], len(counts)
    size = kda.mla_tree_workspace_size(n, total, H)
    assert size == 160 * 128 * (512 + 2) * 4 + 80 * 32
    buf = torch.full((size + 2 * GUARD,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
    ws = buf[GUARD:GUARD + size]
    mask = None if case.mask is None else torch.tensor(case.mask, dtype=torch.int64, device="cuda")
    args = (case.q.cuda(), case.pool.cuda(), ref.i32(case.table), ref.i32(case.lengths), ref.i32(case.cu))
    z = [torch.full((total, H, 512), 7.0, device="cuda") for _ in range(2)]
    lse = torch.full((total, H), 7.0, device="cuda")
    kda.mla_tree_latent(*args, z[0], mask=mask, workspace=ws)
    kda.mla_tree_latent_lse(*args, z[1], lse, mask=mask, workspace=ws)
    kda.kda_check_device_error()
    assert torch.equal(z[0], z[1])
    check_lse(case, lse)
    assert (buf[:GUARD] == 0xFF).all() and (buf[GUARD + size:] == 0xFF).all()
