"""GPU: a step without a drafted node."""
import pytest
import torch

from hybrid_linear_attention_gb300 import kda
from tests import _gpu
from tests import _tree_ref as ref

pytestmark = pytest.mark.gpu


def test_a_sparse_call_without_nodes_leaves_its_outputs():
    """Nothing is launched: scores, selection and z stay as an earlier step left them; mla_block_select on its
    own writes empty rows."""
    _gpu.lib()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    pool, keys, q, z = torch.zeros(8, 16, 576, **bf), torch.zeros(8, 576, **bf), torch.zeros(0, 16, 576, **bf), torch.zeros(0, 16, 512, **bf)
    table, lengths, cu = ref.i32([[0, 1, 2], [3, 4, -1]]), ref.i32([40, 30]), ref.i32([0, 0, 0])
    scores, sel, cut = torch.full((2, 3), 7.0, device="cuda"), ref.i32([[9] * 4] * 2), ref.i32([5, 5])
    ws = torch.zeros(kda.mla_sparse_workspace_size(2, 1, 16, 3), dtype=torch.uint8, device="cuda")
    kda.mla_sparse_latent(q, pool, keys, table, lengths, cu, scores, sel, cut, z, blocks=2, workspace=ws)
    kda.kda_check_device_error()
    assert (scores == 7.0).all() and (sel == 9).all() and (cut == 5).all()
    kda.mla_block_select(scores, 16, table, lengths, cu, sel, cut, blocks=2, total_nodes=0)
    kda.kda_check_device_error()
    assert (sel == -1).all() and (cut == 0).all()
