"""GPU: key sums whose rows end inside a chunk of 128 at every padded width (32, 64, 96 and 128 columns; of
blocks 64 and 128), the only chunk of a sequence or behind others."""
import pytest

from hybrid_linear_attention_gb300 import kda
from tests.test_gpu_cache_weights import Case, check_weights, run_weights, true_lse
from tests.test_gpu_sparse import block_batch, check_scores, run_scores

pytestmark = pytest.mark.gpu
NODES = [1, 2, 4, 6, 7, 8, 9, 11, 12, 64]  # of 20 heads: 20, 40, 80, 120 rows, then 12, 32, 52, 92, 112 and 128 in the last chunk


@pytest.mark.parametrize("w", NODES)
def test_weights(w):
    case = Case([300, 17], [w, 1], H=20, page=32, seed=500 + w)
    given = true_lse(case)
    check_weights(case, run_weights(case, given), given)
    u = [float(i % 3 > 0) for i in range(w + 1)]  # some chunks without a node that counts
    check_weights(case, run_weights(case, given, node_weight=u), given, node_weight=u)
    kda.kda_check_device_error()


@pytest.mark.parametrize("w", NODES)
def test_scores(w):
    lengths, counts = [5000, 40, 700], [w, 2, w]
    b = block_batch(lengths, counts, H=20, page=16, seed=600 + w)
    check_scores(run_scores(b[0], b[1], 16, b[2], lengths, b[3]), b[0], b[1], 16, b[2], lengths, b[3])
    kda.kda_check_device_error()
