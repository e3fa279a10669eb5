"""GPU: a refused sequence keeps its weights in a separate row of new weights too."""
import numpy as np
import pytest

from hybrid_linear_attention_gb300 import kda
from tests.test_gpu_cache_evict import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [199, 64, None])
def test_bad_lengths_keep_the_whole_row(width):
    """Below 0, more than the table row holds, more than the weights' row holds; beside a good one."""
    c = Cache([200, 200, 200, 40], page=16, seed=21, width=width)
    c.lengths[0], c.lengths[1] = -3, 10**6
    if width is None:
        c.lengths[2] = 209  # the table row holds 208
    d = c.run(80, recent=3)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX
    got = d["new_w"].cpu().numpy()
    assert np.array_equal(got[:3], c.w[:3].numpy())
    c.check(d, 80, recent=3, refused=(0, 1, 2))


def test_a_long_row_by_a_cluster():
    c = Cache([70000], page=64, layers=1, seed=22, width=70001)
    c.lengths[0] = 70002
    d = c.run(500)
    with pytest.raises(kda.KdaError):
        kda.kda_check_device_error()
    assert np.array_equal(d["new_w"].cpu().numpy(), c.w.numpy())
