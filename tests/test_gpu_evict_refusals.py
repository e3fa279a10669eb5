"""GPU: which sequences an eviction refuses for their pages: those of which a row would move from or to a
page that is not there, or into a shared one, and no others."""
import pytest
import torch

from hybrid_linear_attention_gb300 import kda
from tests.test_gpu_cache_evict import Cache

pytestmark = pytest.mark.gpu


def reported(wanted):
    if not wanted:
        return kda.kda_check_device_error()
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX


class Pages(Cache):
    """Pages may be missing; `check` reads only those that kept rows come from or go to."""

    def missing(self, n, *pages):
        for j in pages:
            self.table[n][j] = -1


@pytest.mark.parametrize("length", [200, 9000, 70001])  # one CTA, and clusters
@pytest.mark.parametrize("kind", ["random", "ties"])
@pytest.mark.parametrize("new", ["aside", "own"])
def test_pages_without_a_kept_row_may_be_missing(length, kind, new):
    c = Pages([length] * 2, page=16, layers=1, seed=1, kind=kind)
    c.w[:, 100:160] = float("nan")           # never kept: more than the budget are left
    c.w[0, length - 60:] = float("nan")
    budget = 70
    c.w[0, :16] = c.w[1, :16] = 50.0         # page 0 stays
    c.missing(0, 7, 8, 9, length // 16 - 1)  # wholly inside what is dropped
    c.missing(1, 7)
    d = c.run(budget, new=new)
    reported(False)
    c.check(d, budget, new=new)


def test_missing_pages_behind_rows_that_all_stay():
    """The budget's first positions are kept as they are: nothing moves, whatever the pages behind them are."""
    c = Pages([200, 200, 9000], page=16, layers=2, seed=2)
    c.w[:, :100] = 50.0
    c.missing(0, 7, 12), c.missing(2, 400)
    c.refs[c.table[1][6]] = 2                # the page that position 100 is in, shared: not written
    d = c.run(100)
    reported(False)
    c.check(d, 100)


@pytest.mark.parametrize("length", [200, 9000, 70001])
def test_pages_that_are_needed(length):
    """A kept position's page, a target's, and a shared target's, each alone in its sequence."""
    c = Pages([length] * 4, page=16, layers=1, seed=3)
    c.w[:, :16] = 50.0
    c.w[:, 16:40] = float("nan")             # a gap from position 16 on
    for n in range(4):
        c.w[n, 150] = 60.0
    c.missing(0, 9)                          # position 150's
    c.missing(1, 1)                          # where the first moved rows go
    c.refs[c.table[2][4]] = 2                # where the last ones go (positions 64 .. 69)
    c.refs[c.table[3][5]] = 2                # behind the budget: read at most
    d = c.run(70)
    reported(True)
    c.check(d, 70, refused=(0, 1, 2))


def test_equal_weights_are_looked_at_one_by_one():
    """Of equal weights the first are kept: the page of the last kept one counts, the one behind does not."""
    c = Pages([320, 320], page=16, layers=1, seed=4, kind="same")
    c.w[:, 5] = -1.0                         # kept: 0 .. 4, 6 .. 80, that is pages 0 .. 5
    c.missing(0, 6, 19)
    c.missing(1, 5)
    d = c.run(80)
    reported(True)
    c.check(d, 80, refused=(1,))
