"""A sparse call without a drafted node launches nothing, and refuses what it would refuse with one."""
import pytest

from hybrid_linear_attention_gb300 import kda
from tests.test_long_context_abi import BAD, CHOICE, OK, STEP, go  # noqa: F401

PAGED = ["pool", "keys", "n_pages", "page", "table", "max_pages", "lengths"]
LATENT = ["q", "H"] + PAGED + STEP + ["mask", "scale"] + CHOICE + ["z", "zt", "ws", "wsb", "stream"]
DECODE = ["qn", "qr", "uk", "uv"] + PAGED + STEP + ["mask", "gate", "scale"] + CHOICE + ["q", "z", "out", "ws", "wsb", "stream"]


@pytest.mark.parametrize("name,order", [("mla_sparse_latent", LATENT), ("mla_sparse_decode", DECODE)])
def test_a_bad_choice_is_refused_without_nodes(go, name, order):  # noqa: F811
    for bad in (dict(blocks=0), dict(blocks=-1), dict(first=-1), dict(recent=-1), dict(first=7, recent=2),
                dict(first=2**31 - 1, recent=2**31 - 1)):
        assert go(name, order, **bad) == BAD and go(name, order, total=0, **bad) == BAD, bad
    before = kda.kda_launch_count()
    assert go(name, order, total=0) == OK and go(name, order, total=0, n=0) == OK
    assert go(name, order, total=0, first=6, recent=2) == OK
    assert kda.kda_launch_count() == before
