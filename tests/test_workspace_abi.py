"""The tree attention's workspace: the partial sums of 160 row tiles of 128 rows (512 values, a maximum and a
normaliser each) and 32 bytes a pair of CTAs.  Buffers of that size were enough before the calls that leave
log-sums came, and are for all of them."""
from hybrid_linear_attention_gb300 import kda
from tests.test_long_context_abi import PAGED, STEP, WS, go  # noqa: F401

SIZE = 160 * 128 * (512 + 2) * 4 + 80 * 32


def test_a_buffer_of_the_size_asked_before_is_taken(go):  # noqa: F811
    latent = ["q", "H"] + PAGED + STEP + ["mask", "scale", "z", "zt"]
    decode = ["qn", "qr", "uk", "uv"] + PAGED + STEP + ["mask", "gate", "scale", "q", "z", "out"]
    assert kda.mla_tree_workspace_size(2, 5, 64) <= SIZE
    # a byte less than is asked for is too small, for each of the calls
    tail = ["ws", "wsb", "stream"]
    for name, order in (("mla_tree_latent", latent + tail), ("mla_tree_decode", decode + tail),
                        ("mla_tree_latent_lse", latent + ["lse"] + tail), ("mla_tree_decode_lse", decode + ["lse"] + tail)):
        assert go(name, order, wsb=kda.mla_tree_workspace_size(2, 5, 64) - 1) == WS, name
