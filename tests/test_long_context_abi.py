"""The long-context calls refuse bad arguments on the host, before any CUDA call."""
import pytest

from hybrid_linear_attention_gb300 import build as kbuild
from hybrid_linear_attention_gb300 import kda

BAD, UNSUPPORTED, WS, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE, kda.KDA_OK
PAGED = ["pool", "n_pages", "page", "table", "max_pages", "lengths"]
LAYERS = ["pool", "layers", "n_pages", "page", "table", "max_pages", "lengths"]
STEP = ["cu", "n", "total"]
CHOICE = ["blocks", "first", "recent", "scores", "stride", "sel", "sel_pages", "cut"]
D = dict(q=16, H=64, pool=16, keys=16, layers=2, n_pages=4, page=64, table=16, max_pages=2, lengths=16, cu=16, n=2, total=5,
         mask=None, scale=0.1, z=16, zt=0, lse=16, ws=16, wsb=1 << 40, stream=None, u=None, w=16, stride=128, refs=None,
         budget=10, first=1, recent=2, kept=16, new_lengths=16, new_w=None, held=16, slots=16, n_slots=4, refcount=16,
         before=16, parent=16, accept=16, scores=16, blocks=8, sel=16, sel_pages=12, cut=16, qn=16, qr=16, uk=16, uv=16, gate=16, out=16)


@pytest.fixture(scope="module")
def go():
    kbuild.build()
    lib = kda.load()

    def call(name, order, **kw):
        assert set(kw) <= set(order)
        return getattr(lib, name)(*(dict(D, **kw)[k] for k in order))
    return call


def pointers(go, name, order, needed, optional=()):
    for k in needed:
        assert go(name, order, **{k: None}) == BAD and go(name, order, **{k: 8}) == BAD, k
    for k in optional:
        assert go(name, order, **{k: 8}) == BAD, k


def geometry(go, name, order):
    for page in (1, 8, 24, 48, 512):
        assert go(name, order, page=page) == UNSUPPORTED
    assert go(name, order, page=0) == BAD and go(name, order, max_pages=0) == BAD
    assert go(name, order, max_pages=2**20 + 1) == BAD and go(name, order, n=-1) == BAD and go(name, order, n=65536) == BAD


def test_attention_with_lse(go):
    order = ["q", "H"] + PAGED + STEP + ["mask", "scale", "z", "zt", "lse", "ws", "wsb", "stream"]
    pointers(go, "mla_tree_latent_lse", order, ("q", "pool", "table", "lengths", "cu", "z", "lse"), ("mask", "ws"))
    geometry(go, "mla_tree_latent_lse", order)
    size = kda.mla_tree_workspace_size(2, 5, 64)
    assert go("mla_tree_latent_lse", order, wsb=size - 1) == WS and go("mla_tree_latent_lse", order, total=0, lse=None) == OK
    order = ["qn", "qr", "uk", "uv"] + PAGED + STEP + ["mask", "gate", "scale", "q", "z", "out", "lse", "ws", "wsb", "stream"]
    pointers(go, "mla_tree_decode_lse", order, ("qn", "qr", "uk", "uv", "gate", "out", "q", "z", "lse"))
    assert go("mla_tree_decode_lse", order, wsb=size - 1) == WS


def test_cache_weights(go):
    order = ["q", "H"] + PAGED + STEP + ["mask", "u", "lse", "scale", "w", "stride", "stream"]
    name = "mla_cache_weights"
    pointers(go, name, order, ("q", "pool", "table", "lengths", "cu", "lse", "w"), ("mask", "u"))
    geometry(go, name, order)
    assert go(name, order, H=0) == BAD and go(name, order, H=129) == BAD and go(name, order, stride=0) == BAD
    assert go(name, order, total=-1) == BAD and go(name, order, total=2**22 + 1) == BAD and go(name, order, n=0) == BAD
    assert go(name, order, scale=0.0) == BAD and go(name, order, scale=float("nan")) == BAD
    assert go(name, order, total=0, q=None) == OK


def test_weights_accept(go):
    order = ["w", "stride", "lengths", "cu", "n", "total", "parent", "accept", "stream"]
    name = "mla_weights_accept"
    pointers(go, name, order, ("w", "lengths", "cu", "parent", "accept"))
    assert go(name, order, stride=0) == BAD and go(name, order, n=-1) == BAD and go(name, order, n=65536) == BAD
    assert go(name, order, total=-1) == BAD and go(name, order, total=2**22 + 1) == BAD
    assert go(name, order, total=0, w=None) == OK and go(name, order, n=0, w=None) == OK


def test_cache_evict(go):
    order = LAYERS + ["refs", "n", "w", "stride", "budget", "first", "recent", "kept", "new_lengths", "new_w", "stream"]
    name = "mla_cache_evict"
    pointers(go, name, order, ("pool", "table", "lengths", "w", "kept", "new_lengths"), ("refs", "new_w"))
    geometry(go, name, order)
    assert go(name, order, layers=0) == BAD and go(name, order, n_pages=0) == BAD and go(name, order, stride=0) == BAD
    assert go(name, order, budget=0) == BAD and go(name, order, first=-1) == BAD and go(name, order, recent=-1) == BAD
    assert go(name, order, first=8, recent=3) == BAD and go(name, order, first=2**31 - 1, recent=2**31 - 1) == BAD
    assert go(name, order, n=0) == OK


def test_pages_trim(go):
    order = ["n_pages", "page", "refcount", "table", "max_pages", "held", "lengths", "n_slots", "slots", "n", "stream"]
    pointers(go, "mla_pages_trim", order, ("refcount", "table", "held", "lengths", "slots"))
    geometry(go, "mla_pages_trim", order)
    assert go("mla_pages_trim", order, n_slots=0) == BAD and go("mla_pages_trim", order, n_pages=0) == BAD
    assert go("mla_pages_trim", order, n=0, slots=None) == OK


def test_block_keys(go):
    order = ["pool", "layers", "n_pages", "page", "table", "max_pages", "before", "lengths", "n", "keys", "stream"]
    pointers(go, "mla_block_keys", order, ("pool", "table", "before", "lengths", "keys"))
    geometry(go, "mla_block_keys", order)
    assert go("mla_block_keys", order, n=0) == OK


def test_block_scores(go):
    size = kda.mla_block_scores_workspace_size(5, 64, 2)
    assert size > 0
    assert kda.mla_block_scores_workspace_size(0, 64, 2) == kda.mla_block_scores_workspace_size(5, 129, 2) == 0
    assert kda.mla_block_scores_workspace_size(5, 64, 0) == kda.mla_block_scores_workspace_size(5, 64, 2**20 + 1) == 0
    order = ["q", "H", "keys", "n_pages", "page", "table", "max_pages", "lengths"] + STEP + ["scale", "scores", "stride", "ws",
                                                                                              "wsb", "stream"]
    name = "mla_block_scores"
    pointers(go, name, order, ("q", "keys", "table", "lengths", "cu", "scores"), ("ws",))
    geometry(go, name, order)
    assert go(name, order, stride=1) == BAD and go(name, order, wsb=size - 1) == WS and go(name, order, ws=None) == WS
    assert go(name, order, total=0) == OK


def test_block_select(go):
    order = ["scores", "stride", "page", "table", "max_pages", "lengths"] + STEP + ["blocks", "first", "recent", "sel",
                                                                                    "sel_pages", "cut", "stream"]
    name = "mla_block_select"
    pointers(go, name, order, ("scores", "table", "lengths", "cu", "sel", "cut"))
    geometry(go, name, order)
    assert go(name, order, stride=1) == BAD and go(name, order, sel_pages=0) == BAD and go(name, order, blocks=0) == BAD
    assert go(name, order, first=7, recent=2) == BAD and go(name, order, first=-1) == BAD and go(name, order, n=0) == OK


def test_sparse(go):
    size = kda.mla_sparse_workspace_size(2, 5, 64, 2)
    assert size >= max(kda.mla_block_scores_workspace_size(5, 64, 2), kda.mla_tree_workspace_size(2, 5, 64)) > 0
    assert kda.mla_sparse_workspace_size(0, 5, 64, 2) == kda.mla_sparse_workspace_size(2, 5, 64, 0) == 0
    paged = ["pool", "keys", "n_pages", "page", "table", "max_pages", "lengths"]
    order = ["q", "H"] + paged + STEP + ["mask", "scale"] + CHOICE + ["z", "zt", "ws", "wsb", "stream"]
    name = "mla_sparse_latent"
    pointers(go, name, order, ("q", "pool", "keys", "table", "lengths", "cu", "scores", "sel", "cut", "z"), ("mask", "ws"))
    geometry(go, name, order)
    assert go(name, order, blocks=2) == BAD and go(name, order, sel_pages=0) == BAD and go(name, order, stride=1) == BAD
    assert go(name, order, wsb=size - 1) == WS and go(name, order, total=0) == OK and go(name, order, zt=2) == BAD
    order = ["qn", "qr", "uk", "uv"] + paged + STEP + ["mask", "gate", "scale"] + CHOICE + ["q", "z", "out", "ws", "wsb", "stream"]
    pointers(go, "mla_sparse_decode", order, ("qn", "qr", "uk", "uv", "pool", "keys", "gate", "q", "z", "out"))
    assert go("mla_sparse_decode", order, wsb=size - 1) == WS and go("mla_sparse_decode", order, total=0) == OK
