"""The tree-verification calls refuse bad arguments on the host, before any CUDA call."""
import ctypes

import pytest
import torch

from hybrid_linear_attention_gb300 import build as kbuild
from hybrid_linear_attention_gb300 import kda

BAD, UNSUPPORTED, WS, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE, kda.KDA_OK


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def _call(lib, name, order, defaults, **kw):
    a = dict(defaults, **kw)
    assert set(kw) <= set(order)
    return getattr(lib, name)(*(a[k] for k in order))


TREE = ["p", "x", "w", "cs", "g", "beta", "state", "n_slots", "slots", "cu", "parent", "n", "total"]
TREE_D = dict(x=16, w=16, cs=16, g=16, beta=16, state=16, n_slots=4, slots=None, cu=16, parent=16, n=2, total=5,
              most=8, gate=None, nw=None, out=16, accept=16, stream=None)


@pytest.mark.parametrize("name,tail", [("kda_tree_verify", ["most", "gate", "nw", "out", "stream"]),
                                       ("kda_tree_accept", ["accept", "stream"])])
def test_kda_tree_calls(lib, name, tail):
    p = kda.params()
    d = dict(TREE_D, p=ctypes.byref(p))
    go = lambda **kw: _call(lib, name, TREE + tail, d, **kw)  # noqa: E731
    for k in ("x", "w", "cs", "g", "beta", "state", "cu", "parent"):
        assert go(**{k: None}) == BAD and go(**{k: 8}) == BAD, k
    assert go(p=None) == BAD
    assert go(n=-1) == BAD and go(n=65536) == BAD and go(total=-1) == BAD and go(total=2**22 + 1) == BAD
    assert go(n=0) == BAD and go(n_slots=1) == BAD and go(slots=8) == BAD
    assert go(total=0) == OK and go(total=0, n=0, x=None) == OK
    if name == "kda_tree_verify":
        assert go(most=0) == BAD and go(most=65) == BAD and go(out=None) == BAD and go(gate=8) == BAD and go(nw=4) == BAD
    else:
        assert go(accept=None) == BAD
    assert go(p=ctypes.byref(kda.params(d=64))) == UNSUPPORTED


PAGED = ["pool", "n_pages", "page", "table", "max_pages", "lengths"]


def test_tree_attention(lib):
    size = kda.mla_tree_workspace_size(2, 5, 64)
    assert size > 0
    assert kda.mla_tree_workspace_size(0, 5) == kda.mla_tree_workspace_size(2, 0) == kda.mla_tree_workspace_size(2, 5, 129) == 0
    order = ["q", "H"] + PAGED + ["cu", "n", "total", "mask", "scale", "z", "zt", "ws", "wsb", "stream"]
    d = dict(q=16, H=64, pool=16, n_pages=4, page=64, table=16, max_pages=2, lengths=16, cu=16, n=2, total=5, mask=None,
             scale=0.1, z=16, zt=0, ws=16, wsb=size, stream=None)
    go = lambda **kw: _call(lib, "mla_tree_latent", order, d, **kw)  # noqa: E731
    for k in ("q", "pool", "table", "lengths", "cu", "z"):
        assert go(**{k: None}) == BAD and go(**{k: 8}) == BAD, k
    assert go(H=0) == BAD and go(H=129) == BAD and go(n=-1) == BAD and go(total=-1) == BAD and go(n=0) == BAD
    assert go(scale=0.0) == BAD and go(scale=float("nan")) == BAD and go(zt=2) == BAD and go(mask=8) == BAD
    assert go(n_pages=0) == BAD and go(max_pages=0) == BAD and go(max_pages=2**20 + 1) == BAD
    for page in (1, 8, 24, 48, 512):
        assert go(page=page) == UNSUPPORTED
    assert go(ws=None, wsb=0) == WS and go(wsb=size - 1) == WS and go(ws=8) == BAD
    assert go(total=0, q=None) == OK
    order = ["qn", "qr", "uk", "uv"] + PAGED + ["cu", "n", "total", "mask", "gate", "scale", "q", "z", "out", "ws", "wsb",
                                                "stream"]
    d.update(qn=16, qr=16, uk=16, uv=16, gate=16, out=16)
    go = lambda **kw: _call(lib, "mla_tree_decode", order, d, **kw)  # noqa: E731
    for k in ("q", "pool", "table", "lengths", "cu", "z"):
        assert go(**{k: None}) == BAD, k
    assert go(wsb=size - 1) == WS and go(total=0) == OK
    assert lib.mla_tree_mask(16, 16, 2, -1, 16, None) == BAD and lib.mla_tree_mask(None, 16, 2, 3, 16, None) == BAD
    assert lib.mla_tree_mask(16, 16, 2, 3, None, None) == BAD and lib.mla_tree_mask(None, None, 2, 0, None, None) == OK


LAYERS = ["pool", "layers", "n_pages", "page", "table", "max_pages", "lengths"]
LAYERS_D = dict(pool=16, layers=9, n_pages=4, page=64, table=16, max_pages=2, lengths=16, stream=None)


def test_cache_rows(lib):
    d = dict(LAYERS_D, cu=16, n=2, total=5, rows=16, parent=16, accept=16, new=16)
    calls = (("mla_cache_append", LAYERS + ["cu", "n", "total", "rows", "stream"], ("pool", "table", "lengths", "cu", "rows")),
             ("mla_cache_accept", LAYERS + ["cu", "n", "total", "parent", "accept", "new", "stream"],
              ("pool", "table", "lengths", "cu", "parent", "accept", "new")))
    for name, order, pointers in calls:
        go = lambda **kw: _call(lib, name, order, d, **kw)  # noqa: E731, B023
        for k in pointers:
            assert go(**{k: None}) == BAD and go(**{k: 8}) == BAD, (name, k)
        assert go(layers=0) == BAD and go(n_pages=0) == BAD and go(page=40) == UNSUPPORTED and go(n=-1) == BAD
        assert go(total=-1) == BAD and go(max_pages=0) == BAD
    assert _call(lib, *calls[0][:2], d, total=0) == OK and _call(lib, *calls[1][:2], d, n=0) == OK


def test_pages(lib):
    assert kda.mla_pages_workspace_size(0) == 0 == kda.mla_pages_workspace_size(65536)
    size = kda.mla_pages_workspace_size(3)
    book = ["refs", "table", "max_pages", "held", "lengths", "n_slots"]
    d = dict(LAYERS_D, refs=16, held=16, n_slots=4, slots=16, src=16, dst=16, extra=16, n=3, ws=16, wsb=size)
    calls = {"mla_pages_free": ["n_pages"] + book + ["slots", "n", "stream"],
             "mla_pages_fork": ["pool", "layers", "n_pages", "page"] + book + ["src", "dst", "n", "ws", "wsb", "stream"],
             "mla_pages_reserve": ["n_pages", "page"] + book + ["slots", "extra", "n", "ws", "wsb", "stream"]}
    for name, order in calls.items():
        go = lambda **kw: _call(lib, name, order, d, **kw)  # noqa: E731, B023
        for k in set(order) & {"pool", "refs", "table", "held", "lengths", "slots", "src", "dst", "extra"}:
            assert go(**{k: None}) == BAD and go(**{k: 8}) == BAD, (name, k)
        assert go(n=-1) == BAD and go(n=65536) == BAD and go(n_slots=0) == BAD and go(n_pages=0) == BAD
        assert go(n=0) == OK
        if "ws" in order:
            assert go(ws=None, wsb=0) == WS and go(wsb=size - 1) == WS
    order = ["pool", "layers", "n_pages", "page", "src", "dst", "n", "stream"]
    go = lambda **kw: _call(lib, "mla_pages_copy", order, d, **kw)  # noqa: E731
    assert go(pool=None) == BAD and go(src=None) == BAD and go(dst=None) == BAD and go(n=-1) == BAD and go(n=0) == OK
    assert go(page=3) == UNSUPPORTED


def test_page_copies_are_limited(lib):
    go = lambda n: lib.mla_pages_copy(16, 9, 4, 64, 16, 16, n, None)  # noqa: E731
    assert go(8193) == BAD and go(2**31 - 1) == BAD and go(0) == OK


def test_the_binding_checks_shapes(lib):
    p = kda.params(H=2)
    t = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError, match="x_raw"):
        kda.kda_tree_verify(p, t(5, 700), t(768, 4), t(3, 3, 768), t(5, 2, 128), t(5, 2), t(3, 2, 128, 128),
                            t(3, dtype=torch.int32), t(5, dtype=torch.int32), t(5, 2, 128))
    with pytest.raises(ValueError, match="z: expected shape"):
        kda.mla_tree_latent(t(5, 2, 576), t(4, 16, 576), t(2, 3), t(2), t(3), t(5, 2, 511))
    with pytest.raises(ValueError, match="fewer rows"):
        kda.mla_tree_latent(t(5, 2, 576), t(4, 16, 576), t(1, 3), t(1), t(3), t(5, 2, 512))
    with pytest.raises(ValueError, match="n_layers"):
        kda.mla_cache_append(t(4, 16, 576), t(2, 3), t(2), t(3), t(4, 5, 576))
    assert kda.status_string(-8).startswith("KDA_ERR_NO_PAGES")


def test_reserve_takes_the_page_sizes_of_the_pool(lib):
    size = kda.mla_pages_workspace_size(3)
    go = lambda page: lib.mla_pages_reserve(4, page, 16, 16, 2, 16, 16, 4, 16, 16, 3, 16, size, None)  # noqa: E731
    assert go(0) == BAD and go(-16) == BAD
    for page in (1, 8, 24, 48, 255, 512):
        assert go(page) == UNSUPPORTED
