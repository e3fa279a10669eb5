"""GPU: eviction and trimming against lists: the kept positions, the rows' bits in every layer, the
weights, lengths, tables and counts are exact."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_gb300 import kda
from tests import _gpu
from tests import _long_ref as long
from tests import _tree_ref as ref

pytestmark = pytest.mark.gpu


class Cache:
    def __init__(self, lengths, *, page=16, layers=2, seed=0, spare=3, kind="random", width=None):
        g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        self.lengths, self.page, self.layers = list(lengths), page, layers
        needs = [-(-n // page) for n in lengths]
        self.n_pages = sum(needs) + spare
        order = [int(x) for x in rng.permutation(self.n_pages)]
        most = max(max(needs), 1)
        self.table, at = [], 0
        for k in needs:
            self.table.append(order[at:at + k] + [-1] * (most - k))
            at += k
        self.held = needs
        self.refs = [0] * self.n_pages
        for row in self.table:
            for p in row:
                if p >= 0:
                    self.refs[p] = 1
        self.pool = torch.randint(-2**15, 2**15, (layers, self.n_pages, page, 576), generator=g, dtype=torch.int16)
        n, width = len(lengths), width or most * page
        if kind == "random":
            self.w = torch.rand(n, width, generator=g)
        elif kind == "ties":
            self.w = torch.randint(0, 4, (n, width), generator=g).float() - 1.0
        elif kind == "same":
            self.w = torch.full((n, width), 0.25)
        else:  # close together: the last bits decide, over any number of them
            most = {"close": 300, "near": 6000, "apart": 1 << 16}[kind]
            self.w = 1.0 + torch.randint(0, most, (n, width), generator=g).float() * 2.0**-23

    def run(self, budget, *, first=0, recent=0, refs="own", new="aside", in_place_lengths=False):
        _gpu.lib()
        n = len(self.lengths)
        d = dict(pool=self.pool.view(torch.bfloat16).cuda(), w=self.w.cuda(), lengths=ref.i32(self.lengths))
        d["kept"] = torch.full((n, budget), 77, dtype=torch.int32, device="cuda")
        d["new_lengths"] = d["lengths"] if in_place_lengths else torch.full((n,), 77, dtype=torch.int32, device="cuda")
        d["new_w"] = {"aside": torch.full_like(d["w"], 9.0), "own": d["w"], "none": None}[new]
        kda.mla_cache_evict(d["pool"], ref.i32(self.table), d["lengths"], d["w"], d["kept"], d["new_lengths"], d["new_w"],
                            first=first, recent=recent, refcount=ref.i32(self.refs) if refs == "own" else refs)
        torch.cuda.synchronize()
        return d

    def check(self, d, budget, *, first=0, recent=0, refused=(), new="aside"):
        pool, w = self.pool.clone(), self.w.numpy()
        for n, x in enumerate(self.lengths):
            kept = d["kept"][n].tolist()
            got_w = None if d["new_w"] is None else d["new_w"][n].cpu().numpy()
            rest = w[n] if new == "own" else np.full_like(w[n], 9.0)
            if n in refused:
                assert kept == [-1] * budget and int(d["new_lengths"][n]) == x
                if got_w is not None and 0 <= x <= len(w[n]):
                    assert np.array_equal(got_w[:x], w[n, :x], equal_nan=True)
                continue
            want = long.choose(w[n].tolist(), x, first, recent, budget)
            assert kept == want + [-1] * (budget - len(want)), f"sequence {n}"
            assert int(d["new_lengths"][n]) == len(want)
            for j, t in enumerate(want):
                pool[:, self.table[n][j // self.page], j % self.page] = self.pool[:, self.table[n][t // self.page], t % self.page]
            if got_w is not None:
                assert np.array_equal(got_w[:len(want)], w[n, want], equal_nan=True)
                assert not got_w[len(want):x].any() and np.array_equal(got_w[x:], rest[x:], equal_nan=True)
        assert torch.equal(d["pool"].view(torch.int16).cpu(), pool)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kind", ["random", "ties", "same", "close", "near", "apart"])
def test_ragged_lengths(page, kind):
    c = Cache([0, 1, 39, 40, 41, 63, 64, 300, 700, 1025], page=page, seed=page, kind=kind)
    for budget, first, recent in ((40, 0, 0), (40, 4, 8), (40, 40, 0), (40, 0, 40), (1, 0, 0), (64, 3, 60), (2000, 1, 1)):
        c.check(c.run(budget, first=first, recent=recent), budget, first=first, recent=recent)
    kda.kda_check_device_error()


@pytest.mark.parametrize("new", ["aside", "own", "none"])
@pytest.mark.parametrize("in_place", [False, True])
def test_outputs_in_place(new, in_place):
    c = Cache([500, 90, 100, 3000], seed=5, layers=1)
    c.check(c.run(100, first=2, recent=5, new=new, in_place_lengths=in_place) if not in_place else
            self_lengths(c, new), 100, first=2, recent=5, new=new)


def self_lengths(c, new):
    d = c.run(100, first=2, recent=5, new=new, in_place_lengths=True)
    assert d["lengths"] is d["new_lengths"]
    return d


@pytest.mark.parametrize("kind", ["ties", "near", "apart", "random"])
@pytest.mark.parametrize("n,length", [(1, 9000), (2, 20001), (1, 70001), (40, 9000)])
def test_long_sequences_by_clusters(n, length, kind):
    """One to eight CTAs a sequence, with many equal weights or such as differ in their last bits."""
    c = Cache([length - 7 * i for i in range(n)], layers=1, page=64, seed=n, kind=kind)
    for budget in (length // 3, length - 400):
        c.check(c.run(budget, first=4, recent=32, new="own"), budget, first=4, recent=32, new="own")


@pytest.mark.parametrize("width", [1025, 1026, 1027, 1039])
def test_rows_of_weights_of_any_width(width):
    c = Cache([1025, 700, 1, 999], layers=1, seed=width, width=width)
    for budget in (1, 130, 513, 1024):
        c.check(c.run(budget, first=1, new="own"), budget, first=1, new="own")


@pytest.mark.parametrize("bit", range(0, 32, 3))
def test_every_bit_counts(bit):
    """Weights that differ in a few neighbouring bits alone, whichever they are."""
    c = Cache([900, 333], layers=1, seed=bit)
    g = torch.Generator().manual_seed(bit)
    span = min(4, 32 - bit)
    low = torch.randint(0, 1 << span, c.w.shape, generator=g) << bit
    c.w = (low ^ 0x3F800000 if bit < 22 else low).to(torch.int64).to(torch.int32).view(torch.float32)
    for budget in (100, 200, 320):
        c.check(c.run(budget, recent=7), budget, recent=7)


def test_special_values():
    """Infinities order as numbers, -0 equals 0, NaN is below everything, subnormals count."""
    c = Cache([64], seed=9)
    v = [float("nan"), float("inf"), -float("inf"), -0.0, 0.0, 1e-45, -1e-45, 1.0]
    c.w[0, :64] = torch.tensor((v * 8)[:64])
    for budget in range(1, 64, 5):
        c.check(c.run(budget), budget)


def test_many_layers_and_rows_that_do_not_move():
    c = Cache([400, 260], layers=11, page=32, seed=13)
    c.w[0, :200] = 5.0  # the first 200 stay where they are
    c.check(c.run(256, recent=16), 256, recent=16)


def test_shared_pages_are_not_written():
    """A shared prefix that stays where it is may be shared; one that rows move into is refused."""
    c = Cache([200, 200, 200], page=16, seed=14)
    c.w[0, :64] = 5.0             # pages 0 .. 3 stay
    c.refs[c.table[0][2]] = 2
    c.w[1, :64] = 5.0
    c.w[1, 10] = -1.0             # a gap inside page 0
    c.refs[c.table[1][2]] = 2
    c.refs[c.table[2][11]] = 3    # only read: behind the budget
    d = c.run(100, recent=4)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_check_device_error()
    assert e.value.status == kda.KDA_ERR_BAD_INDEX
    c.check(d, 100, recent=4, refused=(1,))
    c.check(c.run(100, recent=4, refs=None), 100, recent=4)  # nobody counts
    kda.kda_check_device_error()


def test_bad_lengths_and_pages_are_refused_and_reported():
    c = Cache([200, 200, 200, 200, 50], page=16, seed=15)
    c.lengths[0], c.lengths[1] = -3, 10**6
    c.table[2][12] = -1           # page of the last positions
    c.table[3][0] = 10**6         # not touched: the first sixteen stay
    c.w[3, :16] = 5.0
    for new in ("aside", "own"):
        d = c.run(100, recent=4, new=new)
        with pytest.raises(kda.KdaError) as e:
            kda.kda_check_device_error()
        assert e.value.status == kda.KDA_ERR_BAD_INDEX
        kept = [d["kept"][n].tolist() for n in range(5)]
        assert kept[0] == kept[1] == kept[2] == [-1] * 100 and kept[3][:16] == list(range(16))
        assert d["new_lengths"].tolist() == [-3, 10**6, 200, 100, 50]
    c = Cache([200, 90], page=16, seed=16, width=199)  # the weights hold one position less
    d = c.run(80)
    with pytest.raises(kda.KdaError):
        kda.kda_check_device_error()
    c.check(d, 80, refused=(0,))


@pytest.mark.parametrize("page", [16, 256])
def test_trim(page):
    _gpu.lib()
    p = ref.Pages(60, 5, 12, page)
    slots = [0, 1, 2, 3, 4]
    p.lengths = [0] * 5
    p.reserve(slots, [5 * page, 3 * page + 1, 9 * page, 1, 0])
    table, refs, held = ref.i32(p.table), ref.i32(p.refs), ref.i32(p.held)
    refs[p.table[2][8]] = 2  # also named elsewhere
    lengths = ref.i32([2 * page + 1, 3 * page + 1, page, 0, 0])
    kda.mla_pages_trim(page, refs, table, held, lengths, ref.i32([2, 0, 1, 2, 4, 3]))
    kda.kda_check_device_error()
    assert held.tolist() == [3, 4, 1, 0, 0]
    for s in range(5):
        assert table[s].tolist() == [x if j < held[s] else -1 for j, x in enumerate(p.table[s])]
    left = {x for s in range(5) for x in table[s].tolist() if x >= 0}
    assert refs.tolist() == [1 if x in left or x == p.table[2][8] else 0 for x in range(60)]
    # errors: an index out of range, a bad length, fewer pages than the length needs
    for lengths, slot in (([page] * 5, 5), ([-1] * 5, 0), ([10 * page] * 5, 1)):
        before = [t.clone() for t in (refs, table, held)]
        kda.mla_pages_trim(page, refs, table, held, ref.i32(lengths), ref.i32([slot]))
        with pytest.raises(kda.KdaError) as e:
            kda.kda_check_device_error()
        assert e.value.status == kda.KDA_ERR_BAD_INDEX
        assert all(torch.equal(a, b) for a, b in zip(before, (refs, table, held)))


def test_same_bits_every_time():
    c = Cache([5000, 3000], layers=2, page=32, seed=17, kind="ties")
    a, b = c.run(1000, recent=100), c.run(1000, recent=100)
    assert torch.equal(a["pool"].view(torch.int16), b["pool"].view(torch.int16))  # random bits, NaN among them
    assert all(torch.equal(a[k], b[k]) for k in ("kept", "new_lengths", "new_w"))
