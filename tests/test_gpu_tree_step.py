"""GPU: a whole verification step over paged caches captured into one graph, on two streams."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from hybrid_linear_attention_gb300 import kda
from tests import _gpu
from tests import _tree_ref as ref
from tests.test_gpu_tree_kda import make

pytestmark = pytest.mark.gpu
COUNTS, H, PAGE, LAYERS, TOTAL = [5, 1, 7, 3], 64, 32, 2, 16


class Step:
    """Buffers of a step for four sequences; fill() loads a state and inputs, run() enqueues the step."""

    def __init__(self):
        dev = dict(device="cuda")
        self.p = kda.params(H=H)
        self.pool = torch.zeros(LAYERS, 40, PAGE, 576, dtype=torch.bfloat16, **dev)
        self.refs, self.held, self.lengths = (torch.zeros(n, dtype=torch.int32, **dev) for n in (40, 4, 4))
        self.table = torch.full((4, 8), -1, dtype=torch.int32, **dev)
        self.cu, self.extra = ref.i32([0] + [int(x) for x in np.cumsum(COUNTS)]), ref.i32(COUNTS)
        self.parent = torch.zeros(TOTAL, dtype=torch.int32, **dev)
        self.accept, self.slots = ref.i32([0] * 4), ref.i32([0, 1, 2, 3])
        self.rows = torch.zeros(LAYERS, TOTAL, 576, dtype=torch.bfloat16, **dev)
        self.q = torch.zeros(TOTAL, H, 576, dtype=torch.bfloat16, **dev)
        self.z = torch.zeros(LAYERS, TOTAL, H, 512, **dev)
        self.mask = torch.zeros(TOTAL, dtype=torch.int64, **dev)
        self.x = torch.zeros(TOTAL, 3 * H * 128, dtype=torch.bfloat16, **dev)
        self.w = torch.zeros(3 * H * 128, 4, dtype=torch.bfloat16, **dev)
        self.tail = torch.zeros(4, 3, 3 * H * 128, dtype=torch.bfloat16, **dev)
        self.g, self.beta = torch.zeros(TOTAL, H, 128, **dev), torch.zeros(TOTAL, H, **dev)
        self.state = torch.zeros(4, H, 128, 128, **dev)
        self.out = torch.zeros(TOTAL, H, 128, dtype=torch.bfloat16, **dev)
        self.ws = torch.empty(kda.mla_tree_workspace_size(4, TOTAL, H), dtype=torch.uint8, **dev)
        self.pages = torch.empty(kda.mla_pages_workspace_size(4), dtype=torch.uint8, **dev)
        self.side = torch.cuda.Stream()

    def fill(self, seed):
        m = make(COUNTS, H, 128, seed=seed, slots=[0, 1, 2, 3], n_slots=4)
        rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.x.copy_(m["x"]), self.w.copy_(m["conv_w"]), self.tail.copy_(m["conv_state"]), self.state.copy_(m["state"])
        self.g.copy_(m["g"]), self.beta.copy_(m["beta"]), self.parent.copy_(ref.i32(m["parent"]))
        self.rows.copy_(torch.randn(self.rows.shape, generator=g)), self.q.copy_(torch.randn(self.q.shape, generator=g))
        self.pool.copy_(torch.randn(self.pool.shape, generator=g))
        lengths = [int(x) for x in rng.integers(0, 150, 4)]
        pages = [-(-n // PAGE) for n in lengths]
        order = [int(x) for x in rng.permutation(40)]
        table, refs = [], [0] * 40
        for k in pages:
            table.append([order.pop() for _ in range(k)])
            for page in table[-1]:
                refs[page] = 1
        self.table.copy_(ref.i32([r + [-1] * (8 - len(r)) for r in table]))
        self.refs.copy_(ref.i32(refs)), self.held.copy_(ref.i32(pages)), self.lengths.copy_(ref.i32(lengths))
        self.accept.copy_(ref.i32([int(rng.integers(-1, c)) for c in COUNTS]))
        for t in (self.z, self.out, self.mask):
            t.zero_()

    def run(self):
        args = (self.p, self.x, self.w, self.tail, self.g, self.beta, self.state, self.cu, self.parent)
        main = torch.cuda.current_stream()
        kda.mla_pages_reserve(PAGE, self.refs, self.table, self.held, self.lengths, self.slots, self.extra,
                              workspace=self.pages)
        kda.mla_cache_append(self.pool, self.table, self.lengths, self.cu, self.rows)
        self.side.wait_stream(main)
        with torch.cuda.stream(self.side):
            kda.kda_tree_verify(*args, self.out, max_nodes=7)
            kda.kda_tree_accept(*args, self.accept)
        kda.mla_tree_mask(self.parent, self.cu, self.mask)
        for layer in range(LAYERS):  # the same workspace, one after another
            kda.mla_tree_latent(self.q, self.pool[layer], self.table, self.lengths, self.cu, self.z[layer],
                                mask=self.mask, workspace=self.ws)
        main.wait_stream(self.side)
        kda.mla_cache_accept(self.pool, self.table, self.lengths, self.cu, self.parent, self.accept, self.lengths)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.pool, self.refs, self.table, self.held, self.lengths, self.mask, self.z,
                                    self.tail, self.state, self.out)]


def test_a_captured_step_gives_the_eager_bits():
    _gpu.lib()
    s, want = Step(), []
    for seed in (1, 2, 3):
        s.fill(seed)
        torch.cuda.synchronize()
        s.run()
        kda.kda_check_device_error()
        want.append(s.results())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (3, 1, 2):
        s.fill(seed)
        torch.cuda.synchronize()
        graph.replay()
        kda.kda_check_device_error()
        for a, b in zip(s.results(), want[seed - 1]):
            assert torch.equal(a, b)


def test_the_first_calls_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import torch\n"
            "from tests.test_gpu_tree_step import Step, kda\n"
            "s = Step(); s.fill(4); torch.cuda.synchronize()\n"
            "graph = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(graph): s.run()\n"
            "graph.replay(); kda.kda_check_device_error(); a = s.results()\n"
            "s.fill(4); torch.cuda.synchronize(); s.run(); kda.kda_check_device_error()\n"
            "assert all(torch.equal(x, y) for x, y in zip(a, s.results()))\n")
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
