"""Calls captured into CUDA graphs: what a replay computes is what the call
computes, however often it runs and whatever runs beside it."""
import numpy as np
import pytest

from tests import _gpu

pytestmark = pytest.mark.gpu
PAIRS = 76


def rand(*shape, seed, std=1.0):
    rng = np.random.default_rng([seed, *shape])
    return _gpu.to_dev((rng.standard_normal(shape) * std).astype(np.float32))


def empty(*shape):
    import torch
    return torch.empty(shape, device=_gpu.device())


class Product:
    """C = A B^T by emu_sgemm alone in a graph."""
    kernels = 1

    def __init__(self, M, N, K, mode):
        self.size, self.mode = (M, N, K), mode
        self.a, self.b, self.c = empty(M, K), empty(N, K), empty(M, N)
        self.inputs, self.outputs = [self.a, self.b], [self.c]

    def draw(self, seed):
        M, N, K = self.size
        return [rand(M, K, seed=seed), rand(N, K, seed=seed + 100)]

    def run(self):
        import fp32_emulated_gemm_gb300 as emu
        M, N, K = self.size
        emu.emu_sgemm(emu.MODES[self.mode], 0, 1, M, N, K, 1.0, self.a, K, self.b, K, 0.0, self.c, N)


class GatedForward:
    """emu_gated_fwd alone: the gated epilogue on a split product."""

    def __init__(self, M, F, K, mode):
        self.size, self.mode = (M, F, K), mode
        self.x, self.w, self.d, self.h = empty(M, K), empty(2 * F, K), empty(M, 2 * F), empty(M, F)
        self.inputs, self.outputs = [self.x, self.w], [self.d, self.h]

    def draw(self, seed):
        M, F, K = self.size
        return [rand(M, K, seed=seed), rand(2 * F, K, seed=seed + 100, std=K ** -0.5)]

    def run(self):
        import fp32_emulated_gemm_gb300 as emu
        M, F, K = self.size
        emu.emu_gated_fwd(emu.MODES[self.mode], emu.EMU_ACT_SILU, M, F, K, self.x, K, self.w, K, None, self.d, 2 * F,
                          self.h, F)


class LinearBackward:
    """emu_linear_act_bwd alone: two split products side by side."""

    def __init__(self, M, N, K, mode):
        self.size, self.mode = (M, N, K), mode
        self.dy, self.x, self.w, self.d = empty(M, N), empty(M, K), empty(N, K), empty(M, N)
        self.dz, self.dx, self.dw, self.db = empty(M, N), empty(M, K), empty(N, K), empty(N)
        self.inputs, self.outputs = [self.dy, self.x, self.w, self.d], [self.dz, self.dx, self.dw, self.db]

    def draw(self, seed):
        M, N, K = self.size
        return [rand(M, N, seed=seed), rand(M, K, seed=seed + 100), rand(N, K, seed=seed + 200), rand(M, N, seed=seed + 300)]

    def run(self):
        import fp32_emulated_gemm_gb300 as emu
        M, N, K = self.size
        emu.emu_linear_act_bwd(emu.MODES[self.mode], M, N, K, self.dy, N, self.x, K, self.w, K, self.d, N, self.dz, N,
                               self.dx, K, self.dw, K, self.db)


CASES = {
    "chained_bf16x9": lambda: Product(2000, 2500, 200, "bf16x9"),
    "chained_tf32x3": lambda: Product(2000, 2500, 200, "tf32x3"),
    "split_19_bf16x9": lambda: Product(300, 260, 3000, "bf16x9"),
    "split_32_tf32x3": lambda: Product(256, 256, 4096, "tf32x3"),
    "gated_split": lambda: GatedForward(300, 132, 3000, "bf16x9"),
    "backward_tf32x3": lambda: LinearBackward(1536, 300, 500, "tf32x3"),
    "backward_bf16x9": lambda: LinearBackward(1536, 300, 500, "bf16x9"),
}


def test_the_products_are_the_kinds_named():
    import fp32_emulated_gemm_gb300 as emu
    assert emu.emu_plan_query(2000, 2500, 200, PAIRS)["chain"] == 1
    assert emu.emu_plan_query(300, 260, 3000, PAIRS)["split_a"] == 19
    assert emu.emu_plan_query(256, 256, 4096, PAIRS)["split_a"] == 32


def prepared(name):
    """The case's call, warmed up on the stream that it is then captured on."""
    import torch
    case = CASES[name]()
    for t in case.inputs:
        t.zero_()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        case.run()
    stream.synchronize()
    return case, stream


@pytest.mark.parametrize("name", CASES)
def test_a_graph_clears_the_counters_of_split_products(name):
    """A captured launch has the same epoch in every replay, so the graph has to
    clear the counters that its split and chained products arrive on."""
    from tests import _graphs
    case, stream = prepared(name)
    graph = _graphs.Graph(stream, case.run)
    types = graph.types()
    graph.close()
    assert types.count(_graphs.MEMSET) >= 1, types


@pytest.mark.parametrize("name", CASES)
def test_many_replays_with_new_inputs(name):
    """300 replays (more than an 8-bit count holds), each bit for bit the call
    on the inputs then in place; nothing else runs on the captured stream."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    from tests import _graphs
    case, stream = prepared(name)
    sets = [case.draw(seed) for seed in range(5)]
    want = []
    for data in sets:                     # the calls themselves, on another stream's buffers
        for t, v in zip(case.inputs, data):
            t.copy_(v)
        case.run()
        want.append([t.clone() for t in case.outputs])
    torch.cuda.synchronize()
    graph = _graphs.Graph(stream, case.run)
    with torch.cuda.stream(stream):
        for i in range(300):
            for t, v in zip(case.inputs, sets[i % 5]):
                t.copy_(v)
            for t in case.outputs:
                t.fill_(float("nan"))
            graph.launch()
            for k, (got, w) in enumerate(zip(case.outputs, want[i % 5])):
                assert torch.equal(got, w), f"replay {i}, output {k}"
    assert emu.emu_stream_check(stream) == 0
    graph.close()


class OddBackward(LinearBackward):
    """Rows off the 16-byte boundaries (aligned copies), column sums, a product
    split ahead (tf32x3) and split along k: every kind of buffer."""

    def __init__(self, M, N, K, mode="tf32x3"):
        super().__init__(M, N, K, mode)
        self.k4 = (K + 3) // 4 * 4
        self.dx, self.dw = empty(M, self.k4), empty(N, self.k4)
        self.outputs = [self.dz, self.dx, self.dw, self.db]

    def run(self):
        import fp32_emulated_gemm_gb300 as emu
        M, N, K = self.size
        emu.emu_linear_act_bwd(emu.MODES[self.mode], M, N, K, self.dy, N, self.x, K, self.w, K, self.d, N, self.dz, N,
                               self.dx, self.k4, self.dw, self.k4, self.db)

    def results(self):
        K = self.size[2]
        return [self.dz, self.dx[:, :K], self.dw[:, :K], self.db]


class NormBackward:
    def __init__(self, M, N):
        self.size = (M, N)
        self.dy, self.x, self.mean, self.rstd = empty(M, N), empty(M, N), empty(M), empty(M)
        self.dx, self.dw, self.db = empty(M, N), empty(N), empty(N)
        self.inputs, self.outputs = [self.dy, self.x, self.mean, self.rstd], [self.dx, self.dw, self.db]

    def draw(self, seed):
        M, N = self.size
        return [rand(M, N, seed=seed), rand(M, N, seed=seed + 100), rand(M, seed=seed), rand(M, seed=seed + 100)]

    def run(self):
        import fp32_emulated_gemm_gb300 as emu
        M, N = self.size
        emu.emu_layer_norm_bwd(M, N, self.dy, N, self.x, N, None, self.mean, self.rstd, None, 0, self.dx, N, self.dw,
                               self.db)

    def results(self):
        return self.outputs


def filled(case, seed):
    for t, v in zip(case.inputs, case.draw(seed)):
        t.copy_(v)
    return case


@pytest.mark.parametrize("small,large", [
    (lambda: OddBackward(1300, 300, 499), lambda: OddBackward(9000, 1100, 2047)),
    (lambda: NormBackward(500, 260), lambda: NormBackward(70000, 1500)),
])
def test_a_larger_call_leaves_a_graphs_buffers_alone(small, large):
    """A graph's replays after calls of other sizes on its stream, which need
    larger buffers: each computes its own."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    from tests import _graphs
    emu.emu_shutdown()                    # the stream may have larger buffers from before
    a, b = filled(small(), 1), filled(large(), 2)
    a.run()
    b.run()
    want_a, want_b = [t.clone() for t in a.results()], [t.clone() for t in b.results()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        a.run()
    graph = _graphs.Graph(stream, a.run)
    with torch.cuda.stream(stream):
        for rep in range(6):
            for t in a.outputs + b.outputs:
                t.fill_(float("nan"))
            if rep % 2:
                graph.launch()
                b.run()
            else:
                b.run()
                graph.launch()
            for got, want in zip(a.results() + b.results(), want_a + want_b):
                assert torch.equal(got, want), rep
    assert emu.emu_stream_check(stream) == 0
    graph.close()


@pytest.mark.parametrize("make", [lambda: Product(300, 260, 3000, "bf16x9"), lambda: Product(2000, 2500, 200, "tf32x3"),
                                  lambda: OddBackward(1300, 300, 499), lambda: NormBackward(500, 260)])
def test_no_allocation_under_capture(make):
    """A captured call whose buffers its stream does not have is refused; the
    capture stays valid and the library as it was."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    from tests import _graphs
    emu.emu_shutdown()
    case = filled(make(), 3)
    case.run()
    want = [t.clone() for t in case.outputs]
    stream = torch.cuda.Stream()
    status = []

    def refused():
        try:
            case.run()
        except emu.EmuError as e:
            status.append(e.status)

    graph = _graphs.Graph(stream, refused)
    assert status == [4] and graph.nodes() == []
    graph.close()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        case.run()                        # now the stream has them
    graph = _graphs.Graph(stream, case.run)
    with torch.cuda.stream(stream):
        for t in case.outputs:
            t.zero_()
        graph.launch()
        if hasattr(case, "results"):
            case.outputs = case.results()
        for got, w in zip(case.outputs, want):
            assert torch.equal(got, w[:, :got.shape[1]] if got.dim() == 2 else w)
    assert emu.emu_stream_check(stream) == 0
    graph.close()


@pytest.mark.parametrize("priority", [0, -1])
def test_side_by_side_products_keep_the_streams_priority(priority):
    """Both products of a backward pass run at the priority of the caller's
    stream (which a captured kernel node records)."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    from tests import _graphs
    emu.emu_shutdown()
    case = filled(LinearBackward(1536, 300, 500, "bf16x9"), 4)
    stream = torch.cuda.Stream(priority=priority)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        case.run()
    graph = _graphs.Graph(stream, case.run)
    got = graph.kernel_priorities()
    graph.close()
    assert len(got) >= 4 and set(got) == {priority}, got


OVERLAPS = """
import torch, fp32_emulated_gemm_gb300 as emu
from tests import _graphs, test_gpu_graphs as t
norm = t.filled(t.NormBackward(500, 260), 1)
x, wi, wo = t.rand(3, 64, seed=1), t.rand(2 * 96, 64, seed=2), t.rand(64, 96, seed=3)
h, y = t.empty(3, 96), t.empty(3, 64)
def few():
    emu.emu_gated_ffn_fwd(0, emu.EMU_ACT_SILU, 3, 64, 96, 64, x, 64, wi, 64, None, wo, 96, None, None, 0, None, 0, h, 96, y, 64)
for work in (norm.run, few):
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        work()
    g = _graphs.Graph(stream, work)
    print(g.types().count(_graphs.KERNEL), g.programmatic_edges())
"""


@pytest.mark.parametrize("pdl", [1, 0])
def test_pdl_off_means_no_overlap(pdl):
    """EMU_PDL=0 holds for the sums of partial sums and for the few-row form's
    second kernel too."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", OVERLAPS], capture_output=True, text=True, timeout=300, cwd=root,
                       env=dict(os.environ, EMU_PDL=str(pdl), PYTHONPATH=root))
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["2", str(pdl), "2", str(pdl)], r.stdout


@pytest.mark.parametrize("rows", [3, 1500])
def test_a_module_in_a_graph(rows):
    """Inference through the sub-layer's module captured as PyTorch does it,
    after one call on the capturing stream; and larger calls meanwhile."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(rows)
    block = emu.EmuFeedForward(96, 130, mode="tf32x3").to(_gpu.device())
    x = torch.zeros(rows, 96, device=_gpu.device())
    large = rand(5000, 96, seed=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.no_grad():
        block(x)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s), torch.no_grad():
        y = block(x)
    for seed in range(20):
        x.copy_(rand(rows, 96, seed=seed))
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.no_grad():
            block(large)                  # grows the stream's buffers the first time
        torch.cuda.current_stream().wait_stream(s)
        g.replay()
        with torch.no_grad():
            assert torch.equal(y, block(x))
    assert emu.emu_stream_check() == 0
