"""The clipped path behind sequence operators in graphs and across streams, on the GPU: its norm kernels may
start and load under the launch in front of them, which must then not be one that writes their inputs."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture()
def step(lib):
    """A distillation gradient over rows whose last ones come late, as the G of a head's norms."""
    import torch

    class Step:
        B, T, V, d = 3, 104, 65536, 64
        g = torch.Generator(device="cuda").manual_seed(5)
        z = torch.randn(B, T, V, generator=g, device="cuda").bfloat16()
        idx = torch.randint(0, V, (B, T, 16), generator=g, device="cuda", dtype=torch.int32)
        top = torch.randn(B, T, 16, generator=g, device="cuda").bfloat16()
        A = torch.randn(B, T, d, generator=g, device="cuda").bfloat16()
        head = lib.layer_desc(lib.DP_LINEAR, lib.DP_BF16, B=B, p=V, T=T, d=d)
        ws = torch.empty(lib.dp_workspace_size(head, lib.DP_NORM_GHOST), dtype=torch.uint8, device="cuda")
        dz = torch.empty_like(z)
        sq = torch.empty(B, device="cuda")
        desc = lib.DistillDesc(lib.DP_BF16, lib.DP_BF16, B, T, V, 16, 0, 0, V, V, 1.0, 0.0)

        def operator(self):
            lib.dp_distill(self.desc, self.z, self.idx, self.top, dlogits=self.dz)

        def norm(self):
            lib.dp_layer_sqnorms(self.head, self.A, self.dz, self.sq, self.ws, mode=lib.DP_NORM_GHOST)

        def want(self):
            self.operator()
            torch.cuda.synchronize()
            self.norm()
            torch.cuda.synchronize()
            return self.sq.clone()

        def clear(self):
            self.dz.zero_()
            self.sq.zero_()
            torch.cuda.synchronize()

    return Step()


def _edges(graph):
    """(from, to, may start under it) of a captured graph's nodes, by their numbers."""
    rt = ctypes.CDLL("libcudart.so.13")
    h, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t()
    assert rt.cudaGraphGetNodes(h, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert rt.cudaGraphGetNodes(h, nodes, ctypes.byref(n)) == 0
    number = {v: i for i, v in enumerate(nodes)}
    assert rt.cudaGraphGetEdges(h, None, None, None, ctypes.byref(n)) == 0
    a, b, data = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (ctypes.c_ubyte * (8 * n.value))()
    assert rt.cudaGraphGetEdges(h, a, b, data, ctypes.byref(n)) == 0
    # an edge's data: from port, to port, type (1: programmatic)
    return sorted((number[a[i]], number[b[i]], data[8 * i + 2] == 1) for i in range(n.value))


def test_captured_behind_an_operator_of_another_stream(step):
    """Operator on one stream, an event, the norms on another: the edge must be an ordinary one (an event's
    wait alone does not make it one)."""
    import torch
    want = step.want()
    graph, side = torch.cuda.CUDAGraph(keep_graph=True), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        step.operator()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step.norm()
            step.norm()
        torch.cuda.current_stream().wait_stream(side)
    assert _edges(graph) == [(0, 1, False), (1, 2, True)]
    graph.instantiate()
    for _ in range(3):
        step.clear()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(step.sq, want)


def test_captured_behind_an_operator_and_a_launch(step):
    import torch
    want = step.want()
    graph, side = torch.cuda.CUDAGraph(keep_graph=True), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            step.norm()
        step.operator()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            step.norm()
        main.wait_stream(side)
    assert all(not early for _, _, early in _edges(graph))
    graph.instantiate()
    step.clear()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.sq, want)


def test_captured_on_one_stream(step):
    import torch
    want = step.want()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        step.operator()
        step.norm()
        step.norm()
    assert _edges(graph) == [(0, 1, False), (1, 2, True)]
    graph.instantiate()
    for _ in range(3):
        step.clear()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(step.sq, want)


def test_behind_a_graph_and_behind_an_event(step):
    """The operator in a replayed graph, or on another stream before an event, and the norms called
    right behind: both keep stream order in full."""
    import torch
    want = step.want()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        step.operator()
    for _ in range(3):
        step.clear()
        step.norm()                    # nothing is left to wait for on this stream
        torch.cuda._sleep(1_000_000)
        graph.replay()
        step.norm()
        torch.cuda.synchronize()
        assert torch.equal(step.sq, want)
        step.clear()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000)
            step.operator()
        step.norm()
        torch.cuda.current_stream().wait_stream(side)
        step.norm()
        torch.cuda.synchronize()
        assert torch.equal(step.sq, want)
