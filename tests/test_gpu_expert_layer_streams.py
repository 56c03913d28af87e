"""Two expert layers at once, on two streams with buffers of their own: eagerly
and as graphs, each gives what it gives alone."""
import pytest
import torch

from gpu_helpers import check_device_error_word
from test_gpu_expert_layer import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [8, 333])
def test_two_layers_at_once(M):
    layers = [Layer(M, 512, 256, 16, 4, seed) for seed in (1, 2)]
    streams = [torch.cuda.Stream() for _ in layers]
    want = []
    for L in layers:
        L.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in L.outputs()])
    graphs = []
    for L, st in zip(layers, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            L.run()
        graphs.append(g)

    def eager(i):
        with torch.cuda.stream(streams[i]):
            layers[i].run()

    def replay(i):
        with torch.cuda.stream(streams[i]):
            graphs[i].replay()

    for run in (eager, replay):
        for L in layers:
            for t in L.outputs():
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for i in (0, 1):
                run(i)
        torch.cuda.synchronize()
        check_device_error_word()
        for L, w in zip(layers, want):
            assert all(torch.equal(a, b) for a, b in zip(L.outputs(), w))
