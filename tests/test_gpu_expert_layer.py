"""The norms, the experts and the 4-bit projection together, as a layer over virtual ranks uses them."""
import importlib.util
import os

import pytest
import torch

from shot_allreduce_ranks_gb300 import build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    build.build()
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_served_and_trained(layer):
    """Every value passes at most eight roundings to bfloat16 on its way (y, h, a rank's part, the sum, r, y2, z and one for
    what they are made of), each of at most 2^-8 of its value; a gradient passes four (y, dgate and dup, dy, itself),
    and where r is rounded before it is differentiated one more."""
    for name, v in layer.main(say=lambda *_: None).items():
        assert v < (8 if name == "served" else 5) * 2.0 ** -8, (name, v)


def test_in_a_graph_the_same_bits(layer):
    served = layer.Served()
    x, residual = layer.make((13, 1024), seed=40), layer.make((13, 1024), 2.0, seed=41)
    want = served.step(x, residual)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = served.step(x, residual)
    for _ in range(10):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    served.allreduce.close()


def test_two_steps_at_once_on_two_streams(layer):
    """Steps on streams of their own share weights and nothing else."""
    a, b = layer.Served(), layer.Served()
    x, residual = layer.make((13, 1024), seed=50), layer.make((13, 1024), 2.0, seed=51)
    want = a.step(x, residual)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for layer_, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(layer_.step(x, residual))
        torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(p, q) for p, q in zip(g, want))
    a.allreduce.close()
    b.allreduce.close()
