"""The example's decoder layers (delta mixer, norms and gates, MoE block)
together: eager steps, a captured step and another slot order agree bit for
bit, and streams do not see one another."""
import importlib.util
import os

import pytest

from util import gpu_env

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def stack():
    _, dev = gpu_env()
    spec = importlib.util.spec_from_file_location(
        "hybrid_layer", os.path.join(ROOT, "examples", "hybrid_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module.HybridStack(2, 5, hidden=512, inter=128, qk_heads=2, v_heads=4, head_dim=64,
                              max_tokens=160, max_seqs=5, device=dev)


def tokens(n, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((n, 512), generator=g, device="cuda").bfloat16()


def ints(*v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def reset(stack):
    for s in stack.states:
        s.zero_()


def test_eager_and_captured_steps_agree(stack):
    import torch
    reset(stack)
    slots = ints(4, 0, 2)
    h = stack(tokens(150, 1), slots, ints(0, 70, 71, 150))
    assert h.shape == (150, 512) and h.isfinite().all()
    after = [s.clone() for s in stack.states]
    x = [tokens(3, 10 + i) for i in range(3)]
    eager = [stack(t, slots).clone() for t in x]
    end = [s.clone() for s in stack.states]
    for s, a, e in zip(stack.states, after, end):
        assert not torch.equal(a[[4, 0, 2]], e[[4, 0, 2]])
        assert (e[[1, 3]] == 0).all()
        s.copy_(a)
    token = x[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = stack(token, slots)
    for t, want in zip(x, eager):
        token.copy_(t)
        graph.replay()
        assert torch.equal(out, want)
    for s, e in zip(stack.states, end):
        assert torch.equal(s, e)
    assert stack.status() == 0


def test_streams_in_another_order(stack):
    """The same prompts in other slots leave the same states there (rows of one
    token: the routes of the matrix products and of the block are the same)."""
    import torch
    x = tokens(4, 2)
    reset(stack)
    a = stack(x, ints(0, 1, 2, 3)).clone()
    first = [s.clone() for s in stack.states]
    reset(stack)
    b = stack(x, ints(3, 4, 0, 1))
    assert torch.equal(a, b)
    for s, f in zip(stack.states, first):
        assert torch.equal(s[[3, 4, 0, 1]], f[[0, 1, 2, 3]])
