"""Cache, attention and verification of drafts together, as a decoder uses them:
by themselves against the fp64 definitions, and in the example's layers, eager
and captured."""
import importlib.util
import os

import numpy as np
import pytest

from attn_ref import verify
from test_gpu_attention import Batch
from util import gpu_env

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def env():
    return gpu_env()


def ints(*v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check_tokens(p, q, d, u, tokens, accepted):
    """Every sequence's answer is the definition's (or, within the sums' rounding of
    2^-45, the neighbouring token's)."""
    p, q, d, u, tokens, accepted = (x.cpu().numpy() for x in (p, q, d, u, tokens, accepted))
    for b in range(len(p)):
        a, token, cum, aim = verify(p[b], q[b], d[b], u[b])
        assert accepted[b] == a and (tokens[b, :a] == d[b, :a]).all()
        assert (tokens[b, a + 1:] == -1).all()
        if tokens[b, a] != token:
            lo = cum[tokens[b, a] - 1] if tokens[b, a] else 0.0
            assert min(abs(lo - aim), abs(cum[tokens[b, a]] - aim)) <= 2.0 ** -45 * cum[-1]


@pytest.mark.parametrize("kv", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("heads,t", [((8, 2), 3), ((8, 1), 3)])  # 16 and 32 rows a sequence
def test_write_attend_verify_in_one_graph(env, kv, heads, t):
    """New rows written, attended to and verified in a captured call; each replay's rows, lengths
    and tokens are its own."""
    import torch
    moe, dev = env
    V, d, B = 500, 64, 6
    lens = [4, 65, 130, 300, 64, 17]
    g = torch.Generator(device=dev).manual_seed(5)
    batch = Batch(env, [t + 1] * B, lens, heads, d, 16, kv, uniform=True).fill()
    head = torch.randn((heads[0] * d, V), generator=g, device=dev) * 0.3
    q = torch.softmax(torch.randn((B, t, V), generator=g, device=dev) * 2, -1)
    drafted = q.argmax(-1).int()
    u = torch.rand((B, t + 1), generator=g, device=dev)
    n = B * (t + 1)
    k = torch.randn((n, heads[1], d), generator=g, device=dev).bfloat16()
    v = torch.randn((n, heads[1], d), generator=g, device=dev).bfloat16()
    verifier, length = moe.DraftVerifier(dev), batch.lens.clone()

    def run():
        batch.attn.write(batch.cache, k, v, batch.table, length)
        o = batch.attn.attend(batch.cache, batch.q, batch.table, length)
        p = torch.softmax(o.flatten(1).float() @ head, -1).view(B, t + 1, V)
        return (o, p) + verifier.verify(p, drafted, u, draft=q)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, p, tokens, accepted = run()
    ends = np.cumsum(lens)
    for seed in range(3):
        g.manual_seed(100 + seed)
        k.normal_(generator=g), v.normal_(generator=g), u.uniform_(generator=g)
        for b in range(B):  # the definition's inputs: the new rows are each sequence's last
            rows = slice(b * (t + 1), (b + 1) * (t + 1))
            batch.k[ends[b] - t - 1:ends[b]] = k[rows]
            batch.v[ends[b] - t - 1:ends[b]] = v[rows]
        graph.replay()
        batch.check(o)
        check_tokens(p, q, drafted, u, tokens, accepted)
    assert verifier.status() == 0 and batch.attn.status() == 0


def test_graphs_share_a_workspace(env):
    """Two captured calls of different batches on one object, replayed in turn."""
    import torch
    a = Batch(env, [300, 2, 90], [700, 44, 90], (8, 2), 128, 64, "int8").fill()
    b = Batch(env, [1] * 5, [40, 3000, 1, 700, 64], (8, 2), 128, 64, "int8", uniform=True).fill()
    b.attn = a.attn
    want = [a.attend().clone(), b.attend().clone()]
    graphs, outs = [], []
    for x in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(x.attend())
        graphs.append(graph)
    for i in (0, 1, 1, 0, 0, 1):
        outs[i].fill_(7.0)
        graphs[i].replay()
        assert torch.equal(outs[i], want[i])


def test_two_streams_at_once(env):
    """Objects of their own on streams of their own, their calls overlapping."""
    import torch
    moe, dev = env
    batches = [Batch(env, [300, 2, 90], [700, 44, 90], (8, 2), 128, 64, "int8").fill(),
               Batch(env, [1000], [3000], (8, 2), 256, 16, "bf16", seed=1).fill(),
               Batch(env, [1] * 5, [40, 3000, 1, 700, 64], (8, 2), 64, 64, "e4m3").fill()]
    p = torch.softmax(torch.randn((40, 3, 20000), device=dev) * 3, -1)
    drafted, u = p[:, :2].argmax(-1).int(), torch.rand((40, 3), device=dev)
    verifier = moe.DraftVerifier(dev)
    calls = [b.attend for b in batches] + [lambda **kw: verifier.verify(p, drafted, u, **kw)[0]]
    want = [f().clone() for f in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[] for _ in calls]
    for _ in range(10):
        for f, s, r in zip(calls, streams, got):
            r.append(f(stream=s))
    torch.cuda.synchronize()
    for w, r in zip(want, got):
        assert all(torch.equal(x, w) for x in r)
    assert not any(b.attn.status() for b in batches) and verifier.status() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_sequences_share_pages(env, new):
    """A prefix in pages that several sequences name."""
    import torch
    b = Batch(env, [new] * 3, [200, 200, 200], (8, 2), 128, 16, "e4m3", uniform=True).fill()
    want = b.attend()
    table = b.table.clone()
    for s in (1, 2):  # the first 160 positions of all are those of the first
        b.k[200 * s:200 * s + 160] = b.k[:160]
        b.v[200 * s:200 * s + 160] = b.v[:160]
    table[1:, :10] = table[:1, :10]
    b.table = table
    got = b.attend()
    b.check(got)
    assert torch.equal(got[:new], want[:new])


# ------------------------------------------------------- the example's layers
@pytest.fixture(scope="module")
def example(env):
    spec = importlib.util.spec_from_file_location(
        "hybrid_layer", os.path.join(ROOT, "examples", "hybrid_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


SLOTS, HIDDEN, VOCAB = 5, 512, 300


def make(example, kv="int8", drafts=3):
    import torch
    torch.manual_seed(3)  # the order of the pages
    stack = example.HybridStack(3, SLOTS, 2, 256, q_heads=8, kv_heads=2, kv_type=kv, page_size=16,
                                hidden=HIDDEN, inter=128, qk_heads=2, v_heads=4, head_dim=64,
                                max_tokens=160, max_seqs=2 * SLOTS)
    return stack, example.Speculator(stack, VOCAB, HIDDEN, drafts)


def held(stack):
    """Everything that a stack keeps."""
    import torch
    return [stack.lens.clone()] + [
        x.clone() for s in stack.states for x in (s if isinstance(s, tuple) else (s,))
        if torch.is_tensor(x)]


def put_back(stack, was):
    import torch
    now = [stack.lens] + [x for s in stack.states for x in (s if isinstance(s, tuple) else (s,))
                          if torch.is_tensor(x)]
    for x, y in zip(now, was):
        x.copy_(y)


def same(a, b):
    import torch
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def embeddings(n, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((n, HIDDEN), generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("kv", ["bf16", "int8", "e4m3"])
def test_drafting_eager_and_captured(example, kv):
    import torch
    stack, spec = make(example, kv)
    slots = ints(4, 0, 2)
    stack(embeddings(150, 1), slots, ints(0, 70, 71, 150))
    assert stack.lens.tolist() == [1, 0, 79, 0, 70]
    g = torch.Generator(device="cuda").manual_seed(2)
    u = [torch.rand((3, 7), generator=g, device="cuda") for _ in range(6)]
    last = ints(5, 290, 17)
    start, eager = held(stack), []
    for x in u:
        before = stack.lens.clone()
        tokens, accepted = spec.step(last, slots, x)
        eager.append((tokens.clone(), accepted.clone()))
        assert torch.equal(stack.lens[slots.long()] - before[slots.long()], accepted + 1)
        last = tokens.gather(1, accepted.long()[:, None])[:, 0]
        assert (last >= 0).all() and (last < VOCAB).all()
    # (some drafts stood and some did not, or this tests little)
    count = torch.stack([a for _, a in eager])
    assert (count > 0).any() and (count < 3).any()
    end = held(stack)
    put_back(stack, start)
    last, uniform = ints(5, 290, 17), u[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens, accepted = spec.step(last, slots, uniform)
        last.copy_(tokens.gather(1, accepted.long()[:, None])[:, 0])
    for x, (t, a) in zip(u, eager):
        uniform.copy_(x)
        graph.replay()
        assert torch.equal(tokens, t) and torch.equal(accepted, a)
    assert same(held(stack), end)
    assert spec.status() == 0


def test_rejected_tokens_leave_nothing(example):
    """What is kept of a draft does not depend on the tokens behind; a draft kept whole is
    as if it had been so from the start."""
    import torch
    stack, _ = make(example)
    slots, x, y = ints(1, 3), embeddings(8, 5), embeddings(8, 6)
    stack(embeddings(90, 4), slots, ints(0, 33, 90))
    start = held(stack)
    for count in (1, 2):
        z = torch.where((torch.arange(8, device="cuda") % 4 < count)[:, None], x, y)
        after, nexts = [], []
        for rows in (x, z):
            put_back(stack, start)
            stack(rows, slots, keep=False)
            stack.accept(slots, ints(count, count), 4)
            assert (stack.lens - start[0]).tolist() == [0, count, 0, count, 0]
            after.append([s.clone() for s in stack.states if torch.is_tensor(s)])
            nexts.append(stack(y[:2], slots).clone())
        assert same(*after) and torch.equal(*nexts)
    put_back(stack, start)
    h = stack(x, slots, keep=False).clone()
    stack.accept(slots, ints(4, 4), 4)
    kept = held(stack)
    put_back(stack, start)
    assert torch.equal(stack(x, slots), h)
    assert same(held(stack), kept)
    assert stack.status() == 0


def test_example_runs(example, capsys):
    example.main(["--layers", "2", "--attention-every", "2", "--tokens", "200", "--streams", "4",
                  "--hidden", "512", "--inter", "128", "--steps", "3", "--vocab", "1000"])
    assert "drafts of 3" in capsys.readouterr().out
