"""Decoder layers of a hybrid model, from the framework's own calls: gated
delta mixer or attention over a paged cache, norms and gates around it,
sparse-MoE block.

    python examples/hybrid_layer.py [--layers 4] [--tokens 2048] [--streams 32]

Prompts of different lengths go through the layers in one call each
(``GatedDelta.chunk``, ``PagedAttention.write`` and ``.attend``); then every
stream decodes token by token on the state and the pages that its prompt left
(``GatedDelta.step``), the whole stack captured in one CUDA graph; then drafts of
a few tokens are verified against the stack's probabilities (``DraftVerifier``)
and those that stand are kept, drafting and all in one graph.  Random weights;
the projections are plain matrix products, without rotary positions.

    x -> q, k, v, z, decay, beta                      (matrix products)
      -> delta rule -> norm per head, gated by z      (GatedDelta, norm_gate_residual)
      or q, k, v -> the cache -> attention            (PagedAttention)
      -> projection -> residual + norm                (matrix product, norm_gate_residual)
      -> MoE block -> gated residual + the next norm  (MoEBlock, norm_gate_residual)
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_moe_decode_gb300 as moe  # noqa: E402


class Weights:
    """Random ones, each seed's own."""

    def __init__(self, device, seed):
        self.gen, self.device = torch.Generator(device=device).manual_seed(seed), device

    def normal(self, *shape, std=1.0):
        return (torch.randn(shape, generator=self.gen, device=self.device) * std).bfloat16()

    def block(self, hidden, inter, max_tokens):
        def int8(*shape):
            return torch.randint(-127, 128, shape, generator=self.gen, device=self.device,
                                 dtype=torch.int8)

        def scale(*shape, std):
            return self.normal(*shape, std=std).abs()

        E, G, std = 256, 128, hidden ** -0.5
        s = std / 73  # int8 values have a deviation of 73
        return moe.MoEBlock(hidden, inter, inter, {
            "w_router": self.normal(E, hidden, std=0.02),
            "w_shared_gate": self.normal(hidden, std=0.02),
            "w13_q": int8(E, 2 * inter, hidden), "w13_s": scale(E, 2 * inter, hidden // G, std=s),
            "w2_q": int8(E, hidden, inter), "w2_s": scale(E, hidden, inter // G, std=s),
            "ws13_q": int8(2 * inter, hidden), "ws13_s": scale(2 * inter, hidden // G, std=s),
            "ws2_q": int8(hidden, inter), "ws2_s": scale(hidden, inter // G, std=s)},
            max_tokens, self.device)


class Layer:
    """What follows a mixer: ``mix`` gives its output [N][hidden]."""

    def __call__(self, x, resid, *where):
        """x (normed) and resid [N][hidden] -> the next layer's."""
        y = self.mix(x, *where)
        resid, x = moe.norm_gate_residual(y, resid=resid, gamma_pre=self.norm_moe)
        y = self.block.forward(x)
        return moe.norm_gate_residual(y, gate=self.gate, resid=resid, gamma_pre=self.norm_next)

    def status(self):
        return self.mixer.status() | self.block.status()


class HybridLayer(Layer):
    def __init__(self, hidden=2048, qk_heads=16, v_heads=32, head_dim=128, inter=512,
                 max_tokens=2048, max_seqs=64, device="cuda", seed=0):
        new = Weights(device, seed)
        self.qk, self.v, self.heads = qk_heads * head_dim, v_heads * head_dim, v_heads
        self.dim = head_dim
        std = hidden ** -0.5
        self.w_in = new.normal(hidden, 2 * self.qk + 2 * self.v, std=std)  # q, k, v, z
        self.w_gates = new.normal(hidden, 2 * v_heads, std=std)            # decay, beta
        self.w_out = new.normal(self.v, hidden, std=self.v ** -0.5)
        self.decay = -torch.rand(v_heads, generator=new.gen, device=device)
        self.norm_moe, self.gate = new.normal(hidden, std=0.1) + 1, new.normal(hidden)
        self.norm_next = new.normal(hidden, std=0.1) + 1
        self.norm_head = new.normal(head_dim, std=0.1) + 1
        self.mixer = moe.GatedDelta(qk_heads, v_heads, head_dim, head_dim, max_tokens, max_seqs,
                                    device=device)
        self.block = new.block(hidden, inter, max_tokens)

    def state(self, slots):
        return torch.zeros((slots, self.heads, self.dim, self.dim), device=self.w_in.device)

    def mix(self, x, state, slots, cu_seqlens=None, keep=True):
        """With ``cu_seqlens`` whole prompts, without it as many tokens of each stream;
        ``keep`` False leaves the states for ``commit``."""
        q, k, v, z = (x @ self.w_in).split([self.qk, self.qk, self.v, self.v], 1)
        a, b = (x @ self.w_gates).float().chunk(2, 1)
        g, beta = self.decay * F.softplus(a), torch.sigmoid(b)
        q, k, v, z = (t.unflatten(1, (-1, self.dim)) for t in (q, k, v, z))
        if cu_seqlens is not None:
            o = self.mixer.chunk(q, k, v, g, beta, cu_seqlens, state, state, slots)
        else:
            o = self.mixer.step(q, k, v, g, beta, state, state if keep else None, slots)
        self.drafted = None if keep else (q, k, v, g, beta)
        o, _ = moe.norm_gate_residual(o, self.norm_head, gate=z, gate_act="silu")
        return o.flatten(1) @ self.w_out

    def commit(self, state, slots, cut):
        """The states after the first tokens of each stream (bounds ``cut``: those and the
        rest of each)."""
        both = torch.stack([slots, torch.full_like(slots, -1)], 1).flatten()
        self.mixer.chunk(*self.drafted, cut, state, state, both)


class AttentionLayer(Layer):
    def __init__(self, hidden=2048, q_heads=32, kv_heads=8, head_dim=128, inter=512,
                 max_tokens=2048, page_size=64, kv_type="int8", device="cuda", seed=0):
        new = Weights(device, seed)
        self.dim = head_dim
        self.split = [q_heads * head_dim, kv_heads * head_dim, kv_heads * head_dim]
        self.w_in = new.normal(hidden, sum(self.split), std=hidden ** -0.5)  # q, k, v
        self.w_out = new.normal(self.split[0], hidden, std=self.split[0] ** -0.5)
        self.norm_moe, self.gate = new.normal(hidden, std=0.1) + 1, new.normal(hidden)
        self.norm_next = new.normal(hidden, std=0.1) + 1
        self.mixer = moe.PagedAttention(q_heads, kv_heads, head_dim, page_size, kv_type,
                                        device=device)
        self.block = new.block(hidden, inter, max_tokens)

    def mix(self, x, cache, table, lens, cu_seqlens=None):
        """``lens``: the streams' positions with these."""
        q, k, v = (t.unflatten(1, (-1, self.dim)) for t in (x @ self.w_in).split(self.split, 1))
        self.mixer.write(cache, k, v, table, lens, cu_seqlens)
        return self.mixer.attend(cache, q, table, lens, cu_seqlens).flatten(1) @ self.w_out


class HybridStack:
    """``layers`` layers over ``slots`` streams; with ``attention_every`` n the n-th, 2n-th and
    so on are attention, over pages for ``max_len`` positions a stream."""

    def __init__(self, layers, slots, attention_every=0, max_len=4096, q_heads=32, kv_heads=8,
                 kv_type="int8", qk_heads=16, v_heads=32, max_seqs=64, page_size=64, device="cuda",
                 **kw):
        def attends(i):
            return attention_every and (i + 1) % attention_every == 0

        self.layers = [
            AttentionLayer(q_heads=q_heads, kv_heads=kv_heads, kv_type=kv_type,
                           page_size=page_size, device=device, seed=i, **kw) if attends(i) else
            HybridLayer(qk_heads=qk_heads, v_heads=v_heads, max_seqs=max_seqs, device=device,
                        seed=i, **kw) for i in range(layers)]
        each = -(-max_len // page_size)  # any order of the pages will do
        self.table = torch.randperm(slots * each, device=device).int().view(slots, each)
        self.lens = torch.zeros(slots, dtype=torch.int32, device=device)
        self.states = [layer.mixer.new_cache(slots * each) if isinstance(layer, AttentionLayer)
                       else layer.state(slots) for layer in self.layers]

    def __call__(self, x, slots, cu_seqlens=None, keep=True):
        """The tokens' embeddings [N][hidden] -> the last norm's output.  ``keep`` False: a
        draft, of which ``accept`` keeps the first tokens."""
        resid, h = x, F.rms_norm(x, x.shape[1:])
        at = slots.long()
        new = x.shape[0] // slots.shape[0] if cu_seqlens is None else cu_seqlens.diff()
        table, lens = self.table[at], self.lens[at] + new
        for layer, state in zip(self.layers, self.states):
            if isinstance(layer, AttentionLayer):
                resid, h = layer(h, resid, state, table, lens, cu_seqlens)
            else:
                resid, h = layer(h, resid, state, slots, cu_seqlens, keep)
        if keep:
            self.lens[at] = lens
        return h

    def accept(self, slots, count, tokens):
        """Keeps the first ``count`` [B] of the ``tokens`` that each stream had drafted."""
        start = tokens * torch.arange(slots.shape[0], dtype=torch.int32, device=slots.device)
        cut = torch.cat([torch.stack([start, start + count], 1).flatten(), start[-1:] + tokens])
        for layer, state in zip(self.layers, self.states):
            if isinstance(layer, HybridLayer):
                layer.commit(state, slots, cut)
        self.lens[slots.long()] += count  # (what lies behind in the pages is not read)

    def status(self):
        return sum(layer.status() for layer in self.layers)


class Speculator:
    """Streams that draft ``drafts`` tokens at a time with a small model (here: the stack's
    head on the last token's embedding) and verify them with the stack."""

    def __init__(self, stack, vocab, hidden, drafts, device="cuda", seed=7):
        new = Weights(device, seed)
        self.stack, self.drafts, self.vocab = stack, drafts, vocab
        self.embedding = new.normal(vocab, hidden)
        self.head = new.normal(hidden, vocab, std=hidden ** -0.5)
        self.verifier = moe.DraftVerifier(device)

    def probabilities(self, x):
        return torch.softmax((x @ self.head).float(), -1)

    def step(self, token, slots, uniform):
        """``token`` int32 [B], which no stream has seen yet, and ``uniform`` [B][2 drafts + 1]
        numbers in [0, 1) -> tokens [B][drafts + 1] (-1 behind the last), accepted [B]."""
        B, T = token.shape[0], self.drafts
        none = token.new_empty((B, 0))
        row, q, u = [token], [], uniform.contiguous()
        for i in range(T):
            p = self.probabilities(F.rms_norm(self.embedding[row[-1].long()], (self.head.shape[0],)))
            new, _ = self.verifier.verify(p[:, None], none, u[:, i:i + 1].contiguous())
            row.append(new[:, 0])
            q.append(p)
        row = torch.stack(row, 1)
        h = self.stack(self.embedding[row.long()].flatten(0, 1), slots, keep=False)
        p = self.probabilities(h).view(B, T + 1, self.vocab)
        tokens, accepted = self.verifier.verify(p, row[:, 1:].contiguous(), u[:, T:].contiguous(),
                                                torch.stack(q, 1))
        self.stack.accept(slots, accepted + 1, T + 1)
        return tokens, accepted

    def status(self):
        return self.stack.status() | self.verifier.status()


def timed(f, n):
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    f()
    torch.cuda.synchronize()
    start.record()
    for _ in range(n):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / n


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--tokens", type=int, default=2048, help="of all prompts")
    p.add_argument("--streams", type=int, default=32)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inter", type=int, default=512)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--attention-every", type=int, default=4, help="0: no attention layer")
    p.add_argument("--drafts", type=int, default=3)
    p.add_argument("--vocab", type=int, default=32768)
    args = p.parse_args(argv)
    dev = torch.device("cuda")
    n, b = args.tokens, args.streams
    drafted = b * (args.drafts + 1)
    # (every call below is repeated to time it)
    most = 7 * n + (args.steps + 2) * (args.drafts + 2)
    stack = HybridStack(args.layers, b, args.attention_every, most, hidden=args.hidden,
                        inter=args.inter, max_tokens=max(n, drafted), max_seqs=2 * b, device=dev)
    gen = torch.Generator(device=dev).manual_seed(99)
    cuts = torch.randint(0, n + 1, (b - 1,), generator=gen, device=dev).sort().values
    cu = F.pad(cuts, (1, 1))
    cu[-1] = n
    cu = cu.int()
    slots = torch.arange(b, dtype=torch.int32, device=dev)
    prompts = torch.randn((n, args.hidden), generator=gen, device=dev).bfloat16()
    h = stack(prompts, slots, cu)
    assert stack.status() == 0 and bool(h.isfinite().all())
    print("prompts: %d tokens in %d streams, %d layers: %.3f ms" % (
        n, b, args.layers, timed(lambda: stack(prompts, slots, cu), 5)))
    # decode: the last norm's output stands in for the next token's embedding
    token = torch.randn((b, args.hidden), generator=gen, device=dev).bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stack(token, slots)  # warm
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token.copy_(stack(token, slots))
    ms = timed(graph.replay, args.steps)
    assert stack.status() == 0 and bool(token.isfinite().all())
    print("decode: %d streams, %d layers: %.3f ms a step, %.0f tokens/s" % (
        b, args.layers, ms, b / ms * 1e3))
    # drafts: the tokens that stand, and one more
    spec = Speculator(stack, args.vocab, args.hidden, args.drafts, dev)
    last = torch.randint(args.vocab, (b,), generator=gen, device=dev, dtype=torch.int32)
    uniform = torch.empty((b, 2 * args.drafts + 1), device=dev)
    made = torch.zeros((), dtype=torch.int64, device=dev)

    def step():
        uniform.uniform_()
        tokens, accepted = spec.step(last, slots, uniform)
        last.copy_(tokens.gather(1, accepted.long()[:, None])[:, 0])
        made.add_(accepted.sum() + b)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # warm
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    made.zero_()
    ms = timed(graph.replay, args.steps)
    each = made.item() / (args.steps + 1)
    assert spec.status() == 0
    print("drafts of %d: %.3f ms a step, %.2f tokens a stream, %.0f tokens/s" % (
        args.drafts, ms, each / b, each / ms * 1e3))


if __name__ == "__main__":
    main()
