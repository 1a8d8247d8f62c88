"""A decoder layer of a hybrid model, from the framework's own calls: gated
delta mixer, norms and gates around it, sparse-MoE block.

    python examples/hybrid_layer.py [--layers 4] [--tokens 2048] [--streams 32]

Prompts of different lengths go through the layers in one call each
(``GatedDelta.chunk``); then every stream decodes token by token on the state
that its prompt left (``GatedDelta.step``), the whole stack captured in one
CUDA graph.  Random weights; the projections are plain matrix products.

    x -> q, k, v, z, decay, beta                      (matrix products)
      -> delta rule -> norm per head, gated by z      (GatedDelta, norm_gate_residual)
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


class HybridLayer:
    def __init__(self, hidden=2048, qk_heads=16, v_heads=32, head_dim=128, inter=512,
                 max_tokens=2048, max_seqs=64, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=gen, device=device) * std).bfloat16()

        def int8(*shape):
            return torch.randint(-127, 128, shape, generator=gen, device=device, dtype=torch.int8)

        def scale(*shape, std):
            return normal(*shape, std=std).abs()

        self.qk, self.v, self.heads = qk_heads * head_dim, v_heads * head_dim, v_heads
        self.dim = head_dim
        std = hidden ** -0.5
        self.w_in = normal(hidden, 2 * self.qk + 2 * self.v, std=std)  # q, k, v, z
        self.w_gates = normal(hidden, 2 * v_heads, std=std)            # decay, beta
        self.w_out = normal(self.v, hidden, std=self.v ** -0.5)
        self.decay = -torch.rand(v_heads, generator=gen, device=device)
        self.norm_moe, self.gate = normal(hidden, std=0.1) + 1, normal(hidden)
        self.norm_next, self.norm_head = normal(hidden, std=0.1) + 1, normal(head_dim, std=0.1) + 1
        self.delta = moe.GatedDelta(qk_heads, v_heads, head_dim, head_dim, max_tokens, max_seqs,
                                    device=device)
        E, G = 256, 128
        s = std / 73  # int8 values have a deviation of 73
        self.block = moe.MoEBlock(hidden, inter, inter, {
            "w_router": normal(E, hidden, std=0.02), "w_shared_gate": normal(hidden, std=0.02),
            "w13_q": int8(E, 2 * inter, hidden), "w13_s": scale(E, 2 * inter, hidden // G, std=s),
            "w2_q": int8(E, hidden, inter), "w2_s": scale(E, hidden, inter // G, std=s),
            "ws13_q": int8(2 * inter, hidden), "ws13_s": scale(2 * inter, hidden // G, std=s),
            "ws2_q": int8(hidden, inter), "ws2_s": scale(hidden, inter // G, std=s)},
            max_tokens, device)

    def state(self, slots):
        return torch.zeros((slots, self.heads, self.dim, self.dim), device=self.w_in.device)

    def __call__(self, x, resid, state, slots, cu_seqlens=None):
        """x (normed) and resid [N][hidden] -> the next layer's.  With
        ``cu_seqlens`` whole prompts, without it one token of each stream."""
        q, k, v, z = (x @ self.w_in).split([self.qk, self.qk, self.v, self.v], 1)
        a, b = (x @ self.w_gates).float().chunk(2, 1)
        g, beta = self.decay * F.softplus(a), torch.sigmoid(b)
        q, k, v, z = (t.unflatten(1, (-1, self.dim)) for t in (q, k, v, z))
        if cu_seqlens is not None:
            o = self.delta.chunk(q, k, v, g, beta, cu_seqlens, state, state, slots)
        else:
            o = self.delta.step(q, k, v, g, beta, state, state, slots)
        o, _ = moe.norm_gate_residual(o, self.norm_head, gate=z, gate_act="silu")
        y = o.flatten(1) @ self.w_out
        resid, x = moe.norm_gate_residual(y, resid=resid, gamma_pre=self.norm_moe)
        y = self.block.forward(x)
        return moe.norm_gate_residual(y, gate=self.gate, resid=resid, gamma_pre=self.norm_next)

    def status(self):
        return self.delta.status() | self.block.status()


class HybridStack:
    def __init__(self, layers, slots, **kw):
        self.layers = [HybridLayer(seed=i, **kw) for i in range(layers)]
        self.states = [layer.state(slots) for layer in self.layers]

    def __call__(self, x, slots, cu_seqlens=None):
        """The tokens' embeddings [N][hidden] -> the last norm's output."""
        resid, h = x, F.rms_norm(x, x.shape[1:])
        for layer, state in zip(self.layers, self.states):
            resid, h = layer(h, resid, state, slots, cu_seqlens)
        return h

    def status(self):
        return sum(layer.status() for layer in self.layers)


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
    args = p.parse_args(argv)
    dev = torch.device("cuda")
    n, b = args.tokens, args.streams
    stack = HybridStack(args.layers, b, hidden=args.hidden, inter=args.inter, max_tokens=max(n, b),
                        max_seqs=b, device=dev)
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


if __name__ == "__main__":
    main()
