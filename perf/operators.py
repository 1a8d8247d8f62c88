"""Workloads of the operators beside the sparse-MoE block in a hybrid decoder
layer: the gated delta rule (the layer's token mixer, over whole prompts in
chunks and token by token) and the norms around a block fused with its gate
and its scaled residual add.

Each operator has a plain form in elementary torch operations (fp32, angles
and long sums in fp64) and, with ``own`` true, the call of this package that
computes the same.  ``exact`` is the operator's definition in fp64, token by
token and without the package's code.
"""
import math

import torch
import torch.nn.functional as F

own = False

DEV = "cuda"
CHUNK = 64  # tokens per chunk of the plain chunked form
EPS = 1e-6

# One decoder layer of the block's width (hidden 2048) has 16 query/key heads
# of 128 and 32 value heads of 128 in its delta mixer.
FULL = dict(hk=16, hv=32, dk=128, dv=128)


def listed():
    return [
        # A short chat turn: one prompt just over a chunk.
        dict(name="delta_prompt_67", op="chunk", n=67, b=1, mix=0, state=False, **FULL),
        # The block's prefill size, one prompt.
        dict(name="delta_prompt_2048", op="chunk", n=2048, b=1, mix=0, state=False, **FULL),
        # Continuous batching: prompts of very different lengths (one empty,
        # one of a single token), each with a state carried over.
        dict(name="delta_ragged_13", op="chunk", n=6007, b=13, mix=1, state=True, **FULL),
        # A long prompt: the sequential axis decides.
        dict(name="delta_prompt_8192", op="chunk", n=8192, b=1, mix=0, state=True, **FULL),
        # A small model's heads over a batch of prompts.
        dict(name="delta_small_heads", op="chunk", n=8192, b=8, mix=2, state=True,
             hk=8, hv=8, dk=64, dv=64),
        # Decode: one stream (latency), a serving batch, a large one.
        dict(name="delta_step_1", op="step", b=1, t=1, **FULL),
        dict(name="delta_step_32", op="step", b=32, t=1, **FULL),
        dict(name="delta_step_256", op="step", b=256, t=1, **FULL),
        # Verification of a 7-token draft and its anchor for a few streams.
        dict(name="delta_verify_4x8", op="step", b=4, t=8, **FULL),
        # The residual step between two blocks: decode, then a large prefill
        # with a gate per element and both norms.
        dict(name="norm_decode_1", op="norm", rows=1, inner=1, width=2048, post=True, pre=True,
             resid=True, gate="channel", act="sigmoid", scale=0.5),
        dict(name="norm_prefill_16384", op="norm", rows=16384, inner=1, width=2048, post=True,
             pre=True, resid=True, gate="element", act="sigmoid", scale=0.5),
        # The delta mixer's output norm: one row per head, gated by silu(z).
        dict(name="norm_heads_2048x32", op="norm", rows=2048 * 32, inner=32, width=128, post=True,
             pre=False, resid=False, gate="element", act="silu", scale=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "step", "step", "norm", "norm"])
    if op == "norm":
        width = rng.choice([128, 2048, _log(rng, 1, 8192), _log(rng, 1, 1024) * 8])
        inner = rng.choice([1, 1, 32])
        pre = rng.random() < 0.6
        gate = rng.choice(["none", "channel", "element", "row"])
        rows = _log(rng, 1, max(2, min(1 << 20, (16384 * 2048) // width) // inner)) * inner
        return dict(op="norm", rows=rows, inner=inner, width=width, post=rng.random() < 0.7,
                    pre=pre, resid=rng.random() < 0.7, gate=gate,
                    act=rng.choice(["identity", "sigmoid", "silu"]),
                    scale=round(rng.uniform(0.1, 1.5), 3))
    hk = rng.choice([1, 2, 4, 8, 16])
    heads = dict(hk=hk, hv=hk * rng.choice([1, 2] if hk > 8 else [1, 2, 4]),
                 dk=rng.choice([64, 128, 128]), dv=rng.choice([64, 128, 128]))
    if op == "step":
        return dict(op="step", b=_log(rng, 1, 256), t=rng.choice([1, 1, 2, 3, 5, 8]), **heads)
    return dict(op="chunk", n=_log(rng, 1, 8192), b=_log(rng, 1, 16), mix=rng.randint(1, 1 << 20),
                state=rng.random() < 0.6, **heads)


def lengths(case):
    """The sequences' lengths: one prompt, or a ragged batch of n tokens in all."""
    n, b = case["n"], case["b"]
    if b == 1:
        return [n]
    g = torch.Generator().manual_seed(case["mix"])
    cuts = torch.randint(0, n + 1, (b - 1,), generator=g).tolist()
    if b > 3:  # an empty sequence, and one of a single token
        cuts[1] = cuts[0]
        cuts[2] = min(cuts[0] + 1, n)
    cuts = [0] + sorted(cuts) + [n]
    return [cuts[i + 1] - cuts[i] for i in range(b)]


def work(case):
    if case["op"] == "norm":
        e = case["rows"] * case["width"]
        per = 1 + case["resid"] + (case["gate"] == "element") + 1 + case["pre"]
        small = case["width"] * (case["post"] + case["pre"] + (case["gate"] == "channel"))
        small += case["rows"] * (case["gate"] == "row")
        return {"bytes": 2 * e * per + 2 * small, "flops": 10 * e}
    if case["op"] == "chunk":
        n, b, states = case["n"], case["b"], 1 + case["state"]
    else:
        n, b, states = case["b"] * case["t"], case["b"], 2
    per_token = 2 * (2 * case["hk"] * case["dk"] + 2 * case["hv"] * case["dv"]) + 8 * case["hv"]
    s = case["hv"] * case["dk"] * case["dv"]
    return {"bytes": n * per_token + 4 * b * s * states, "flops": 6 * n * s}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=DEV) * std

    if case["op"] == "norm":
        rows, width, inner = case["rows"], case["width"], case["inner"]
        shape = (rows // inner, inner, width) if inner > 1 else (rows, width)
        s = dict(case=case, x=normal(*shape).bfloat16(), scale=case["scale"])
        s["resid"] = normal(*shape, std=3.0).bfloat16() if case["resid"] else None
        s["post"] = (1 + normal(width, std=0.2)).bfloat16() if case["post"] else None
        s["pre"] = (1 + normal(width, std=0.2)).bfloat16() if case["pre"] else None
        gate = {"none": None, "channel": (width,), "element": shape, "row": shape[:-1] + (1,)}
        s["gate"] = normal(*gate[case["gate"]]).bfloat16() if gate[case["gate"]] else None
        return s
    b, hk, hv, dk, dv = (case[x] for x in ("b", "hk", "hv", "dk", "dv"))
    step = case["op"] == "step"
    n = b * case["t"] if step else case["n"]
    # q, k and v are slices of one projected row, after the short convolution's silu
    row = F.silu(normal(n, 2 * hk * dk + hv * dv)).bfloat16()
    q, k, v = row.split([hk * dk, hk * dk, hv * dv], dim=1)
    rate = torch.rand(hv, generator=g, device=DEV) * 15.0 + 0.1
    width = torch.exp(normal(n, hv) - 4.0)  # softplus(a + dt_bias): log-normal around 0.02
    s = dict(case=case, q=q.unflatten(1, (hk, dk)), k=k.unflatten(1, (hk, dk)),
             v=v.unflatten(1, (hv, dv)), g=-rate * width, beta=torch.sigmoid(normal(n, hv)))
    carried = step or case["state"]
    s["state"] = normal(b, hv, dv, dk, std=0.1) if carried else None
    s["slots"] = torch.randperm(b, generator=g, device=DEV).int()
    if not step:
        lens = lengths(case)
        s["lens"] = lens
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(b + 1)], dtype=torch.int32, device=DEV)
    s["new_state"] = torch.empty(b, hv, dv, dk, device=DEV)
    if own:
        import sparse_moe_decode_gb300 as moe
        s["mixer"] = moe.GatedDelta(hk, hv, dk, dv, max_tokens=n, max_seqs=b, qk_norm=True,
                                    device=DEV)
    return s


# --------------------------------------------------------------------- run

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "norm":
        return _plain_norm(s)
    return _plain_chunk(s) if op == "chunk" else _plain_step(s)


def _run_own(s, op):
    import sparse_moe_decode_gb300 as moe
    if op == "norm":
        resid, x_next = moe.norm_gate_residual(
            s["x"], gamma_post=s["post"], gate=s["gate"], gate_act=s["case"]["act"],
            resid=s["resid"], res_scale=s["scale"], gamma_pre=s["pre"], eps=EPS)
        return {"resid": resid} if x_next is None else {"resid": resid, "x_next": x_next}
    if op == "chunk":
        out = s["mixer"].chunk(s["q"], s["k"], s["v"], s["g"], s["beta"], cu_seqlens=s["cu"],
                               state_in=s["state"], state_out=s["new_state"], slots=s["slots"])
    else:
        out = s["mixer"].step(s["q"], s["k"], s["v"], s["g"], s["beta"], state_in=s["state"],
                              state_out=s["new_state"], slots=s["slots"])
    return {"out": out, "state": s["new_state"]}


def _gate(gate, act):
    if act == "identity":
        return gate
    return torch.sigmoid(gate) * (gate if act == "silu" else 1.0)


def _plain_norm(s):
    y = s["x"].float()
    if s["post"] is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["post"].float()
    if s["gate"] is not None:
        y = y * _gate(s["gate"].float(), s["case"]["act"])
    y = y * s["scale"]
    if s["resid"] is not None:
        y = y + s["resid"].float()
    resid = y.bfloat16()
    if s["pre"] is None:
        return {"resid": resid}
    r = resid.float()
    x_next = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["pre"].float()
    return {"resid": resid, "x_next": x_next.bfloat16()}


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)


def _states(s):
    """The sequences' states in order [B][Hv][dv][dk], zeros where none is carried."""
    if s["state"] is None:
        return torch.zeros_like(s["new_state"])
    return s["state"][s["slots"].long()]


def _plain_step(s):
    c = s["case"]
    b, t, r = c["b"], c["t"], c["hv"] // c["hk"]
    q = _unit(s["q"].float()).repeat_interleave(r, 1).unflatten(0, (b, t)) * c["dk"] ** -0.5
    k = _unit(s["k"].float()).repeat_interleave(r, 1).unflatten(0, (b, t))
    v = s["v"].float().unflatten(0, (b, t))
    decay, beta = s["g"].exp().unflatten(0, (b, t)), s["beta"].unflatten(0, (b, t))
    S, out = _states(s), []
    for i in range(t):  # the recurrence: each token reads the state the last one left
        S = S * decay[:, i, :, None, None]
        u = beta[:, i, :, None] * (v[:, i] - torch.matmul(S, k[:, i, :, :, None])[..., 0])
        S = S + u[..., None] * k[:, i, :, None, :]
        out.append(torch.matmul(S, q[:, i, :, :, None])[..., 0])
    state = torch.empty_like(s["new_state"])
    state[s["slots"].long()] = S
    return {"out": torch.stack(out, 1).flatten(0, 1).bfloat16(), "state": state}


def _plain_chunk(s):
    """The chunked form: within a chunk the tokens' corrections u solve a unit
    lower-triangular system; the state passes from chunk to chunk."""
    c = s["case"]
    b, n, hv, dk, dv, r = c["b"], c["n"], c["hv"], c["dk"], c["dv"], c["hv"] // c["hk"]
    nc = max(1, -(-max(s["lens"]) // CHUNK))
    at = torch.arange(nc * CHUNK, device=DEV)
    cu = s["cu"].long()
    tok = cu[:-1, None] + at  # [B][nc * CHUNK]
    live = tok < cu[1:, None]
    tok = torch.where(live, tok, 0)

    def cut(x, heads):  # [n][H][..] -> [B][H][nc][CHUNK][..], zeros past a sequence's end
        y = torch.where(live.reshape(b, -1, *[1] * (x.dim() - 1)), x[tok], 0.0)
        return y.unflatten(1, (nc, CHUNK)).movedim(3, 1)

    q = cut(_unit(s["q"].float()).repeat_interleave(r, 1) * dk ** -0.5, hv)
    k = cut(_unit(s["k"].float()).repeat_interleave(r, 1), hv)
    v, beta = cut(s["v"].float(), hv), cut(s["beta"], hv)
    total = cut(s["g"].double(), hv).cumsum(-1)  # [B][Hv][nc][CHUNK]
    pair = (total[..., :, None] - total[..., None, :]).tril().exp().float().tril()
    gamma, rest = total.exp().float(), (total[..., -1:] - total).exp().float()
    low = (beta[..., None] * pair * (k @ k.transpose(-1, -2))).tril(-1)
    inv = torch.eye(CHUNK, device=DEV).expand_as(low).clone()
    for i in range(1, CHUNK):  # forward substitution, all chunks at once
        inv[..., i, :i] = -(low[..., i:i + 1, :i] @ inv[..., :i, :i])[..., 0, :]
    seen = pair * (q @ k.transpose(-1, -2))
    S, out = _states(s).transpose(-1, -2), []
    for i in range(nc):  # the state passes from chunk to chunk
        x = beta[:, :, i, :, None] * (v[:, :, i] - gamma[:, :, i, :, None] * (k[:, :, i] @ S))
        u = inv[:, :, i] @ x
        out.append(gamma[:, :, i, :, None] * (q[:, :, i] @ S) + seen[:, :, i] @ u)
        S = gamma[:, :, i, -1, None, None] * S + (
            (rest[:, :, i, :, None] * k[:, :, i]).transpose(-1, -2) @ u)
    o = torch.stack(out, 2).flatten(2, 3).transpose(1, 2)  # [B][nc * CHUNK][Hv][dv]
    state = torch.empty_like(s["new_state"])
    state[s["slots"].long()] = S.transpose(-1, -2)
    return {"out": o[live].bfloat16(), "state": state}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in fp64: the delta rule one token after another."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        y = s["x"].double()
        if s["post"] is not None:
            y = y / ((y ** 2).sum(-1, keepdim=True) / case["width"] + EPS).sqrt()
            y = y * s["post"].double()
        if s["gate"] is not None:
            z = s["gate"].double()
            y = y * {"identity": lambda: z, "sigmoid": lambda: 1 / (1 + (-z).exp()),
                     "silu": lambda: z / (1 + (-z).exp())}[case["act"]]()
        y = case["scale"] * y + (0.0 if s["resid"] is None else s["resid"].double())
        if s["pre"] is None:
            return {"resid": y}
        r = y.bfloat16().double()  # the stored residual is what the next norm reads
        nxt = r / ((r ** 2).sum(-1, keepdim=True) / case["width"] + EPS).sqrt()
        return {"resid": y, "x_next": nxt * s["pre"].double()}
    b, hk, hv, dk, dv = (case[x] for x in ("b", "hk", "hv", "dk", "dv"))
    lens = s["lens"] if case["op"] == "chunk" else [case["t"]] * b
    if s["state"] is None:
        S = torch.zeros(b, hv, dv, dk, dtype=torch.float64, device=DEV)
    else:
        S = s["state"].double()[s["slots"].long()]
    starts = torch.tensor([sum(lens[:i]) for i in range(b)], device=DEV)
    ends = starts + torch.tensor(lens, device=DEV)
    head = torch.arange(hv, device=DEV) // (hv // hk)
    qd, kd = s["q"].double(), s["k"].double()
    qd = qd / ((qd ** 2).sum(-1, keepdim=True) + EPS).sqrt() / math.sqrt(dk)
    kd = kd / ((kd ** 2).sum(-1, keepdim=True) + EPS).sqrt()
    vd, gd, bd = s["v"].double(), s["g"].double(), s["beta"].double()
    out = torch.zeros(qd.shape[0], hv, dv, dtype=torch.float64, device=DEV)
    for i in range(max(lens)):
        on = (starts + i < ends).nonzero()[:, 0] if b > 1 else slice(None)
        t = (starts + i)[on]
        k, q = kd[t][:, head], qd[t][:, head]
        P = S[on] * gd[t].exp()[:, :, None, None]
        err = vd[t] - (P * k[:, :, None, :]).sum(-1)
        P = P + (bd[t][:, :, None] * err)[..., None] * k[:, :, None, :]
        out[t] = (P * q[:, :, None, :]).sum(-1)
        S[on] = P
    state = torch.empty_like(S)
    state[s["slots"].long()] = S
    return {"out": out, "state": state}
