"""fp64 definitions (numpy) of the gated delta rule and of the norms around a
block, with the bounds that the kernels' roundings allow."""
from __future__ import annotations

import numpy as np

BF16 = 2.0 ** -8   # one rounding to bf16, relative
FP16 = 2.0 ** -11  # one rounding to fp16, relative


def delta_rule(q, k, v, g, beta, S0, scale, qk_norm, eps):
    """One sequence: q, k [L][Hk][dk], v [L][Hv][dv], g, beta [L][Hv], S0
    [Hv][dv][dk].  Returns out [L][Hv][dv], the last state, and for both the
    sums of absolute terms they are made of (what a relative error of every
    operand scales with)."""
    q, k, v, g, beta = (np.asarray(x, np.float64) for x in (q, k, v, g, beta))
    if qk_norm:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + eps)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + eps)
    L, Hv, dv = v.shape
    r = Hv // q.shape[1]
    q, k = q.repeat(r, 1) * scale, k.repeat(r, 1)
    S = np.array(S0, np.float64)
    A = np.abs(S)  # the state's terms without their signs
    out, oabs = np.zeros((L, Hv, dv)), np.zeros((L, Hv, dv))
    for t in range(L):
        a = np.exp(g[t])[:, None, None]
        S, A = a * S, a * A
        u = beta[t][:, None] * (v[t] - np.einsum("hvk,hk->hv", S, k[t]))
        S = S + u[:, :, None] * k[t][:, None, :]
        A = A + np.abs(u)[:, :, None] * np.abs(k[t])[:, None, :]
        out[t] = np.einsum("hvk,hk->hv", S, q[t])
        oabs[t] = np.einsum("hvk,hk->hv", A, np.abs(q[t]))
    return out, S, oabs, A


def out_bound(out, oabs, chunks):
    """One rounding to bf16; each product has two fp16 operands at the least
    exact (2 FP16); the state behind it is off by state_bound's share."""
    return BF16 * np.abs(out) + (2 * FP16 + chunks * 2.0 ** -18) * oabs + 1e-30


def state_bound(A, chunks):
    """Operands of 22 bits and fp32 sums: per run of 64 tokens at most 2^-18 of
    the row's terms."""
    return chunks * 2.0 ** -18 * A.max(-1, keepdims=True) + 1e-30


def rms(x, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def act(z, kind):
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-z))
    return {"identity": z, "sigmoid": s, "silu": z * s}[kind]


def norm_gate(x, post, gate, kind, resid, scale, eps):
    """y before its rounding (fp64)."""
    y = np.asarray(x, np.float64)
    if post is not None:
        y = rms(y, eps) * post
    if gate is not None:
        y = y * act(gate, kind)
    y = y * scale
    return y if resid is None else y + resid
