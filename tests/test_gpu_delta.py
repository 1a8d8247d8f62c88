"""The gated delta rule (moe_delta_chunk, moe_delta_step) against its fp64
definition, token by token; the bounds stand in mixer_ref."""
import numpy as np
import pytest

from mixer_ref import delta_rule, out_bound, state_bound
from util import gpu_env

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def env():
    return gpu_env()


def f64(t):
    return t.double().cpu().numpy()


def make(env, n, heads=(2, 4), dims=(128, 128), seed=0, k_std=1.0, v_std=1.0, guard=3):
    """Token rows as slices of one projected buffer with `guard` NaN rows
    before and after them."""
    import torch
    _, dev = env
    (hk, hv), (dk, dv) = heads, dims
    g = torch.Generator(device=dev).manual_seed(1000 * seed + n)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def guarded(t):
        buf = torch.full((n + 2 * guard, t.shape[1]), float("nan"), dtype=t.dtype, device=dev)
        buf[guard:guard + n] = t
        return buf[guard:guard + n]

    row = torch.cat([normal(n, hk * dk), k_std * normal(n, hk * dk), v_std * normal(n, hv * dv)], 1)
    q, k, v = guarded(row.bfloat16()).split([hk * dk, hk * dk, hv * dv], 1)
    gb = guarded(torch.cat([-torch.exp(1.5 * normal(n, hv) - 2.0), torch.sigmoid(normal(n, hv))], 1))
    return dict(q=q.unflatten(1, (hk, dk)), k=k.unflatten(1, (hk, dk)),
                v=v.unflatten(1, (hv, dv)), g=gb[:, :hv], beta=gb[:, hv:])


def states(env, slots, heads, dims, seed=0):
    import torch
    _, dev = env
    g = torch.Generator(device=dev).manual_seed(77 + seed)
    return torch.randn((slots, heads[1], dims[1], dims[0]), generator=g, device=dev) * 0.2


def mixer(env, heads, dims, n, b, qk_norm=True):
    moe, dev = env
    return moe.GatedDelta(*heads, *dims, max_tokens=n, max_seqs=b, qk_norm=qk_norm, qk_eps=EPS,
                          device=dev)


def cu_of(env, lens):
    import torch
    _, dev = env
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)


def check_seq(s, rows, S0, out, S1, dims, qk_norm=True):
    """One sequence's rows (a slice) against the definition."""
    c = {x: f64(s[x][rows]) for x in ("q", "k", "v", "g", "beta")}
    want, S, oabs, A = delta_rule(**c, S0=f64(S0), scale=dims[0] ** -0.5, qk_norm=qk_norm, eps=EPS)
    chunks = 1 + want.shape[0] // 64
    err = np.abs(f64(out[rows]) - want)
    assert not (err > out_bound(want, oabs, chunks)).any() and not np.isnan(err).any(), err.max()
    if S1 is not None:
        err = np.abs(f64(S1) - S)
        assert not (err > state_bound(A, chunks)).any() and not np.isnan(err).any(), err.max()


def run_chunk(env, s, lens, heads, dims, state=True, qk_norm=True, in_place=False, seed=0):
    import torch
    _, dev = env
    n, b = sum(lens), len(lens)
    m = mixer(env, heads, dims, n, b, qk_norm)
    pool = states(env, b + 2, heads, dims, seed)
    slots = torch.from_numpy(np.random.RandomState(seed).permutation(b + 2)[:b].astype(np.int32))
    slots = slots.to(dev)
    given = pool.clone()
    S1 = pool if in_place else torch.full_like(pool, 7.0)
    out = m.chunk(**s, cu_seqlens=cu_of(env, lens), slots=slots, state_in=pool if state else None,
                  state_out=S1)
    assert m.status() == 0
    at = 0
    for i, L in enumerate(lens):
        S0 = given[slots[i]] if state else torch.zeros_like(given[0])
        check_seq(s, slice(at, at + L), S0, out, S1[slots[i]], dims, qk_norm)
        at += L
    rest = [x for x in range(b + 2) if x not in slots.tolist()]
    assert torch.equal(S1[rest], given[rest] if in_place else torch.full_like(given[rest], 7.0))
    return out, S1


@pytest.mark.parametrize("n", [1, 2, 7, 15, 16, 17, 31, 33, 63, 64, 65, 100, 128, 129, 200])
def test_chunk_one_sequence(env, n):
    s = make(env, n)
    run_chunk(env, s, [n], (2, 4), (128, 128))
    run_chunk(env, s, [n], (2, 4), (128, 128), state=False)


@pytest.mark.parametrize("dims", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("heads", [(1, 1), (1, 3), (2, 2), (3, 12)])
def test_chunk_ragged(env, heads, dims):
    lens = [70, 0, 1, 64, 130, 3]
    run_chunk(env, make(env, sum(lens), heads, dims, seed=1), lens, heads, dims)


def test_chunk_many_sequences_in_place(env):
    lens = [int(x) for x in np.random.RandomState(3).randint(0, 90, 40)]
    run_chunk(env, make(env, sum(lens), (1, 2), (64, 64)), lens, (1, 2), (64, 64), in_place=True)


@pytest.mark.parametrize("lens,heads", [
    ([int(x) for x in np.random.RandomState(4).randint(0, 140, 40)], (2, 8)),
    ([int(x) for x in np.random.RandomState(5).randint(0, 4, 290)] + [130, 0, 70] + [1] * 10, (1, 4)),
    ([1] * 70, (4, 16)), ([64, 0] * 20, (2, 16)), ([0] * 30 + [200] + [0] * 30, (2, 16))])
def test_chunk_more_work_than_blocks(env, lens, heads):
    """Several pieces of work for every block of the second kernel; more
    sequences than are put in order at a time; sequences without tokens.  The
    order of the batch changes no bit of any sequence."""
    import torch
    moe, dev = env
    dims, n, b = (128, 64), sum(lens), len(lens)
    s = make(env, n, heads, dims, seed=7)
    m = mixer(env, heads, dims, n, b)
    pool = states(env, b, heads, dims)
    S1 = torch.full_like(pool, 7.0)
    out = m.chunk(**s, cu_seqlens=cu_of(env, lens), state_in=pool, state_out=S1)
    assert m.status() == 0 and out.isfinite().all() and S1.isfinite().all()
    ends = np.cumsum(lens)
    for i, L in enumerate(lens):
        assert L or torch.equal(S1[i], pool[i])
        assert not L or not torch.equal(S1[i], pool[i])
    rows = torch.tensor([r for e, L in zip(ends[::-1], lens[::-1]) for r in range(e - L, e)],
                        device=dev)
    slots = torch.arange(b - 1, -1, -1, dtype=torch.int32, device=dev)
    again = m.chunk(**{x: t[rows].contiguous() for x, t in s.items()},
                    cu_seqlens=cu_of(env, lens[::-1]), state_in=pool, state_out=pool, slots=slots)
    assert m.status() == 0
    assert torch.equal(again, out[rows]) and torch.equal(pool, S1)


@pytest.mark.parametrize("heads,dims", [((2, 4), (128, 128)), ((4, 16), (64, 64))])
def test_chunk_sequence_alone_and_in_a_batch(env, heads, dims):
    """No bit of a sequence depends on the call it is part of: short ones and
    long ones, among others of both kinds, some of them not finite."""
    import torch
    moe, dev = env
    lens = [24, 25, 1, 0, 64, 200, 23, 3, 65, 130, 26, 2] + [5, 90] * 20
    n, b = sum(lens), len(lens)
    s = make(env, n, heads, dims, seed=11)
    pool = states(env, b, heads, dims)
    m = mixer(env, heads, dims, n, b)
    S1 = torch.full_like(pool, 7.0)
    out = m.chunk(**s, cu_seqlens=cu_of(env, lens), state_in=pool, state_out=S1)
    assert m.status() == 0
    ends = np.cumsum(lens)
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 10, b - 2, b - 1):
        r = slice(ends[i] - lens[i], ends[i])
        S2 = torch.empty_like(pool[:1])
        o = m.chunk(**{x: t[r] for x, t in s.items()}, cu_seqlens=cu_of(env, [lens[i]]),
                    state_in=pool[i:i + 1].clone(), state_out=S2)
        assert torch.equal(o, out[r]) and torch.equal(S2[0], S1[i])
    bad = {x: t.clone() for x, t in s.items()}
    for i in (4, 6, b - 3):  # infinities and NaN in a few sequences
        r = slice(ends[i] - lens[i], ends[i])
        bad["v"][r] = float("inf")
        bad["k"][r] = float("nan")
    S2 = torch.full_like(pool, 7.0)
    o = m.chunk(**bad, cu_seqlens=cu_of(env, lens), state_in=pool, state_out=S2)
    for i in range(b):
        if i not in (4, 6, b - 3):
            r = slice(ends[i] - lens[i], ends[i])
            assert torch.equal(o[r], out[r]) and torch.equal(S2[i], S1[i])


def test_chunk_tiny_values_beside_large_ones(env):
    """A reset, then values far below those of the tokens before it: the
    prompt form keeps 2^-36 of the largest value of the same 64 tokens and state
    row (two fp16 terms, their scale from a bound up to 2^4 above it, sums of 64
    products: 2^-33 in all), and 22 bits of what is above 2^-17 of it."""
    import torch
    _, dev = env
    heads, dims, n = (2, 4), (128, 128), 60
    s = make(env, n, heads, dims, seed=9)
    s["g"][50] = -40.0
    s["v"][50:] *= 2.0 ** -21
    m = mixer(env, heads, dims, n, 1)
    S1 = torch.empty((1, 4, 128, 128), device=dev)
    m.chunk(**s, state_out=S1)
    c = {x: f64(s[x]) for x in ("q", "k", "v", "g", "beta")}
    zero = np.zeros((4, 128, 128))
    _, S, _, A = delta_rule(**c, S0=zero, scale=1.0, qk_norm=True, eps=EPS)
    _, Sb, _, _ = delta_rule(**{x: t[:50] for x, t in c.items()}, S0=zero, scale=1.0, qk_norm=True,
                             eps=EPS)
    most = np.abs(c["v"]).max(0) + np.sqrt((Sb * Sb).sum(-1))  # [Hv][dv]
    err = np.abs(f64(S1[0]) - S)
    assert not (err > state_bound(A, 1) + 2.0 ** -33 * most[:, :, None]).any(), err.max()


def test_chunk_long(env):
    run_chunk(env, make(env, 1500, (1, 2)), [1500], (1, 2), (128, 128))


@pytest.mark.parametrize("heads", [(128, 256), (84, 252), (64, 256), (51, 255)])
def test_chunk_shared_preparation(env, heads):
    """Enough chunks and key heads for a block of the first kernel to serve two,
    three or four value heads; one where their ratio has none of these."""
    lens = [130, 0, 1, 64, 65, 3] + [0] * 13 + [2]
    run_chunk(env, make(env, sum(lens), heads, (64, 64), seed=4), lens, heads, (64, 64))


@pytest.mark.parametrize("dims", [(64, 128), (128, 64)])
@pytest.mark.parametrize("lens", [[16], [1, 0, 3], [0, 5, 11, 0], [1] * 16, [0] * 63 + [9],
                                  [0] * 64 + [9], [17], [8, 9]])
def test_chunk_few_rows(env, lens, dims):
    """Both sides of the rule that sends calls of few rows token by token."""
    run_chunk(env, make(env, sum(lens), (2, 6), dims, seed=5), lens, (2, 6), dims, seed=2)
    run_chunk(env, make(env, sum(lens), (2, 6), dims, seed=6), lens, (2, 6), dims, state=False,
              in_place=True)


@pytest.mark.parametrize("k_std", [0.05, 1e-6])
def test_chunk_without_norm(env, k_std):
    """k as it is (small enough for the rule to contract), tiny k too."""
    lens = [150, 20]
    run_chunk(env, make(env, 170, k_std=k_std, v_std=30.0), lens, (2, 4), (128, 128),
              qk_norm=False)


def test_chunk_without_norm_unit_keys_repeated(env):
    """The same unit key for every token with beta 1: each token replaces
    what the last one wrote, and the inverse's entries alternate."""
    import torch
    s = make(env, 130)
    s["k"].zero_()
    s["k"][:, :, 5] = 1.0
    s["beta"].fill_(1.0)
    run_chunk(env, s, [130], (2, 4), (128, 128), qk_norm=False)


def test_chunk_gate_extremes(env):
    """Resets (-inf, -1000), no decay at all, beta 0 and 1, zero keys and
    queries, and infinite decay beside very slow ones."""
    s = make(env, 200)
    s["g"][10] = -float("inf")
    s["g"][70:72] = -1000.0
    s["g"][90] = -600.0
    s["g"][91:140] = -1e-3
    s["g"][140:180] = 0.0
    s["beta"][20:30] = 0.0
    s["beta"][40:50] = 1.0
    s["k"][60:66] = 0.0
    s["q"][66] = 0.0
    run_chunk(env, s, [200], (2, 4), (128, 128))
    run_chunk(env, s, [64, 136], (2, 4), (128, 128))


def test_chunk_slow_decay_after_a_reset_keeps_its_bits(env):
    """Sums of logarithms that reach -40000 within a run of 64 tokens do not
    cost the later, slow decays their digits."""
    s = make(env, 128)
    s["g"][:] = -0.001
    s["g"][::2] = -120.0
    s["g"][40:] = -0.0123
    run_chunk(env, s, [128], (2, 4), (128, 128))


def test_sequences_do_not_see_one_another(env):
    """A sequence's bits do not depend on its neighbours, NaN among them."""
    import torch
    moe, dev = env
    lens = [80, 40, 200]
    s = make(env, 320)
    want, S = run_chunk(env, s, lens, (2, 4), (128, 128))
    s["v"][85] = float("nan")
    s["k"][90] = float("inf")
    m = mixer(env, (2, 4), (128, 128), 320, 3)
    pool = states(env, 5, (2, 4), (128, 128))
    slots = torch.from_numpy(np.random.RandomState(0).permutation(5)[:3].astype(np.int32)).to(dev)
    S1 = torch.full_like(pool, 7.0)
    out = m.chunk(**s, cu_seqlens=cu_of(env, lens), slots=slots, state_in=pool, state_out=S1)
    for rows, i in ((slice(0, 80), 0), (slice(120, 320), 2)):
        assert torch.equal(out[rows], want[rows])
        assert torch.equal(S1[slots[i]], S[slots[i]])
    assert torch.isnan(out[119]).all()


@pytest.mark.parametrize("api", ["chunk", "step"])
def test_skipped_and_bad_sequences(env, api):
    """A negative slot skips its sequence; a slot out of range does too and
    sets the status bit; nothing of either is written."""
    import torch
    moe, dev = env
    heads, dims = (2, 4), (128, 128)
    T = 70 if api == "chunk" else 5
    s = make(env, 4 * T, heads, dims)
    for third, bit in ((-1, 0), (6, moe.DEV_BAD_INDEX)):
        m = mixer(env, heads, dims, 4 * T, 4)
        pool = states(env, 6, heads, dims)
        slots = torch.tensor([4, -1, third, 0], dtype=torch.int32, device=dev)
        out = torch.full((4 * T, 4, 128), 3.0, dtype=torch.bfloat16, device=dev)
        S1 = torch.full_like(pool, 7.0)
        kw = dict(state_in=pool, state_out=S1, slots=slots, out=out)
        if api == "chunk":
            m.chunk(**s, cu_seqlens=cu_of(env, [T] * 4), **kw)
        else:
            m.step(**s, **kw)
        assert m.status() == bit
        m.clear_status()
        assert m.status() == 0
        assert (out[T:3 * T] == 3.0).all() and (S1[[1, 2, 3, 5]] == 7.0).all()
        for i in (0, 3):
            check_seq(s, slice(i * T, i * T + T), pool[slots[i]], out, S1[slots[i]], dims)


@pytest.mark.parametrize("cu", [[0, 100, 50, 120], [-5, 20, 60, 120], [0, 40, 80, 121],
                                [0, 40, 1 << 30, 120]])
def test_bad_bounds_are_skipped(env, cu):
    """Bounds that are not 0 <= start <= end <= N set the status bit, and
    nothing is written."""
    import torch
    moe, dev = env
    heads, dims = (1, 2), (64, 64)
    s = make(env, 120, heads, dims)
    m = mixer(env, heads, dims, 120, 3)
    S1 = torch.full((3, 2, 64, 64), 7.0, device=dev)
    out = torch.full((120, 2, 64), 3.0, dtype=torch.bfloat16, device=dev)
    m.chunk(**s, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev), state_out=S1, out=out)
    assert m.status() == moe.DEV_BAD_INDEX
    assert (S1 == 7.0).all() and (out == 3.0).all()
    # the next call is not affected
    m.clear_status()
    m.chunk(**s, cu_seqlens=cu_of(env, [50, 0, 70]), state_out=S1, out=out)
    assert m.status() == 0
    check_seq(s, slice(0, 50), torch.zeros_like(S1[0]), out, S1[0], dims)
    check_seq(s, slice(50, 120), torch.zeros_like(S1[0]), out, S1[2], dims)


@pytest.mark.parametrize("cu", [[0, 8, 4, 12], [-1, 4, 6, 12], [0, 4, 8, 13], [0, 4, 1 << 30, 12]])
def test_bad_bounds_of_few_rows_are_skipped(env, cu):
    import torch
    moe, dev = env
    heads, dims = (1, 2), (64, 64)
    s = make(env, 12, heads, dims)
    m = mixer(env, heads, dims, 12, 3)
    S1 = torch.full((3, 2, 64, 64), 7.0, device=dev)
    out = torch.full((12, 2, 64), 3.0, dtype=torch.bfloat16, device=dev)
    m.chunk(**s, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev), state_out=S1, out=out)
    assert m.status() == moe.DEV_BAD_INDEX
    assert (S1 == 7.0).all() and (out == 3.0).all()
    m.clear_status()
    # a slot out of range, and one that skips
    slots = torch.tensor([2, 3, -1], dtype=torch.int32, device=dev)
    m.chunk(**s, cu_seqlens=cu_of(env, [5, 4, 3]), slots=slots, state_out=S1, out=out)
    assert m.status() == moe.DEV_BAD_INDEX
    assert (S1[:2] == 7.0).all() and (out[5:] == 3.0).all()
    check_seq(s, slice(0, 5), torch.zeros_like(S1[0]), out, S1[2], dims)


@pytest.mark.parametrize("dims", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (2, 2), (5, 5), (1, 17), (70, 1)])
def test_step(env, B, T, dims):
    import torch
    _, dev = env
    heads = (2, 4)
    s = make(env, B * T, heads, dims, seed=2)
    m = mixer(env, heads, dims, B * T, B)
    pool = states(env, B + 1, heads, dims)
    given = pool.clone()
    slots = torch.arange(B, 0, -1, dtype=torch.int32, device=dev)
    S1 = torch.full_like(pool, 7.0)
    out = m.step(**s, state_in=pool, state_out=S1, slots=slots)
    for i in range(B):
        check_seq(s, slice(i * T, i * T + T), given[slots[i]], out, S1[slots[i]], dims)
    assert (S1[0] == 7.0).all()
    inp = m.step(**s, state_in=pool, state_out=pool, slots=slots)
    assert torch.equal(inp, out) and torch.equal(pool[1:], S1[1:])
    again = m.step(**s, state_in=given, slots=slots)  # the state is not kept
    assert torch.equal(again, out)


def test_step_zero_state_and_no_norm(env):
    heads, dims = (4, 4), (128, 64)
    s = make(env, 12, heads, dims, k_std=0.05)
    m = mixer(env, heads, dims, 12, 3, qk_norm=False)
    import torch
    S1 = torch.empty((3, 4, 64, 128), device=env[1])
    out = m.step(**s, state_out=S1, tokens=4)
    for i in range(3):
        check_seq(s, slice(4 * i, 4 * i + 4), torch.zeros_like(S1[0]), out, S1[i], dims, False)


def test_prompt_then_steps(env):
    """A prompt in one call, then tokens one at a time on its state, is the
    whole sequence."""
    import torch
    heads, dims = (2, 4), (128, 128)
    n = 140
    s = make(env, n, heads, dims)
    m = mixer(env, heads, dims, n, 1)
    state = torch.zeros((1, 4, 128, 128), device=env[1])
    cut = {k: v[:130] for k, v in s.items()}
    outs = [m.chunk(**cut, state_in=state, state_out=state)]
    for t in range(130, n):
        outs.append(m.step(**{k: v[t:t + 1] for k, v in s.items()}, state_in=state,
                           state_out=state))
    check_seq(s, slice(0, n), torch.zeros_like(state[0]), torch.cat(outs), state[0], dims)


def test_empty_calls(env):
    import torch
    moe, dev = env
    s = make(env, 0, guard=1)
    m = mixer(env, (2, 4), (128, 128), 8, 4)
    pool = states(env, 2, (2, 4), (128, 128))
    S1 = torch.full_like(pool, 7.0)
    out = m.chunk(**s, cu_seqlens=cu_of(env, [0, 0]), state_in=pool, state_out=S1)
    assert out.shape == (0, 4, 128) and torch.equal(S1, pool)  # no tokens: the state as it was
    m.chunk(**s, cu_seqlens=cu_of(env, []), state_in=pool, state_out=S1)
    m.step(**s, state_in=pool, state_out=S1, tokens=0)


def test_tensors_are_checked(env):
    import torch
    moe, dev = env
    s = make(env, 12)
    m = mixer(env, (2, 4), (128, 128), 12, 3)
    st = states(env, 3, (2, 4), (128, 128))
    slots = torch.arange(3, dtype=torch.int32, device=dev)
    bad = [dict(q=s["q"][:11]), dict(k=s["k"].float()), dict(v=s["v"].transpose(1, 2)),
           dict(v=s["v"].cpu()), dict(g=s["g"].double()), dict(beta=s["beta"][:, :2]),
           dict(q=s["q"][:, 0]), dict(state_in=st[:2]), dict(state_in=st.transpose(2, 3)),
           dict(state_in=st.bfloat16()), dict(slots=slots.long()),
           dict(out=torch.empty(12, 4, 64, dtype=torch.bfloat16, device=dev))]
    for kw in bad:
        with pytest.raises(moe.MoEError):
            m.step(**{**s, "state_in": st, "state_out": st, "slots": slots, **kw})
    for kw in bad + [dict(slots=slots[:2])]:
        with pytest.raises(moe.MoEError):
            m.chunk(**{**s, "cu_seqlens": cu_of(env, [4, 4, 4]), "state_in": st, "state_out": st,
                       "slots": slots, **kw})
    with pytest.raises(moe.MoEError):
        m.chunk(**s, cu_seqlens=cu_of(env, [12]).long())
    m.step(**s, state_in=st, state_out=st, slots=slots)


def test_workspace_is_checked(env):
    moe, _ = env
    big = make(env, 4096)
    m = mixer(env, (2, 4), (128, 128), 8, 1)
    with pytest.raises(moe.MoEError):
        m.chunk(**big, cu_seqlens=cu_of(env, [4096]))  # more rows than max_tokens


def test_streams_and_graphs(env):
    import torch
    heads, dims = (2, 4), (128, 128)
    s = make(env, 150, heads, dims)
    m = mixer(env, heads, dims, 150, 1)
    state = states(env, 1, heads, dims)
    S1, S2 = torch.empty_like(state), torch.empty_like(state)
    want = m.chunk(**s, state_in=state, state_out=S1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = m.chunk(**s, state_in=state, state_out=S2)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(want, got) and torch.equal(S1, S2)
    out = torch.zeros_like(want)
    tok = {k: v[:1] for k, v in s.items()}
    tout = torch.zeros_like(want[:1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.chunk(**s, state_in=state, state_out=S2, out=out)
        m.step(**tok, state_in=S2, state_out=S2, out=tout)
    S2.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert torch.equal(tout, m.step(**tok, state_in=S1, state_out=S1))
    assert torch.equal(S1, S2)


def test_state_offsets_beyond_32_bits(env):
    """A pool whose last slot starts past 2^31 values."""
    import torch
    _, dev = env
    heads, dims = (2, 32), (128, 128)
    pool = torch.empty((4200, 32, 128, 128), device=dev)
    last = states(env, 1, heads, dims)[0]
    slots = torch.tensor([4199], dtype=torch.int32, device=dev)
    for n, api in ((3, "step"), (70, "chunk")):
        s = make(env, n, heads, dims)
        m = mixer(env, heads, dims, n, 1)
        pool[4199] = last
        out = getattr(m, api)(**s, state_in=pool, state_out=pool, slots=slots,
                              **({"cu_seqlens": cu_of(env, [n])} if api == "chunk" else {}))
        check_seq(s, slice(0, n), last, out, pool[4199], dims)


def _no_writes(s):
    s["beta"].zero_()


def _last_writes_nothing(s):
    s["beta"][-1] = 0.0


def _run_writes_nothing(s):
    s["beta"][64:128] = 0.0


def _zeros(s):
    for x in "qkv":
        s[x].zero_()


def _padding(rows):
    def apply(s):
        for x in "qkv":
            s[x][:rows] = 0.0
    return apply


def _resets_beside_zero_channels(s):
    s["g"][0] = -float("inf")
    s["g"][64] = -1000.0
    s["v"][:64, :, 3] = 0.0
    s["v"][64:128, 1] = 0.0


def _silent_channels(s):
    s["v"][:, :, 5] = 0.0
    s["v"][:64, 1] = 0.0
    s["beta"].mul_(0.005)
    s["g"][:] = -0.02


def _tiny_values(s):
    s["v"].mul_(2.0 ** -118)


def check_both_forms(env, edit, n, dims, state):
    """A sequence in chunks and token by token, each as the definition has it."""
    import torch
    heads = (2, 4)
    s = make(env, n, heads, dims, seed=12)
    edit(s)
    run_chunk(env, s, [n], heads, dims, state=state)
    m = mixer(env, heads, dims, n, 1)
    S0 = states(env, 1, heads, dims) if state else None
    S1 = torch.empty_like(states(env, 1, heads, dims))
    out = m.step(**s, state_in=S0, state_out=S1, tokens=n)
    check_seq(s, slice(0, n), torch.zeros_like(S1[0]) if S0 is None else S0[0], out, S1[0], dims)


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("dims", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("edit,n", [
    (_no_writes, 70), (_no_writes, 64), (_last_writes_nothing, 65), (_last_writes_nothing, 129),
    (_run_writes_nothing, 200), (_zeros, 70), (_padding(64), 130), (_padding(100), 160),
    (_resets_beside_zero_channels, 150), (_silent_channels, 140)])
def test_chunk_where_little_or_nothing_is_written(env, edit, n, dims, state):
    """Runs of 64 tokens whose corrections are zero or nearly so (masked and
    padded tokens, zero channels), with a carried state and without."""
    check_both_forms(env, edit, n, dims, state)


@pytest.mark.parametrize("dims", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_chunk_values_near_the_smallest(env, dims):
    """(From a zero state: beside a larger one they would be below the prompt
    form's floor.)"""
    check_both_forms(env, _tiny_values, 100, dims, False)


def _large_values(s):
    s["v"].mul_(2.0 ** 118)


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("dims", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_chunk_values_near_the_largest(env, dims, state):
    """Finite as long as the states and outputs themselves are."""
    check_both_forms(env, _large_values, 100, dims, state)


def busy_with(env, like):
    """Work on the current stream that still has to read a block of `like`'s size,
    which nobody holds any more: (where it lies, what was read, what it holds)."""
    import torch
    block = torch.full_like(like, 5.0)
    read = torch.zeros_like(like)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    read.copy_(block)
    return block.data_ptr(), read


@pytest.mark.parametrize("api", ["chunk", "step"])
def test_results_on_a_given_stream(env, api):
    """A result made for a call on another stream is not the memory of work
    that is still to come on the current one."""
    import torch
    heads, dims, n = (2, 4), (128, 128), 3001
    s = make(env, n, heads, dims)
    m = mixer(env, heads, dims, n, 1)
    call = lambda **kw: getattr(m, api)(**s, **kw, **({"tokens": n} if api == "step" else {}))
    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    where, read = busy_with(env, want)
    out = call(stream=side)
    assert out.data_ptr() != where
    torch.cuda.synchronize()
    assert (read == 5.0).all() and torch.equal(out, want)
    assert torch.equal(call(stream=torch.cuda.current_stream().cuda_stream), want)


@pytest.mark.parametrize("api", ["chunk", "step"])
def test_written_tensors_count_a_version(env, api):
    """Autograd learns that a kept tensor has been overwritten; without
    gradients (inference mode) nothing is counted, and nothing else changes."""
    import torch
    heads, dims, n = (2, 4), (64, 64), 40
    s = make(env, n, heads, dims)
    m = mixer(env, heads, dims, n, 1)
    S0 = states(env, 1, heads, dims)
    S1, out = torch.empty_like(S0), torch.empty(n, 4, 64, dtype=torch.bfloat16, device=env[1])
    call = lambda **kw: getattr(m, api)(**s, **kw, **({"tokens": n} if api == "step" else {}))
    read = list(s.values()) + [S0]
    before = [t._version for t in read + [S1, out]]
    call(state_in=S0, state_out=S1, out=out)
    after = [t._version for t in read + [S1, out]]
    assert after == before[:-2] + [before[-2] + 1, before[-1] + 1]
    x = torch.randn(n, 4, 64, dtype=torch.bfloat16, device=env[1], requires_grad=True)
    kept = x.detach()
    y = (x * kept).sum()
    call(out=kept)
    with pytest.raises(RuntimeError):
        y.backward()
    with torch.inference_mode():
        again = torch.empty_like(out)
        assert torch.equal(call(state_in=S0, out=again), out)


@pytest.mark.parametrize("T", [8, 30])
def test_verification_keeps_the_accepted_state(env, T):
    """A verified draft's outputs, then the states after the accepted tokens of
    each sequence: a call over the same rows, the rejected ones in a slot of -1."""
    import torch
    _, dev = env
    heads, dims = (2, 4), (128, 128)
    accepted = torch.tensor([1, T, 0, T - 3, 4], dtype=torch.int32, device=dev)
    B = len(accepted)
    s = make(env, B * T, heads, dims, seed=3)
    m = mixer(env, heads, dims, B * T, 2 * B)
    S = states(env, B + 1, heads, dims)
    given = S.clone()
    slots = torch.arange(B, 0, -1, dtype=torch.int32, device=dev)
    out = m.step(**s, state_in=S, slots=slots)
    assert torch.equal(S, given)
    start = T * torch.arange(B, dtype=torch.int32, device=dev)
    cut = torch.stack([start, start + accepted], 1).flatten()
    rest = slots.new_full((B,), -1)
    m.chunk(**s, cu_seqlens=torch.cat([cut, cut.new_tensor([B * T])]), state_in=S, state_out=S,
            slots=torch.stack([slots, rest], 1).flatten())
    assert m.status() == 0 and torch.equal(S[0], given[0])
    for i, n in enumerate(accepted.tolist()):
        c = slice(i * T, i * T + n)
        check_seq(s, c, given[slots[i]], out, S[slots[i]], dims)
