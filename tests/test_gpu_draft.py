"""Verification of drafted tokens (DraftVerifier) against its definition."""
import numpy as np
import pytest

from attn_ref import verify
from util import gpu_env

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return gpu_env()


def dev_of(env, x, dtype=None):
    import torch
    return torch.tensor(np.asarray(x), dtype=dtype, device=env[1])


def check(env, target, draft, drafted, uniform, strict=True, **kw):
    """All sequences against the definition; where the aim lies within the sums'
    rounding of a border (2^-45 of the total), either side is right."""
    import torch
    moe, dev = env
    v = moe.DraftVerifier(device=dev)
    tokens, accepted = v.verify(target, drafted, uniform, draft=draft, **kw)
    assert tokens.dtype == torch.int32 and accepted.dtype == torch.int32
    p, d, u = (x.cpu().numpy() for x in (target, drafted, uniform))
    q = None if draft is None else draft.cpu().numpy()
    got, acc = tokens.cpu().numpy(), accepted.cpu().numpy()
    for b in range(p.shape[0]):
        a, token, cum, aim = verify(p[b], None if q is None else q[b], d[b], u[b])
        assert acc[b] == a, (b, acc[b], a)
        assert (got[b, :a] == d[b, :a]).all() and (got[b, a + 1:] == -1).all(), b
        if got[b, a] != token:
            lo = cum[got[b, a] - 1] if got[b, a] else 0.0
            assert min(abs(lo - aim), abs(cum[got[b, a]] - aim)) <= 2.0 ** -45 * cum[-1], (
                b, got[b, a], token)
    assert v.status() == 0
    return got, acc


def distributions(env, b, t, v, seed, std=3.0, noise=0.7):
    import torch
    _, dev = env
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((b, t + 1, v), generator=g, device=dev) * std
    target = torch.softmax(x, -1)
    draft = torch.softmax(x[:, :t] + torch.randn((b, t, v), generator=g, device=dev) * noise, -1)
    cum = draft.double().cumsum(-1)
    at = torch.rand((b, t, 1), generator=g, device=dev, dtype=torch.float64) * cum[..., -1:]
    drafted = torch.searchsorted(cum, at, right=True)[..., 0].clamp_max(v - 1).int()
    return target, draft, drafted, torch.rand((b, t + 1), generator=g, device=dev)


@pytest.mark.parametrize("v", [1, 2, 31, 1000, 1023, 1025, 8193, 50257, 151936])
@pytest.mark.parametrize("t", [0, 1, 4, 7])
def test_random(env, v, t):
    b = 40 if v < 10000 else 9
    p, q, d, u = distributions(env, b, t, v, v + t)
    _, acc = check(env, p, q, d, u)
    if v > 100 and t > 1:
        assert 0 < acc.mean() < t  # some stand, some do not
    check(env, p, None, d, u)


@pytest.mark.parametrize("b", [77, 150, 301, 700])
def test_many_sequences(env, b):
    """As many blocks a sequence as the GPU has room for, down to one."""
    p, q, d, u = distributions(env, b, 2, 5000, b)
    check(env, p, q, d, u)
    check(env, p, None, d, u)


def test_the_widest_row(env):
    p, q, d, u = distributions(env, 1, 1, 1 << 24, 3)
    check(env, p, q, d, u)


def test_long_drafts(env):
    p, q, d, u = distributions(env, 6, 90, 300, 5, noise=0.05)
    u *= 0.6
    _, acc = check(env, p, q, d, u)
    assert acc.max() > 32


def test_shorter_drafts_end_at_a_negative_token(env):
    p, q, d, u = distributions(env, 8, 5, 777, 6)
    u[:, :5] = 0.0  # whatever is drafted stands
    for i in range(6):
        d[i, i:] = -1
    d[6, 2] = -(1 << 31)
    got, acc = check(env, p, q, d, u)
    assert acc.tolist() == [0, 1, 2, 3, 4, 5, 2, 5]
    # the place after a draft's end is sampled from the target itself
    want = verify(p[0].cpu().numpy(), None, np.zeros(0, int), u[0, 5:].cpu().numpy())
    assert got[0, 0] == want[1]


def test_borders(env):
    """u q = p is not accepted; sums that meet the aim exactly; zero weights."""
    import torch
    f, i = torch.float32, torch.int32
    p = dev_of(env, [[[0.0, 0.25, 0.25, 0.0, 0.5, 0.0]] * 2] * 8, f)
    q = dev_of(env, [[[0.5, 0.5, 0.0, 0.0, 0.0, 0.0]]] * 8, f)
    d = dev_of(env, [[1], [1], [0], [2], [1], [1], [1], [1]], i)
    e = 2.0 ** -24
    u = dev_of(env, [[0.5, 0.0], [0.5 - 2 * e, 0.0], [0.0, 0.0], [0.9, 0.25], [0.5, 1 / 3],
                     [0.5, 1 - e], [0.5, 0.25], [0.0, 1 - e]], f)
    got, acc = check(env, p, q, d, u)
    # sequence 0: 0.5 * 0.5 = 0.25 falls; rest (0, 0, .25, 0, .5, 0), aim 0: place 2
    assert acc.tolist() == [0, 1, 0, 1, 0, 0, 0, 1]
    # places whose running sum only meets the aim are passed over (sequence 3: aim .25)
    assert got[:, 0].tolist() == [2, 1, 2, 2, 4, 4, 2, 1]
    assert got[:, 1].tolist() == [-1, 1, -1, 2, -1, -1, -1, 4]


def test_target_never_above_draft(env):
    """Nothing is left of p - q: the sample comes from p."""
    import torch
    p = dev_of(env, [[[0.2, 0.3, 0.5], [1.0, 0.0, 0.0]]] * 3, torch.float32)
    q = p[:, :1].clone()
    q[1, 0] = dev_of(env, [0.4, 0.6, 1.0])
    d = dev_of(env, [[2], [2], [2]], torch.int32)
    u = dev_of(env, [[1.0, 0.3], [0.9, 0.9], [0.99, 0.0]], torch.float32)
    got, acc = check(env, p, q, d, u)
    assert acc.tolist() == [0, 0, 1] and got[:, 0].tolist() == [1, 2, 2]


def test_small_differences_keep_their_digits(env):
    """q is p to six digits: the rest is a difference of near values."""
    import torch
    p, _, d, u = distributions(env, 64, 1, 30000, 8)
    g = torch.Generator(device=env[1]).manual_seed(2)
    q = p[:, :1] * (1 + 1e-6 * torch.randn(p[:, :1].shape, generator=g, device=env[1]))
    u[:, 0] = 1.0  # falls wherever q >= p
    _, acc = check(env, p, q, d, u)
    assert (acc == 0).sum() > 10


def test_rows_that_are_no_distributions(env):
    """Any scale, huge and tiny values together, strided and unaligned rows."""
    import torch
    _, dev = env
    p, q, d, u = distributions(env, 7, 3, 3001, 9)
    check(env, p * 1e30, q * 1e30, d, u)
    check(env, p * 1e-30, q * 1e-30, d, u)
    wide = torch.full((7, 5, 3001 + 6), float("nan"), device=dev)
    wide[:, :4, 3:3004] = p
    check(env, wide[:, :4, 3:3004], q, d, u)
    deep = torch.zeros((3, 7, 3001), device=dev)
    deep.copy_(q.transpose(0, 1))
    check(env, p, deep.transpose(0, 1), d, u)
    check(env, p[:1].expand(7, -1, -1), q[:1].expand(7, -1, -1), d, u)


def test_refused_values(env):
    import torch
    moe, dev = env
    p, q, d, u = distributions(env, 6, 2, 2000, 10)
    u[:, :2] = 0.0
    p[0, 2, 1500] = float("nan")
    p[1, 2, 3] = float("inf")
    p[2, 2, 1999] = -1e-9
    p[3, 2] = 0.0
    d[4, 1] = 2000
    d[5, 0] = (1 << 31) - 1
    v = moe.DraftVerifier(device=dev)
    tokens, accepted = v.verify(p[:4], d[:4], u[:4], draft=q[:4])
    assert (tokens == -1).all() and (accepted == 0).all()
    assert v.status() == moe.DEV_NONFINITE
    v.clear_status()
    tokens, accepted = v.verify(p[4:], d[4:], u[4:], draft=q[4:])
    assert (tokens == -1).all() and (accepted == 0).all()
    assert v.status() == moe.DEV_BAD_INDEX
    # rows that no sample is taken from are not looked at
    v.clear_status()
    p[0] = p[4]
    p[0, 0, 7] = float("nan") if d[0, 0] != 7 else p[0, 0, 7]
    p[0, 0, d[0, 0]] = 1.0
    p[0, 1, d[0, 1]] = 1.0
    tokens, accepted = v.verify(p[:1], d[:1], u[:1], draft=q[:1])
    assert accepted.item() == 2 and v.status() == 0


def test_numbers_out_of_range(env):
    """Below 0 and NaN as 0, from 1 on the last weight."""
    import torch
    moe, dev = env
    p = torch.zeros((6, 1, 3000), device=dev)
    p[:, 0, 1000], p[:, 0, 2000] = 0.25, 0.75
    none = torch.empty((6, 0), dtype=torch.int32, device=dev)
    u = torch.tensor([-1.0, float("nan"), -float("inf"), 1.0, 7.0, float("inf")], device=dev)
    v = moe.DraftVerifier(device=dev)
    tokens, accepted = v.verify(p, none, u[:, None])
    assert tokens[:, 0].tolist() == [1000] * 3 + [2000] * 3
    assert (accepted == 0).all() and v.status() == 0


def test_outputs_capture_and_checks(env):
    import torch
    moe, dev = env
    p, q, d, u = distributions(env, 5, 4, 9999, 11)
    v = moe.DraftVerifier(device=dev)
    want = v.verify(p, d, u, draft=q)
    tokens = torch.zeros((5, 5), dtype=torch.int32, device=dev)
    accepted = torch.zeros(5, dtype=torch.int32, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        v.verify(p, d, u, draft=q, tokens=tokens, accepted=accepted)
    for seed in (11, 12, 13):
        for x, y in zip((p, q, d, u), distributions(env, 5, 4, 9999, seed)):
            x.copy_(y)
        graph.replay()
        want = v.verify(p, d, u, draft=q)
        assert torch.equal(tokens, want[0]) and torch.equal(accepted, want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = v.verify(p, d, u, draft=q, stream=side)
    side.synchronize()
    assert torch.equal(other[0], want[0])
    for bad in (lambda: v.verify(p.double(), d, u, draft=q), lambda: v.verify(p, d.long(), u, draft=q),
                lambda: v.verify(p, d, u[:, :4], draft=q), lambda: v.verify(p, d, u, draft=q[:, :3]),
                lambda: v.verify(p[:, :, ::2], d, u), lambda: v.verify(p, d[:3], u, draft=q),
                lambda: v.verify(p, d, u, draft=q, tokens=tokens[:, :4]),
                lambda: v.verify(p.cpu(), d, u, draft=q)):
        with pytest.raises(moe.MoEError):
            bad()
    empty = v.verify(p[:0], d[:0], u[:0], draft=q[:0])
    assert empty[0].shape == (0, 5) and empty[1].shape == (0,)
    assert v.status() == 0
