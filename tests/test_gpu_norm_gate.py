"""moe_norm_gate_residual against the fp64 definition.

Bounds: resid_out is one rounding to bf16 of an fp32 value (a handful of fp32
operations on each term: 2^-20 of the terms); x_next likewise, from the
stored residual."""
import numpy as np
import pytest

from mixer_ref import BF16, norm_gate, rms
from util import gpu_env

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def env():
    return gpu_env()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make(env, rows, width, inner=1, gate="element", post=True, pre=True, resid=True, seed=0,
         pad=0):
    """Inputs whose rows lie `pad` values further apart than they are long,
    with NaN between them."""
    import torch
    _, dev = env
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).bfloat16()

    shape = (rows // inner, inner, width) if inner > 1 else (rows, width)

    def laid(t):
        n = t[0].numel() if t.shape[0] else inner * width
        buf = torch.full((t.shape[0], n + pad), float("nan"), dtype=t.dtype, device=dev)
        buf[:, :n] = t.flatten(1)
        return buf[:, :n].unflatten(1, t.shape[1:])

    s = dict(x=laid(normal(*shape)), resid=laid(normal(*shape, std=3.0)) if resid else None,
             post=normal(width) if post else None, pre=normal(width) if pre else None)
    s["gate"] = {"none": lambda: None, "channel": lambda: normal(width),
                 "element": lambda: laid(normal(*shape)),
                 "row": lambda: normal(*shape[:-1], 1)}[gate]()
    return s


def check(env, s, kind="sigmoid", scale=0.5, **kw):
    moe, _ = env
    with np.errstate(all="ignore"):
        term = norm_gate(f64(s["x"]), f64(s["post"]), f64(s["gate"]), kind, None, scale, EPS)
        res = 0.0 if s["resid"] is None else f64(s["resid"])
        want = term + res
    r, n = moe.norm_gate_residual(s["x"], gamma_post=s["post"], gate=s["gate"], gate_act=kind,
                                  resid=s["resid"], res_scale=scale, gamma_pre=s["pre"], eps=EPS,
                                  **kw)
    got = f64(r)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    bound = BF16 * np.abs(want) + 2.0 ** -20 * (np.abs(term) + np.abs(res)) + 1e-38
    assert not (np.abs(got - want) > bound).any()
    if s["pre"] is None:
        assert n is None
        return r, n
    with np.errstate(all="ignore"):
        nxt = rms(got, EPS) * f64(s["pre"])
    assert not (np.abs(f64(n) - nxt) > (BF16 + 2.0 ** -20) * np.abs(nxt) + 1e-38).any()
    return r, n


@pytest.mark.parametrize("width", [1, 2, 7, 8, 24, 100, 128, 129, 256, 264, 520, 999, 1032, 2048,
                                   2050, 4096, 4104, 8191, 8192, 16383, 16384])
@pytest.mark.parametrize("rows", [1, 5])
def test_widths(env, width, rows):
    check(env, make(env, rows, width, seed=width))


@pytest.mark.parametrize("gate", ["none", "channel", "element", "row"])
@pytest.mark.parametrize("kind", ["identity", "sigmoid", "silu"])
@pytest.mark.parametrize("width", [128, 75])
def test_gates(env, gate, kind, width):
    check(env, make(env, 33, width, gate=gate), kind, -1.25)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("resid", [False, True])
def test_parts(env, post, pre, resid):
    for width in (2048, 61):
        check(env, make(env, 9, width, post=post, pre=pre, resid=resid, gate="none"))


@pytest.mark.parametrize("inner,width,pad", [(1, 128, 8), (1, 128, 3), (32, 128, 64), (3, 40, 8),
                                             (4, 64, 5), (2, 2048, 16), (3, 7, 0)])
@pytest.mark.parametrize("gate", ["element", "row"])
def test_heads_and_strides(env, inner, width, pad, gate):
    check(env, make(env, 6 * inner, width, inner=inner, pad=pad, gate=gate), "silu")


def test_many_rows(env):
    check(env, make(env, 70001, 3))
    check(env, make(env, 4099, 128))


@pytest.mark.parametrize("width", [2048, 333])
def test_in_place(env, width):
    import torch
    a, b = make(env, 17, width, seed=4), make(env, 17, width, seed=4)
    want = check(env, a)
    got = check(env, dict(b, x=b["x"].clone(), resid=b["resid"].clone()))
    x, resid = b["x"].clone(), b["resid"].clone()
    moe, _ = env
    moe.norm_gate_residual(x, gamma_post=b["post"], gate=b["gate"], resid=resid, res_scale=0.5,
                           gamma_pre=b["pre"], eps=EPS, resid_out=resid, x_next=x)
    for w, g, p in zip(want, got, (resid, x)):
        assert torch.equal(w, g) and torch.equal(w, p)


@pytest.mark.parametrize("width", [128, 2048, 4096, 50])
def test_rows_do_not_see_one_another(env, width):
    """Zero rows, and rows with infinities and NaN, beside ordinary ones."""
    import torch
    s = make(env, 8, width, gate="none", resid=False)
    s["x"][1] = 0.0
    s["x"][3, 0] = float("nan")
    s["x"][5, width - 1] = float("inf")
    r, n = check(env, s)
    assert (r[1] == 0).all() and (n[1] == 0).all()
    keep = [0, 2, 4, 6, 7]
    clean = {k: (v[keep] if k == "x" else v) for k, v in s.items()}
    r2, n2 = check(env, clean)
    assert torch.equal(r[keep], r2) and torch.equal(n[keep], n2)


def test_tensors_are_checked(env):
    import torch
    moe, dev = env
    s = make(env, 6, 64)
    x, w = s["x"], s["post"]
    wide = torch.zeros(128, dtype=torch.bfloat16, device=dev)
    for kw in (dict(gamma_post=w.float()), dict(gamma_post=wide[::2]), dict(gamma_pre=wide),
               dict(gate=x[:5]), dict(gate=x.t().contiguous().t()), dict(resid=x.float()),
               dict(resid=x.cpu()), dict(x_next=torch.empty_like(x)), dict(resid_out=x[:, :32]),
               dict(gate=wide)):
        with pytest.raises(moe.MoEError):
            moe.norm_gate_residual(x, **kw)
    for y in (x.float(), x[0], x.t(), x[None, None]):
        with pytest.raises(moe.MoEError):
            moe.norm_gate_residual(y)


def test_no_rows_and_stream(env):
    import torch
    moe, dev = env
    x = torch.empty(0, 128, dtype=torch.bfloat16, device=dev)
    r, _ = moe.norm_gate_residual(x)
    assert r.shape == (0, 128)
    s = make(env, 64, 2048)
    want = check(env, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = check(env, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    out, nxt = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.norm_gate_residual(s["x"], gamma_post=s["post"], gate=s["gate"], resid=s["resid"],
                               res_scale=0.5, gamma_pre=s["pre"], eps=EPS, resid_out=out,
                               x_next=nxt)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(nxt, want[1])


def test_offsets_beyond_32_bits(env):
    """Rows 2^30 values apart: the third starts past 2^31 values."""
    import torch
    moe, dev = env
    buf = torch.empty((1 << 31) + 4096, dtype=torch.bfloat16, device=dev)
    x = torch.as_strided(buf, (3, 1000), (1 << 30, 1))
    s = make(env, 3, 1000, resid=False, gate="none")
    x.copy_(s["x"])
    want = check(env, s)
    got = check(env, dict(s, x=x), resid_out=x)
    assert torch.equal(want[1], got[1])


def test_results_on_a_given_stream(env):
    """Results made for a call on another stream are not the memory of work
    that is still to come on the current one."""
    import torch
    s = make(env, 3001, 2048)
    want = check(env, s)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    blocks = [torch.full_like(w, 5.0) for w in want]
    where = [b.data_ptr() for b in blocks]
    reads = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for r, b in zip(reads, blocks):
        r.copy_(b)
    del blocks, b
    moe, _ = env
    got = moe.norm_gate_residual(s["x"], gamma_post=s["post"], gate=s["gate"], resid=s["resid"],
                                 res_scale=0.5, gamma_pre=s["pre"], eps=EPS, stream=side)
    assert not {g.data_ptr() for g in got} & set(where)
    torch.cuda.synchronize()
    assert all((r == 5.0).all() for r in reads)
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_written_tensors_count_a_version(env):
    import torch
    moe, _ = env
    s = make(env, 9, 128)
    r, n = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    read = [s["x"], s["resid"], s["pre"]]
    before = [t._version for t in read + [r, n]]
    moe.norm_gate_residual(s["x"], resid=s["resid"], gamma_pre=s["pre"], resid_out=r, x_next=n)
    assert [t._version for t in read + [r, n]] == before[:3] + [before[3] + 1, before[4] + 1]
    with torch.inference_mode():
        again, _ = moe.norm_gate_residual(s["x"], resid=s["resid"], resid_out=torch.empty_like(r))
        assert torch.equal(again, r)
