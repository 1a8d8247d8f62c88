"""Host-side checks of the gated delta rule and of the norms around a block:
bad calls are refused before any device work (no GPU)."""
import ctypes

import pytest

FAKE = 1 << 20  # aligned addresses far apart, never dereferenced on these paths


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__ as g
    g.build()
    import sparse_moe_decode_gb300 as m
    return m


def delta_dims(moe, **kw):
    base = dict(qk_heads=2, v_heads=4, qk_dim=128, v_dim=128, qk_norm=1, qk_eps=1e-6, scale=0.1)
    return moe.DeltaDims(**{**base, **kw})


def delta_inputs(moe, **kw):
    base = dict(q=FAKE, k=2 * FAKE, v=3 * FAKE, g=4 * FAKE, beta=5 * FAKE, q_ld=256, k_ld=256,
                v_ld=512, g_ld=4, beta_ld=4)
    return moe.DeltaInputs(**{**base, **kw})


def chunk(moe, d=None, i=None, N=8, cu=8 * FAKE, B=2, slots=9 * FAKE, n_slots=4,
          s_in=64 * FAKE, s_out=128 * FAKE, out=6 * FAKE, out_ld=512, ws=7 * FAKE, ws_bytes=1 << 30):
    d, i = d or delta_dims(moe), i or delta_inputs(moe)
    return moe.lib().moe_delta_chunk(ctypes.byref(d), ctypes.byref(i), N, cu, B, slots, n_slots,
                                     s_in, s_out, out, out_ld, ws, ws_bytes, None)


def step(moe, d=None, i=None, B=2, T=4, slots=9 * FAKE, n_slots=4, s_in=64 * FAKE,
         s_out=128 * FAKE, out=6 * FAKE, out_ld=512, ws=7 * FAKE, ws_bytes=256):
    d, i = d or delta_dims(moe), i or delta_inputs(moe)
    return moe.lib().moe_delta_step(ctypes.byref(d), ctypes.byref(i), B, T, slots, n_slots, s_in,
                                    s_out, out, out_ld, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [chunk, step])
def test_delta_refuses_bad_dims_and_arguments(moe, call):
    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    for kw in (dict(qk_dim=96), dict(v_dim=256), dict(v_heads=3), dict(qk_heads=0),
               dict(v_heads=0), dict(v_heads=512)):
        assert call(moe, d=delta_dims(moe, **kw)) == un, kw
        assert moe.moe_delta_workspace_bytes(delta_dims(moe, **kw), 8, 2) == 0
    for kw in (dict(scale=float("nan")), dict(scale=float("inf")), dict(qk_eps=-1.0),
               dict(qk_eps=float("nan"))):
        assert call(moe, d=delta_dims(moe, **kw)) == bad, kw
    for kw in (dict(q=None), dict(v=3 * FAKE + 8), dict(g=4 * FAKE + 2), dict(q_ld=248),
               dict(v_ld=516), dict(k_ld=-256), dict(g_ld=3), dict(beta=None),
               dict(q_ld=1 << 40)):
        assert call(moe, i=delta_inputs(moe, **kw)) == bad, kw
    for kw in (dict(out=None), dict(out=6 * FAKE + 2), dict(out_ld=504), dict(n_slots=-1),
               dict(slots=9 * FAKE + 2), dict(s_in=64 * FAKE + 4), dict(ws=None),
               dict(ws=7 * FAKE + 16), dict(B=-1), dict(s_out=64 * FAKE + 256),
               dict(out=3 * FAKE), dict(out=3 * FAKE + 1024), dict(slots=None, n_slots=1)):
        assert call(moe, **kw) == bad, kw
    assert call(moe, ws_bytes=128) == moe.MOE_ERR_WORKSPACE
    assert call(moe, B=65537) == un
    L = moe.lib()
    assert L.moe_delta_chunk(None, None, 0, None, 1, None, 0, None, None, None, 0, None, 0,
                             None) == bad


def test_delta_sizes(moe):
    assert chunk(moe, N=-1) == moe.MOE_ERR_INVALID_ARG
    assert chunk(moe, N=(1 << 20) + 1) == moe.MOE_ERR_UNSUPPORTED
    assert chunk(moe, cu=None, B=2) == moe.MOE_ERR_INVALID_ARG  # rows of whom?
    assert step(moe, T=-1) == moe.MOE_ERR_INVALID_ARG
    assert step(moe, B=1 << 10, T=(1 << 10) + 1, n_slots=1 << 10) == moe.MOE_ERR_UNSUPPORTED
    assert chunk(moe, B=0) == moe.MOE_OK and step(moe, B=0) == moe.MOE_OK
    d = delta_dims(moe)
    small, big = (moe.moe_delta_workspace_bytes(d, n, 3) for n in (1, 4096))
    assert 256 <= small <= big
    assert moe.moe_delta_workspace_bytes(d, (1 << 20) + 1, 1) == 0
    assert moe.moe_delta_workspace_bytes(d, 1, 65537) == 0
    assert moe.moe_delta_workspace_bytes(d, -1, 1) == 0


def test_delta_workspace_grows_with_rows_and_sequences(moe):
    """More of either never needs less, so that the largest call's workspace
    serves all; short sequences take none of it each."""
    d = delta_dims(moe)
    size = lambda n, b: moe.moe_delta_workspace_bytes(d, n, b)
    for n in (0, 1, 24, 25, 63, 64, 100, 1000, 4096):
        for b in (1, 2, 3, 40, 41, 300):
            assert size(n, b) <= size(n + 1, b) and size(n, b) <= size(n, b + 1)
    # records of 16 bytes a sequence, and a chunk slot per 25 rows
    slot = size(64, 1) - size(0, 1)
    assert size(256, 256) <= size(0, 1) + 256 * 16 + 256 // 25 * slot


def norm(moe, **kw):
    base = dict(rows=4, width=128, inner=1, x=FAKE, gamma_post=2 * FAKE, gate=3 * FAKE,
                resid_in=4 * FAKE, gamma_pre=5 * FAKE, resid_out=6 * FAKE, x_next=7 * FAKE,
                x_ld=128, gate_ld=128, resid_in_ld=128, resid_out_ld=128, x_next_ld=128,
                gate_kind=moe.GATE_ELEMENT, gate_act=1, res_scale=1.0, eps=1e-6)
    a = moe.NormArgs(**{**base, **kw})
    return moe.lib().moe_norm_gate_residual(ctypes.byref(a), None)


def test_norm_refuses_bad_arguments(moe):
    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    row = 256  # bytes
    for kw in (dict(rows=-1), dict(width=0), dict(inner=0), dict(inner=3), dict(eps=-1.0),
               dict(eps=float("nan")), dict(res_scale=float("inf")), dict(gate_kind=4),
               dict(gate_act=3), dict(gate_kind=-1), dict(x=None), dict(x=FAKE + 2),
               dict(gate=None), dict(gate_kind=0), dict(gamma_pre=None), dict(x_next=None),
               dict(resid_out=None, x_next=None, gamma_pre=None), dict(x_ld=127),
               dict(gate_ld=100), dict(resid_out_ld=0), dict(gate_kind=3, gate_ld=0),
               dict(x_next=6 * FAKE), dict(x_next=6 * FAKE + row), dict(resid_out=4 * FAKE + row),
               dict(x_next=5 * FAKE), dict(resid_out=3 * FAKE),
               dict(resid_out=FAKE, resid_out_ld=136), dict(x_ld=1 << 40)):
        assert norm(moe, **kw) == bad, kw
    assert norm(moe, width=16392, x_ld=16392, gate_ld=16392, resid_in_ld=16392,
                resid_out_ld=16392, x_next_ld=16392) == un
    assert norm(moe, rows=1 << 31) == un
    assert norm(moe, rows=0) == moe.MOE_OK
    assert moe.lib().moe_norm_gate_residual(None, None) == bad


def test_python_entries_check_their_tensors(moe):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 128, dtype=torch.bfloat16)  # host memory
    with pytest.raises(moe.MoEError):
        moe.norm_gate_residual(x)
    with pytest.raises(moe.MoEError):
        moe.norm_gate_residual(x, gate_act="relu")
    with pytest.raises(moe.MoEError):
        moe.GatedDelta(2, 3, 128, 128, max_tokens=8, device="cpu")
    m = moe.GatedDelta(2, 4, 128, 128, max_tokens=8, device="cpu")
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    v = torch.zeros(4, 4, 128, dtype=torch.bfloat16)
    g = torch.zeros(4, 4)
    with pytest.raises(moe.MoEError):
        m.chunk(q, q, v, g, g)
    with pytest.raises(moe.MoEError):
        m.step(q[0], q, v, g, g)


def test_calls_run_on_their_tensors_device(moe, monkeypatch):
    """With another device current than the tensors', every call makes theirs
    current for its time (their stream and the kernels are of the current one)."""
    import contextlib
    import types
    torch = pytest.importorskip("torch")
    now = [0]

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], index
        try:
            yield
        finally:
            now[0] = before

    m = moe.GatedDelta(2, 4, 128, 128, max_tokens=8, device="cpu")
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda *a: types.SimpleNamespace(cuda_stream=100 + now[0]))
    where, status = [], [0]

    def call(*args):  # as the extension: nothing is done on another device
        where.append(now[0])
        return -1 if now[0] != index else status[0] or "result"

    m._chunk = m._step = call
    fake = types.SimpleNamespace(moe_read_status=lambda *a: where.append(a[1]) or 0,
                                 moe_clear_status=lambda *a: where.append(a[1]) or 0,
                                 moe_status_string=moe.lib().moe_status_string)
    monkeypatch.setattr(moe, "lib", lambda: fake)
    monkeypatch.setattr(moe, "_binding", types.SimpleNamespace(norm=call))
    for index, tries in ((0, [0]), (1, [0, 1])):
        m._index = index
        x = types.SimpleNamespace(get_device=lambda: index)
        calls = (lambda: m.chunk(*[None] * 5), lambda: m.step(*[None] * 5),
                 lambda: moe.norm_gate_residual(x))
        del where[:]
        assert [f() for f in calls] == ["result"] * 3 and where == tries * 3
        del where[:]
        m.status()
        m.clear_status()
        assert where == [100 + index] * 2 and now == [0]
        status[0] = moe.MOE_ERR_WORKSPACE  # refusals come through
        for f in calls:
            with pytest.raises(moe.MoEError) as e:
                f()
            assert e.value.status == moe.MOE_ERR_WORKSPACE and now == [0]
        status[0] = 0
