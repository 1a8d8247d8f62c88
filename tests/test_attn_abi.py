"""Host-side checks of paged attention, its cache and the verification of
drafts: bad calls are refused before any device work (no GPU)."""
import ctypes

import pytest

FAKE = 1 << 32  # aligned addresses far apart, never dereferenced on these paths


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__ as g
    g.build()
    import sparse_moe_decode_gb300 as m
    return m


def dims(moe, **kw):
    base = dict(q_heads=8, kv_heads=2, head_dim=128, page_size=64, kv_type=1, window=0, scale=0.1)
    return moe.AttnDims(**{**base, **kw})


def cache(moe, **kw):
    base = dict(k=FAKE, v=2 * FAKE, k_scale=3 * FAKE, v_scale=4 * FAKE, pages=100)
    return moe.KVCacheArgs(**{**base, **kw})


def batch(moe, **kw):
    base = dict(N=8, B=2, cu_seqlens=5 * FAKE, seq_lens=6 * FAKE, page_table=7 * FAKE, table_ld=10,
                table_cols=10)
    return moe.KVBatch(**{**base, **kw})


def call(moe, name, d=None, c=None, b=None, x=8 * FAKE, x_ld=None, y=9 * FAKE, y_ld=None,
         ws=10 * FAKE, ws_bytes=1 << 30):
    d, c, b = d or dims(moe), c or cache(moe), b or batch(moe)
    w = (d.q_heads if name == "moe_paged_attention" else d.kv_heads) * d.head_dim
    return getattr(moe.lib(), name)(ctypes.byref(d), ctypes.byref(c), ctypes.byref(b), x,
                                    w if x_ld is None else x_ld, y, w if y_ld is None else y_ld,
                                    ws, ws_bytes, None)


NAMES = ("moe_kv_write", "moe_kv_read", "moe_paged_attention")


@pytest.mark.parametrize("name", NAMES)
def test_refusals(moe, name):
    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    for kw in (dict(q_heads=7), dict(kv_heads=0), dict(q_heads=0), dict(q_heads=130, kv_heads=2),
               dict(q_heads=1026, kv_heads=513), dict(head_dim=96), dict(head_dim=512),
               dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(kv_type=3),
               dict(kv_type=-1)):
        assert call(moe, name, d=dims(moe, **kw)) == un, kw
        assert moe.moe_attn_workspace_bytes(dims(moe, **kw)) == 0
    for kw in (dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(moe, name, d=dims(moe, **kw)) == bad, kw
    for kw in (dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(pages=0),
               dict(k=FAKE + 8), dict(v_scale=4 * FAKE + 4), dict(v=FAKE + 1024),
               dict(k_scale=FAKE), dict(v_scale=3 * FAKE + 16)):
        assert call(moe, name, c=cache(moe, **kw)) == bad, kw
    # a bf16 cache has no scales
    assert call(moe, name, d=dims(moe, kv_type=0)) == bad
    assert call(moe, name, c=cache(moe, pages=1 << 24)) == un
    for kw in (dict(N=-1), dict(B=-1), dict(B=0), dict(seq_lens=None), dict(page_table=None),
               dict(cu_seqlens=5 * FAKE + 2), dict(seq_lens=6 * FAKE + 1), dict(table_cols=-1),
               dict(table_ld=9), dict(cu_seqlens=None, N=9), dict(page_table=7 * FAKE + 2),
               dict(table_ld=1 << 40)):
        assert call(moe, name, b=batch(moe, **kw)) == bad, kw
    for kw in (dict(N=(1 << 20) + 1), dict(B=65537),
               dict(table_cols=1 << 25, table_ld=1 << 25)):
        assert call(moe, name, b=batch(moe, **kw)) == un, kw
    row = 256 if name != "moe_paged_attention" else 1024
    for kw in (dict(x=8 * FAKE + 8), dict(y=9 * FAKE + 2), dict(x_ld=row - 8), dict(y_ld=row + 4),
               dict(x_ld=-row), dict(y_ld=1 << 40), dict(ws=None), dict(ws=10 * FAKE + 16)):
        assert call(moe, name, **kw) == bad, kw
    assert call(moe, name, ws_bytes=128) == moe.MOE_ERR_WORKSPACE
    L = moe.lib()
    assert getattr(L, name)(None, None, None, None, 0, None, 0, None, 0, None) == bad


def test_overlaps(moe):
    bad = moe.MOE_ERR_INVALID_ARG
    assert call(moe, "moe_kv_write", x=FAKE) == bad            # k inside the cache
    assert call(moe, "moe_kv_write", y=4 * FAKE) == bad        # v inside the scales
    assert call(moe, "moe_kv_write", x=None) == bad
    assert call(moe, "moe_kv_read", x=2 * FAKE + 1024) == bad
    assert call(moe, "moe_kv_read", y=8 * FAKE + 256) == bad   # both outputs
    assert call(moe, "moe_paged_attention", y=8 * FAKE) == bad
    assert call(moe, "moe_paged_attention", y=FAKE) == bad
    assert call(moe, "moe_paged_attention", x=None) == bad
    assert call(moe, "moe_paged_attention", y=None) == bad


def test_empty_calls(moe):
    for name in NAMES:
        assert call(moe, name, b=batch(moe, N=0)) == moe.MOE_OK
        assert call(moe, name, b=batch(moe, N=0, B=0, cu_seqlens=None, seq_lens=None,
                                       page_table=None)) == moe.MOE_OK
    assert call(moe, "moe_kv_read", x=None, y=None) == moe.MOE_OK


def test_workspace_does_not_depend_on_the_batch(moe):
    assert moe.moe_attn_workspace_bytes(dims(moe)) > 256
    n = moe.moe_attn_workspace_bytes(dims(moe, head_dim=256))
    assert n < 128 << 20
    assert call(moe, "moe_paged_attention", ws_bytes=moe.moe_attn_workspace_bytes(dims(moe)) - 1) \
        == moe.MOE_ERR_WORKSPACE


def draft(moe, B=2, T=3, V=100, p=FAKE, p_seq=400, p_ld=100, q=2 * FAKE, q_seq=300, q_ld=100,
          d=3 * FAKE, u=4 * FAKE, tokens=5 * FAKE, accepted=6 * FAKE, ws=7 * FAKE, ws_bytes=256):
    return moe.lib().moe_verify_draft(B, T, V, p, p_seq, p_ld, q, q_seq, q_ld, d, u, tokens,
                                      accepted, ws, ws_bytes, None)


def test_draft_refusals(moe):
    bad, un = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    for kw in (dict(B=-1), dict(T=-1), dict(V=0), dict(p=None), dict(p=FAKE + 2), dict(q=2 * FAKE + 1),
               dict(d=None), dict(u=None), dict(tokens=None), dict(accepted=None),
               dict(tokens=5 * FAKE + 2), dict(p_seq=-1), dict(p_ld=-4), dict(q_ld=1 << 41),
               dict(tokens=FAKE + 4), dict(accepted=5 * FAKE), dict(accepted=4 * FAKE + 8),
               dict(tokens=2 * FAKE), dict(ws=None), dict(ws=7 * FAKE + 16)):
        assert draft(moe, **kw) == bad, kw
    for kw in (dict(B=65537), dict(T=1025), dict(V=(1 << 24) + 1)):
        assert draft(moe, **kw) == un, kw
    assert draft(moe, ws_bytes=255) == moe.MOE_ERR_WORKSPACE
    assert draft(moe, B=0) == moe.MOE_OK


def test_python_entries_check_their_tensors(moe):
    torch = pytest.importorskip("torch")
    with pytest.raises(moe.MoEError):
        moe.PagedAttention(8, 2, 128, kv_type="int4", device="cpu")
    with pytest.raises(moe.MoEError):
        moe.PagedAttention(8, 3, 128, device="cpu")
    a = moe.PagedAttention(8, 2, 128, kv_type="int8", device="cpu")
    c = a.new_cache(4)
    assert c.k.shape == (4, 2, 64, 128) and c.k.dtype == torch.int8
    assert c.k_scale.shape == (4, 2, 64)
    assert a.dims.scale == pytest.approx(128 ** -0.5)
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    kv = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    for f in (lambda: a.attend(c, q, table, lens), lambda: a.write(c, kv, kv, table, lens),
              lambda: a.read(c, table, lens), lambda: a.read(c, table, lens, rows=2)):
        with pytest.raises(moe.MoEError):  # host memory
            f()
    v = moe.DraftVerifier(device="cpu")
    with pytest.raises(moe.MoEError):
        v.verify(torch.ones(1, 1, 4), torch.zeros(1, 0, dtype=torch.int32), torch.zeros(1, 1))
