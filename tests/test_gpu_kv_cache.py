"""The paged cache written and read back: codes and scales are exact."""
import numpy as np
import pytest

from attn_ref import codes, scales
from util import gpu_env

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return gpu_env()


def ints(env, v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device=env[1])


def held(x):
    return x.float().double().cpu().numpy()


def rows_of(env, n, heads, d, seed, kind="normal"):
    """bf16 rows: values of many sizes, ties of the rounding, borders."""
    import torch
    _, dev = env
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((n, heads, d), generator=g, device=dev)
    if kind == "wide":  # rows and values of very different sizes
        x = x * torch.exp2(torch.randint(-120, 120, (n, heads, 1), generator=g, device=dev).float())
        x = x * torch.exp2(torch.randint(-12, 1, (n, heads, d), generator=g, device=dev).float())
    if kind == "ties":  # quotients in the middle of two codes, for int8 and for e4m3
        x = torch.randint(-254, 255, (n, heads, d), generator=g, device=dev).float() / 2
        x[..., 0] = torch.where(torch.arange(n, device=dev) % 2 == 0, 127.0, -112.0)[:, None]
    if kind == "edge":
        x[0] = 0
        x[1] = 0
        x[1, :, 3] = 2.0 ** -133  # the least bf16
        x[2, :, 5] = float(torch.finfo(torch.bfloat16).max)
        x[3] *= 2.0 ** -130
        x[4, :, 7] = float("nan")
        x[5, :, 9] = float("-inf")
        x[6] = 448.0
        x[7] = -1.75 * 2.0 ** 20
        x[8, :, 1] = 1.7578125  # just above 1.75
    return x.bfloat16()


@pytest.mark.parametrize("kv", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["normal", "wide", "ties", "edge"])
def test_codes_and_scales(env, kv, d, kind):
    import torch
    moe, dev = env
    hkv, page = 3, 16
    new, length = [37, 1, 0, 20], [40, 1, 9, 64]
    n = sum(new)
    a = moe.PagedAttention(2 * hkv, hkv, d, page, kv, device=dev)
    c = a.new_cache(11)
    table = ints(env, [[7, 2, 9, -1], [0, -1, -1, -1], [1, -1, -1, -1], [4, 10, 3, 5]])
    lens, cu = ints(env, length), ints(env, [0, 37, 38, 38, 58])
    k, v = rows_of(env, n, hkv, d, 1, kind), rows_of(env, n, hkv, d, 2, kind)
    wide = torch.zeros((n, 2 * hkv * d + 8), dtype=torch.bfloat16, device=dev)  # strided rows
    wide[:, :hkv * d], wide[:, hkv * d + 8:] = k.flatten(1), v.flatten(1)
    a.write(c, wide[:, :hkv * d].unflatten(1, (hkv, d)), wide[:, hkv * d + 8:].unflatten(1, (hkv, d)),
            table, lens, cu)
    back = a.read(c, table, lens, cu, rows=n)
    assert a.status() == 0
    seq = np.repeat(np.arange(4), new)
    pos = np.concatenate([np.arange(l - m, l) for m, l in zip(new, length)])
    pg = table.cpu().numpy()[seq, pos // page]
    for x, store, scale, got in zip((k, v), c[:2], c[2:], back):
        x64 = x.double().cpu().numpy()
        if kv == "bf16":
            assert torch.equal(got.view(torch.int16), x.view(torch.int16))
            want = x64
        else:
            s = scales(x64, kv)
            assert np.array_equal(scale.cpu().numpy()[pg, :, pos % page], s, equal_nan=True)
            want = codes(x64, s, kv)
            value = torch.from_numpy(want * s.astype(np.float64)[..., None])
            # one rounding of the product (a double holds it exactly)
            assert np.array_equal(held(got), value.float().bfloat16().double().numpy(),
                                  equal_nan=True)
        assert np.array_equal(held(store)[pg, :, pos % page], want, equal_nan=True)
        touched = np.zeros((11, page), bool)
        touched[pg, pos % page] = True
        assert (held(store).transpose(0, 2, 1, 3)[~touched] == 0).all()
        if kv != "bf16":
            assert (scale.cpu().numpy().transpose(0, 2, 1)[~touched] == 0).all()


@pytest.mark.parametrize("kv", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("b", [1, 5, 700])
def test_tokens_of_uniform_and_large_batches(env, kv, b):
    """Decode writes (one row each), prompts of thousands of rows."""
    import torch
    moe, dev = env
    a = moe.PagedAttention(4, 2, 128, 32, kv, device=dev)
    for t in (1, 3, 4096 // b):
        per = -(-(t + 40) // 32)
        c = a.new_cache(b * per)
        g = torch.Generator(device=dev).manual_seed(b)
        table = torch.randperm(b * per, generator=g, device=dev).int().view(b, per)
        lens = (t + torch.randint(0, 41, (b,), generator=g, device=dev)).int()
        k, v = rows_of(env, b * t, 2, 128, 3), rows_of(env, b * t, 2, 128, 4)
        a.write(c, k, v, table, lens)
        kb, vb = a.read(c, table, lens, rows=b * t)
        for x, y in ((k, kb), (v, vb)):
            x64 = x.double().cpu().numpy()
            if kv != "bf16":
                s = scales(x64, kv)
                x64 = codes(x64, s, kv) * s.astype(np.float64)[..., None]
            assert np.array_equal(held(y), torch.from_numpy(x64).float().bfloat16().double().numpy())
        assert a.status() == 0


def test_skipped_and_bad_rows(env):
    import torch
    moe, dev = env
    for kv in ("bf16", "int8", "e4m3"):
        a = moe.PagedAttention(2, 1, 64, 16, kv, device=dev)
        k = rows_of(env, 8, 1, 64, 1)
        full, part = a.new_cache(4), a.new_cache(4)
        table = ints(env, [[0, 1], [2, 3]])
        a.write(full, k, k, table, ints(env, [20, 4]))
        same = lambda: all(torch.equal(x.view(torch.uint8), y.view(torch.uint8))
                           for x, y in zip(full, part) if x is not None)

        def write(table, lens, cu=None, bits=moe.DEV_BAD_INDEX):
            a.write(part, k, k, table, ints(env, lens), cu)
            assert a.status() == bits
            a.clear_status()

        zero = part.k.view(torch.uint8)
        write(table, [0, -5], bits=0)
        write(table, [3, 33])                      # fewer positions than rows; more than the table's
        write(table, [20, 4], ints(env, [0, 9, 9]))
        write(table, [20, 4], ints(env, [-1, -1, -1]))
        write(table, [20, 4], ints(env, [4, 3, 2]))
        assert (zero == 0).all()
        write(ints(env, [[0, 4], [2, 3]]), [20, 4])  # positions 16 .. 19 in a page that is not there
        assert not same()
        write(ints(env, [[-1, 1], [-9, 3]]), [20, 0], bits=0)
        assert same()
        out = torch.full((8, 1, 64), 7.0, device=dev).bfloat16()
        a.read(full, ints(env, [[0, 9], [2, -1]]), ints(env, [20, 4]), k=out, v=torch.zeros_like(out))
        assert a.status() == moe.DEV_BAD_INDEX
        assert (out[:4] == 7.0).all() and not (out[4:] == 7.0).any()


def test_capture_and_streams(env):
    """Decode steps in a graph: each replay writes at the lengths' places."""
    import torch
    moe, dev = env
    a = moe.PagedAttention(2, 2, 128, 16, "int8", device=dev)
    c = a.new_cache(8)
    table, lens = ints(env, [[1, 5], [3, 0]]), ints(env, [1, 9])
    k, v = (torch.zeros((2, 2, 128), dtype=torch.bfloat16, device=dev) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.write(c, k, v, table, lens)
        lens.add_(1)
    for x in c:
        x.zero_()
    lens.copy_(ints(env, [1, 9]))
    rows = [rows_of(env, 2, 2, 128, 50 + i) for i in range(12)]
    for x in rows:
        k.copy_(x), v.copy_(-x)
        graph.replay()
    want = a.new_cache(8)
    order = torch.stack([x[0] for x in rows] + [x[1] for x in rows])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    version = want.k._version
    a.write(want, order, -order, table, ints(env, [12, 20]), stream=side)
    assert want.k._version > version
    side.synchronize()
    for x, y in zip(c, want):
        assert torch.equal(x, y)
    assert a.status() == 0
