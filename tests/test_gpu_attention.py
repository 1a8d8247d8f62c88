"""Paged attention over its cache (PagedAttention.attend) against the fp64
definition; the bounds stand in attn_ref."""
import numpy as np
import pytest

from attn_ref import attention
from util import gpu_env

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return gpu_env()


def ints(env, v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device=env[1])


class Batch:
    """Sequences of `new` rows behind contexts (`length` positions with them),
    written through the cache's own call; pages in a random order among others
    that hold NaN."""

    def __init__(self, env, new, length, heads=(8, 2), d=128, page=64, kv="bf16", window=0, seed=0,
                 scale=None, uniform=False, k_std=1.0, v_std=1.0, guard=2):
        import torch
        moe, dev = env
        self.env, self.new, self.length, self.heads, self.d = env, new, length, heads, d
        self.kv, self.window, self.page = kv, window, page
        g = torch.Generator(device=dev).manual_seed(seed * 7919 + sum(length))
        hq, hkv = heads
        n, total = sum(new), sum(length)
        self.attn = moe.PagedAttention(hq, hkv, d, page, kv, window, scale, device=dev)
        per = [-(-x // page) for x in length]
        pages = sum(per) + 3
        self.cache = self.attn.new_cache(pages)
        self.poison(range(pages))
        order = torch.randperm(pages, generator=g, device=dev).tolist()
        table, at = [], 0
        for p in per:
            table.append(order[at:at + p] + [-1] * (max(per) - p))
            at += p
        self.table, self.lens = ints(env, table), ints(env, length)
        self.cu = None if uniform else ints(env, np.concatenate([[0], np.cumsum(new)]).tolist())

        def rows(count, width, std):  # slices of a wider row, NaN rows around them
            x = torch.full((count + 2 * guard, width + 16), float("nan"), device=dev).bfloat16()
            x[guard:guard + count, 8:8 + width] = torch.randn(
                (count, width), generator=g, device=dev) * std
            return x[guard:guard + count, 8:8 + width]

        self.q = rows(n, hq * d, 2.0).unflatten(1, (hq, d))
        self.k = rows(total, hkv * d, k_std).unflatten(1, (hkv, d))
        self.v = rows(total, hkv * d, v_std).unflatten(1, (hkv, d))

    def poison(self, pages):
        import torch
        pages = list(pages)
        for x in self.cache[:2]:
            if self.kv == "bf16":
                x[pages] = float("nan")
            elif self.kv == "int8":
                x[pages] = -128
            else:
                x.view(torch.uint8)[pages] = 0x7F  # NaN
        for x in self.cache[2:]:
            if x is not None:
                x[pages] = float("nan")

    def fill(self):
        whole = ints(self.env, np.concatenate([[0], np.cumsum(self.length)]).tolist())
        self.attn.write(self.cache, self.k, self.v, self.table, self.lens, whole)
        return self

    def attend(self, **kw):
        return self.attn.attend(self.cache, self.q, self.table, self.lens, self.cu, **kw)

    def values(self):
        """What the cache stands for, per sequence (k, v), and the scales."""
        out = []
        for i, length in enumerate(self.length):
            pos = np.arange(length)
            pg = self.table[i].cpu().numpy()[pos // self.page] if length else pos
            both, both_scales = [], []
            for x, s in zip(self.cache[:2], self.cache[2:]):
                y = x.float().double().cpu().numpy()[pg, :, pos % self.page]
                if s is not None:
                    scale = s.double().cpu().numpy()[pg, :, pos % self.page]
                    y = y * scale[..., None]
                    both_scales.append(scale)
                both.append(y)
            out.append((*both, *both_scales))
        return out

    def check(self, out, skip=()):
        got = out.double().cpu().numpy()
        q = self.q.double().cpu().numpy()
        start = 0
        worst = 0.0
        for i, (n, (k, v, *scales)) in enumerate(zip(self.new, self.values())):
            if n and i not in skip:
                want, bound = attention(q[start:start + n], k, v, self.length[i],
                                        self.attn.dims.scale, self.window, *scales)
                err = np.abs(got[start:start + n] - want)
                ok = bool((err <= bound).all())  # (NaN is not)
                assert ok, (i, np.nanmax(err / bound), np.argwhere(~(err <= bound))[:4])
                worst = max(worst, (err / bound).max())
            start += n
        return worst


KV = ["bf16", "int8", "e4m3"]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,t,page", [((8, 2), 1, 64), ((4, 4), 3, 16), ((16, 2), 4, 32),
                                          ((6, 2), 5, 128), ((64, 1), 1, 256)])
def test_decode_and_drafts(env, kv, d, heads, t, page):
    """As many rows each; contexts of one token, around pages' and tiles' ends."""
    length = [t, t + 1, 63 + t, 64, 65, 127, 130, 300]
    length = [max(x, t) for x in length]
    b = Batch(env, [t] * len(length), length, heads, d, page, kv, uniform=True).fill()
    b.check(b.attend())
    assert b.attn.status() == 0


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_ragged_mix(env, kv, d, window):
    """Prompts, chunks behind a context, single tokens, a sequence without rows."""
    new = [130, 1, 0, 257, 1, 1, 33, 2, 64]
    length = [130, 1, 50, 400, 700, 129, 90, 256, 64]
    b = Batch(env, new, length, (6, 2), d, 16, kv, window).fill()
    b.check(b.attend())
    assert b.attn.status() == 0


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("heads,d", [((4, 1), 128), ((3, 3), 64), ((8, 1), 256), ((5, 1), 128)])
def test_prompts(env, kv, heads, d):
    """Whole prompts of sizes around the tiles', in one call and alone."""
    for new, length in (([1025], [1025]), ([700, 129, 128, 127], [700, 129, 128, 127]),
                        ([300, 500], [1300, 777])):
        b = Batch(env, new, length, heads, d, 64, kv).fill()
        b.check(b.attend())
    assert b.attn.status() == 0


@pytest.mark.parametrize("kv", KV)
def test_long_contexts_are_shared_out(env, kv):
    """One and two sequences over thousands of positions: many blocks a tile."""
    for new, length, heads, d in (([1], [20001], (8, 1), 128), ([3], [9000], (4, 2), 256),
                                  ([1, 1], [5000, 12345], (8, 4), 64), ([70], [7001], (2, 1), 128)):
        b = Batch(env, new, length, heads, d, 64, kv).fill()
        b.check(b.attend())


@pytest.mark.parametrize("kv", KV)
def test_many_sequences(env, kv):
    rng = np.random.default_rng(3)
    length = rng.integers(1, 90, 1100).tolist()
    b = Batch(env, [1] * len(length), length, (4, 2), 64, 16, kv, uniform=True).fill()
    b.check(b.attend())
    new = [min(int(x), int(y)) for x, y in zip(rng.integers(0, 4, 1100), length)]
    b = Batch(env, new, length, (4, 2), 64, 16, kv).fill()
    b.check(b.attend())


@pytest.mark.parametrize("kv", KV)
def test_one_key_has_nearly_all_the_weight(env, kv):
    """Sharp softmax: scores of up to some hundreds, maxima that come late."""
    b = Batch(env, [40, 1, 4], [300, 900, 500], (8, 2), 128, 32, kv, k_std=12.0).fill()
    b.check(b.attend())


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("new", [[1, 4], [150, 200]])
def test_scales_far_apart(env, kv, new):
    """Rows of v from 1e-30 to 1e30 and of zeros: each output keeps the digits of
    its own largest term."""
    import torch
    moe, dev = env
    b = Batch(env, new, [400, 330], (4, 2), 128, 64, kv, k_std=20.0)
    g = torch.Generator(device=dev).manual_seed(5)
    power = torch.randint(-100, 101, (b.v.shape[0], 2, 1), generator=g, device=dev)
    power[::7] = -200  # of no weight beside any other
    b.v.copy_((b.v.double() * torch.exp2(power.double())).bfloat16())
    b.v[3::11] = 0
    b.fill()
    b.check(b.attend())


@pytest.mark.parametrize("kv", KV)
def test_large_and_tiny_queries(env, kv):
    b = Batch(env, [5, 200], [70, 300], (4, 2), 128, 64, kv, scale=1.0).fill()
    b.q[::2] *= 1e-20
    b.q[1::2] *= 0.02
    b.q[7] = 0
    b.check(b.attend())
    # the same rows under factors of a power of two that the scale takes back
    b = Batch(env, [1, 130], [70, 300], (4, 2), 128, 64, kv, scale=2.0 ** -60, k_std=0.1).fill()
    b.q *= 2.0 ** 60
    b.check(b.attend())


def test_negative_scale(env):
    for kv in KV:
        b = Batch(env, [1, 150], [70, 300], (4, 2), 128, 64, kv, scale=-0.07).fill()
        b.check(b.attend())


@pytest.mark.parametrize("new", [1, 60])
def test_windows_longer_than_any_sequence(env, new):
    import torch
    b = Batch(env, [new] * 2, [700, 400], (8, 2), 64, 16, "bf16", uniform=True).fill()
    want = b.attend()
    for window in (700, 1 << 30, 2 ** 31 - 1):
        b.attn = env[0].PagedAttention(8, 2, 64, 16, "bf16", window, device=env[1])
        assert torch.equal(b.attend(), want)
    b.check(want)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("new", [[1, 1, 1], [3, 140, 1], [200, 300, 150]])
def test_values_that_are_not_finite_stay_in_their_sequence(env, kv, new):
    import torch
    length = [max(x, y) for x, y in zip(new, [200, 300, 150])]
    b = Batch(env, new, length, (4, 2), 128, 64, kv)
    b.k[length[0] + 10, 0, 5] = float("nan")  # sequence 1, a key that all its last rows see
    b.v[length[0] + 20, 1, 7] = float("inf")
    b.fill()
    out = b.attend()
    b.check(out, skip=(1,))
    last = out[new[0] + new[1] - 1].float()
    assert torch.isnan(last[:2]).all()       # the heads that read the key
    assert not torch.isfinite(last[2:]).all()
    if kv != "bf16":
        # an 8-bit row that is not finite reaches only those that see it
        seen = length[1] - new[1]  # the first row's position
        for i in range(new[1]):
            row = out[new[0] + i].float()
            assert torch.isfinite(row[:2]).all() == (seen + i < 10)
            assert torch.isfinite(row[2:]).all() == (seen + i < 20)


def test_nan_queries_stay_in_their_row(env):
    import torch
    for kv in KV:
        for new in ([1, 4], [100, 150]):
            b = Batch(env, new, [300, 200], (4, 2), 128, 64, kv).fill()
            b.q[1, 1, 3] = float("nan")
            out = b.attend()
            assert torch.isnan(out[1, 1]).all()
            out[1, 1] = 0
            assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [2, 130, 5, 300]])
def test_skipped_and_bad_sequences(env, new):
    """Skipped rows are left as they were; what is out of range is not followed."""
    import torch
    moe, dev = env
    length = [100, 200, 150, 300]
    good = Batch(env, new, length, (4, 2), 64, 16, "int8").fill()
    full = good.attend()
    edges = np.concatenate([[0], np.cumsum(new)])

    def run(lens=None, cu=None, table=None, skip=(), bits=0):
        out = torch.full((sum(new) + 4, 4, 64 + 8), 7.0, device=dev).bfloat16()[2:-2, :, :64]
        whole = torch.full((sum(new) + 4, 4 * 64), 7.0, device=dev).bfloat16()
        out = whole[2:-2].unflatten(1, (4, 64))
        good.attn.attend(good.cache, good.q, good.table if table is None else table,
                         ints(env, lens or length),
                         ints(env, (edges if cu is None else np.array(cu)).tolist()), out=out)
        assert good.attn.status() == bits
        good.attn.clear_status()
        for i in range(4):
            rows = slice(edges[i], edges[i + 1])
            if i in skip:
                assert (out[rows] == 7.0).all(), i
            elif cu is None:
                got, want = out[rows].float(), full[rows].float()
                assert (got - want).abs().max() <= 2.0 ** -6 * want.abs().max(), i
        assert (whole[:2] == 7.0).all() and (whole[-2:] == 7.0).all()

    run()
    run(lens=[0, 200, -3, 300], skip=(0, 2))                       # a padded batch
    run(lens=[0, 0, 0, 0], skip=(0, 1, 2, 3))
    run(lens=[100, 1 << 30, 150, 300], skip=(1,), bits=moe.DEV_BAD_INDEX)
    if new[1] > 1:
        run(lens=[100, new[1] - 1, 150, 300], skip=(1,), bits=moe.DEV_BAD_INDEX)
    n = int(edges[-1])
    run(cu=[0, n + 1, n + 1, n + 1, n + 1], skip=(0, 1, 2, 3), bits=moe.DEV_BAD_INDEX)
    run(cu=[5, 3, 3, 3, 3], skip=(0, 1, 2, 3), bits=moe.DEV_BAD_INDEX)
    run(cu=[-1, -1, -1, -1, -1], skip=(0, 1, 2, 3), bits=moe.DEV_BAD_INDEX)
    for page in (-1, good.cache.k.shape[0], 1 << 30):  # of sequence 2: the others are whole
        table = good.table.clone()
        table[2, 3] = page
        out = good.attn.attend(good.cache, good.q, table, good.lens, good.cu)
        assert good.attn.status() == moe.DEV_BAD_INDEX
        good.attn.clear_status()
        keep = [r for i in (0, 1, 3) for r in range(edges[i], edges[i + 1])]
        assert torch.equal(out[keep], full[keep])


def test_rows_of_no_sequence_are_left(env):
    import torch
    moe, dev = env
    b = Batch(env, [3, 200], [10, 260], (4, 2), 64, 16, "bf16").fill()
    out = torch.full((210, 4, 64), 7.0, device=dev).bfloat16()
    q = torch.cat([b.q, torch.full((7, 4, 64), float("nan"), device=dev).bfloat16()])
    b.attn.attend(b.cache, q, b.table, b.lens, b.cu, out=out)
    assert (out[203:] == 7.0).all()
    b.check(out[:203])


@pytest.mark.parametrize("kv", KV)
def test_repeats_and_batches_agree(env, kv):
    """A call repeated gives the same bits; graph replays follow the lengths."""
    import torch
    b = Batch(env, [1] * 5, [40, 500, 1, 700, 64], (8, 2), 128, 64, kv, uniform=True).fill()
    first = b.attend()
    for _ in range(5):
        assert torch.equal(b.attend(), first)
    p = Batch(env, [300, 3, 90], [700, 44, 90], (8, 2), 128, 64, kv).fill()
    first = p.attend()
    for _ in range(5):
        assert torch.equal(p.attend(), first)
    lens, out = b.lens.clone(), torch.zeros_like(b.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.attn.attend(b.cache, b.q, b.table, lens, out=out)
    for cut in ([40, 500, 1, 700, 64], [1, 3, 1, 650, 0], [39, 64, 1, 65, 63]):
        lens.copy_(ints(env, cut))
        out.fill_(3.0)
        graph.replay()
        want = b.attn.attend(b.cache, b.q, b.table, lens, out=torch.full_like(b.q, 3.0))
        assert torch.equal(out, want)


def test_streams_and_outputs(env):
    """Another stream than the current one, given outputs, column strides."""
    import torch
    moe, dev = env
    b = Batch(env, [4, 150], [300, 200], (4, 2), 128, 32, "e4m3").fill()
    want = b.attend()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = b.attend(stream=side)
    wide = torch.zeros((154, 4 * 128 + 64), dtype=torch.bfloat16, device=dev)
    part = wide[:, 64:].unflatten(1, (4, 128))
    before = part._version
    with torch.cuda.stream(side):
        r = b.attend(out=part)
    side.synchronize()
    assert r.data_ptr() == part.data_ptr() and part._version > before
    assert torch.equal(got, want) and torch.equal(part, want) and (wide[:, :64] == 0).all()


def test_tensors_are_checked(env):
    import torch
    moe, dev = env
    b = Batch(env, [2, 3], [30, 20], (4, 2), 64, 16, "int8").fill()
    a, c = b.attn, b.cache
    refuse = lambda f: pytest.raises(moe.MoEError, f)
    ok = (c, b.q, b.table, b.lens, b.cu)

    def call(cache=c, q=b.q, table=b.table, lens=b.lens, cu=b.cu, **kw):
        return lambda: a.attend(cache, q, table, lens, cu, **kw)

    a.attend(*ok)
    for f in (call(q=b.q.float()), call(q=b.q[:, :2]), call(q=b.q[0]), call(q=b.q.cpu()),
              call(table=b.table.long()), call(table=b.table[:1]), call(table=b.table.t()),
              call(lens=b.lens.float()), call(lens=b.lens[:1]), call(cu=b.cu[:2]),
              call(cu=b.cu.long()), call(cache=moe.KVCache(c.k, c.v)),
              call(cache=c._replace(k=c.k.view(torch.uint8))),
              call(cache=c._replace(v=c.v[:1])), call(cache=c._replace(k_scale=c.k_scale[..., :8])),
              call(out=b.q[:3]), call(out=b.q), call(cu=None),
              call(cache=c._replace(k=c.k.transpose(1, 2).contiguous().transpose(1, 2)))):
        refuse(f)
    assert a.attend(c, b.q[:0], b.table[:0], b.lens[:0]).shape == (0, 4, 64)
    with pytest.raises(TypeError):
        a.attend(c, b.q)


def test_places_beyond_32_bits(env):
    """Pages whose codes lie more than 2^32 bytes into the cache."""
    import torch
    moe, dev = env
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    d, page = 256, 64
    pages = (1 << 32) // (page * d) + 40
    a = moe.PagedAttention(2, 1, d, page, "int8", device=dev)
    c = a.new_cache(pages)
    g = torch.Generator(device=dev).manual_seed(1)
    table = ints(env, [[pages - 1, 3, pages - 30], [5, pages - 2, 7]])
    lens, cu = ints(env, [150, 190]), ints(env, [0, 150, 340])
    k, v = (torch.randn((340, 1, d), generator=g, device=dev).bfloat16() for _ in range(2))
    q = torch.randn((340, 2, d), generator=g, device=dev).bfloat16()
    a.write(c, k, v, table, lens, cu)
    got = a.attend(c, q, table, lens, cu)
    one = a.attend(c, q[[149, 339]].contiguous(), table, lens)
    few = a.new_cache(6)
    low = ints(env, [[0, 1, 2], [3, 4, 5]])
    a.write(few, k, v, low, lens, cu)
    assert torch.equal(got, a.attend(few, q, low, lens, cu))
    assert torch.equal(one, a.attend(few, q[[149, 339]].contiguous(), low, lens))
    back = a.read(c, table, lens, cu, rows=340)
    assert all(torch.equal(x, y) for x, y in zip(back, a.read(few, low, lens, cu, rows=340)))
    assert a.status() == 0
