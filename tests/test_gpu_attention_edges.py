"""PagedAttention.attend where scores, scales and pages lie at an edge: rows and keys of
zeros, scores beyond the digits of fp32, values next to the smallest, pages that a window has
left behind.  The definition and its bounds stand in attn_ref."""
import numpy as np
import pytest

from attn_ref import BF16, FP16, attention
from test_gpu_attention import Batch
from util import gpu_env

pytestmark = pytest.mark.gpu

KV = ["bf16", "int8", "e4m3"]


@pytest.fixture(scope="module")
def env():
    return gpu_env()


def check_heads(b, out, heads):
    """Those query heads of every row against the definition."""
    got, q = out.double().cpu().numpy(), b.q.double().cpu().numpy()
    start = 0
    for n, length, (k, v, *scales) in zip(b.new, b.length, b.values()):
        want, bound = attention(q[start:start + n], k, v, length, b.attn.dims.scale, b.window,
                                *scales)
        err = np.abs(got[start:start + n] - want)[:, heads]
        assert (err <= bound[:, heads]).all()  # (NaN is not)
        start += n


def near_mean(got, values, kv):
    """Whether `got` is the mean over the values' first axis, as near as weights and values that
    enter rounded allow: attn_ref's bound without its term for scores (with a bf16 cache one
    rounding of a weight to bf16, with the others a weight's and a value's two to fp16)."""
    want, size = values.mean(0), np.abs(values).mean(0)
    entering = BF16 if kv == "bf16" else 3 * FP16
    bound = BF16 * np.abs(want) + (entering + 2.0 ** -18) * size + 2.0 ** -21
    return bool((np.abs(got - want) <= bound).all())  # (NaN is not)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [(4, 2), (6, 2)])
def test_zero_queries_beside_others_under_a_window(env, kv, d, heads):
    """One head's queries are 0, keys are tiny, and the rows of a warp see nothing of the key
    tile that the query tile begins with: the search for their maxima ends, and the other
    heads' rows are right."""
    import torch
    b = Batch(env, [190, 40], [400, 300], heads, d, 16, kv, window=7, k_std=2.0 ** -12).fill()
    b.q[:, 0] = 0
    out = b.attend()
    torch.cuda.synchronize()
    assert b.attn.status() == 0
    check_heads(b, out, slice(1, None))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [(4, 2), (6, 2)])
@pytest.mark.parametrize("window", [0, 50])
def test_scores_of_zero(env, kv, d, heads, window):
    """Zero or tiny queries and keys: the mean of the values that a row sees."""
    for q_size, k_size in ((0, 0), (2.0 ** -13, 0), (1, 0), (0, 2.0 ** -10), (0, 1),
                           (2.0 ** -60, 2.0 ** -60), (0, 2.0 ** -120)):
        b = Batch(env, [150, 2, 40], [333, 50, 40], heads, d, 16, kv, window, k_std=k_size).fill()
        b.q *= q_size
        b.check(b.attend())
        assert b.attn.status() == 0


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [[2, 1], [100, 300]])
def test_key_tiles_of_zeros(env, kv, d, new):
    """A key tile of zero keys among others, under queries of different sizes."""
    b = Batch(env, new, [700, 500], (4, 2), d, 64, kv)
    b.k[256:384] = 0
    b.k[700 + 384:] = 0
    b.q[::3] *= 2.0 ** -14
    b.q[1::3, 0] = 0
    b.fill()
    b.check(b.attend())


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("new", [[1, 1], [30, 100]])
def test_pages_never_written(env, kv, new):
    """Scales of 0, as a new cache has them: keys and values of 0."""
    b = Batch(env, new, [200, 130], (4, 2), 128, 64, kv)
    b.cache = b.attn.new_cache(b.cache.k.shape[0])
    assert (b.attend() == 0).all()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("power", [40, 80, 100])
def test_huge_queries_beside_huge_hidden_keys(env, kv, power):
    """The product of a row's and a key tile's powers of two is beyond fp32: rows that do not
    see the huge key, with scores of 0, give the mean of their values."""
    b = Batch(env, [140], [260], (4, 2), 128, 64, kv)
    b.q *= 2.0 ** power
    b.k[250] *= 2.0 ** power
    b.k[:250, :, 1:] = 0  # scores of one product each
    b.q[:130, :, 0] = 0   # ... of 0
    b.fill()
    out = b.attend()[:130].double().cpu().numpy()
    v = b.values()[0][1]
    for i in range(130):
        seen = v[:121 + i].repeat(2, 1)  # each query head's
        assert near_mean(out[i], seen, kv), i


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("heads,d", [((4, 2), 128), ((8, 1), 64), ((4, 2), 256)])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_a_key_that_is_nan_alone_in_its_tile(env, kv, heads, d, new):
    """A row that sees of one block's keys only a NaN one is NaN, whatever the others hold."""
    import torch
    for at in (64, 128, 512, 1024):  # the first position of a key tile
        b = Batch(env, [new, new], [at + new, at + 30], heads, d, 64, kv)
        b.k[at, 0, 3] = float("nan")
        b.fill()
        out = b.attend()
        group = heads[0] // heads[1]
        assert torch.isnan(out[:new, :group].float()).all()
        assert torch.isfinite(out[:new, group:].float()).all()
        b.check(out, skip=(0,))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [3, 150])
def test_scores_beyond_the_digits_of_fp32(env, kv, d, new):
    """Scores of 2^20 to 2^100, some 2^-8 of themselves apart: the largest one's value, up to
    2^26 in sequences of many rows; those say so from there on."""
    moe, _ = env
    for power in (20, 23, 34, 60, 100):
        for sign in (1, -1):
            b = Batch(env, [new], [400], (4, 2), d, 64, kv, scale=1.0)
            b.q[:, :, 1:] = 0
            b.q[:, :, 0] = sign * 2.0 ** power
            b.k[:, :, 1:] = 0
            b.fill()
            out = b.attend().double().cpu().numpy()
            if new > 8 and power > 26:
                assert b.attn.status() == moe.DEV_NONFINITE
                continue
            assert b.attn.status() == 0
            k, v = b.values()[0][:2]
            for i in range(new):
                for h in range(4):
                    s = k[:401 - new + i, h // 2, 0] * sign
                    vv = v[:401 - new + i, h // 2][s == s.max()]
                    assert near_mean(out[i, h], vv, kv), (power, sign, i, h)


def give_back(b, keep):
    """The pages that lie wholly before position `keep[i]` of sequence i are no longer in its
    table; they and page 0, which no sequence has, hold what is not finite.  Returns the table
    as it was."""
    import torch
    whole = b.table.clone()
    for x in b.cache:  # page 0's rows to a page that nobody has
        if x is not None:
            used = set(whole.flatten().tolist())
            spare = max(set(range(x.shape[0])) - used)
            x.view(torch.uint8)[spare] = x.view(torch.uint8)[0]
    b.table[b.table == 0] = spare
    whole[whole == 0] = spare
    for i, first in enumerate(keep):
        gone = max(0, first) // b.page
        b.poison([0] + b.table[i, :gone].tolist())
        b.table[i, :gone] = -1 if i % 2 else 1 << 30
    return whole


def finite(b):
    """What was poisoned made finite, for the definition, which multiplies it by 0."""
    for x, least in zip(b.cache, (0.0, 0.0, 2.0 ** -126, 2.0 ** -126)):
        if x is not None and x.is_floating_point():
            x.copy_(x.float().nan_to_num(least).to(x.dtype))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page,window", [(16, 100), (32, 33), (64, 200), (16, 1), (128, 500),
                                         (256, 260)])
@pytest.mark.parametrize("new,heads", [([1, 2, 1], (4, 2)), ([1, 40, 150], (6, 2))])
def test_pages_before_the_window_are_not_read(env, kv, d, page, window, new, heads):
    """A layer with a window that gives its old pages back."""
    b = Batch(env, new, [700, 333, 1111], heads, d, page, kv, window).fill()
    table = give_back(b, [x - n - window + 1 for x, n in zip(b.length, new)])
    out = b.attend()
    assert b.attn.status() == 0
    b.table = table
    finite(b)
    b.check(out)


@pytest.mark.parametrize("kv", KV)
def test_prompts_whose_first_pages_are_gone(env, kv):
    """A chunk of a long prompt behind a window, page 0 of another's rows that are not finite;
    a page inside the window that is missing is still told."""
    moe, _ = env
    b = Batch(env, [600], [5000], (8, 2), 128, 16, kv, window=777).fill()
    table = give_back(b, [5000 - 600 - 776])
    out = b.attend()
    assert b.attn.status() == 0
    gone, b.table = b.table, table
    finite(b)
    b.check(out)
    gone[0, (5000 - 600 - 776) // 16] = -1
    b.table = gone
    b.attend()
    assert b.attn.status() == moe.DEV_BAD_INDEX


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("new", [2, 20])
def test_values_next_to_the_smallest(env, kv, new):
    """Values of 2^-116 and many equal weights, tiles that one block begins and ends: outputs
    keep their digits (the definition's bound has 1e-37 for what fp32 cannot hold)."""
    b = Batch(env, [new] * 40, [4000] * 40, (8, 8), 64, 256, kv, uniform=True)
    b.q[:] = 0
    b.v.copy_(2.0 ** -116 * (1 + 0.5 * b.v.float().abs()))
    b.fill()
    b.check(b.attend())
