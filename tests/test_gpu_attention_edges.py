"""PagedAttention.attend where scores, scales and pages lie at an edge: rows and keys of
zeros, scores beyond the digits of fp32, values next to the smallest, pages that a window has
left behind.  The definition and its bounds stand in attn_ref."""
import numpy as np
import pytest

from attn_ref import attention
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
