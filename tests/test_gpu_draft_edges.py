"""Verification of drafted tokens where the weights' sum leaves fp32."""
import pytest

from test_gpu_draft import check, distributions
from util import gpu_env

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return gpu_env()


@pytest.mark.parametrize("v", [5, 3000, 151936])
def test_sums_beyond_fp32_are_refused(env, v):
    """Finite values whose sum is not; beside them a sequence whose sum just is."""
    import torch
    moe, dev = env
    most = torch.finfo(torch.float32).max
    p = torch.zeros((3, 1, v), device=dev)
    p[0, 0, :5] = most / 4          # 1.25 times the largest
    p[1, 0, 1:4] = most / 4         # 0.75 times
    p[2, 0, 0] = p[2, 0, 4] = most  # twice
    none = torch.empty((3, 0), dtype=torch.int32, device=dev)
    u = torch.full((3, 1), 0.5, device=dev)
    verifier = moe.DraftVerifier(device=dev)
    tokens, accepted = verifier.verify(p, none, u)
    assert tokens[:, 0].tolist() == [-1, 2, -1] and (accepted == 0).all()
    assert verifier.status() == moe.DEV_NONFINITE


def test_small_sums_keep_their_bits(env):
    p, q, d, u = distributions(env, 20, 3, 2000, 4)
    check(env, p * 2.0 ** -95, q * 2.0 ** -95, d, u)
    check(env, p * 2.0 ** 100, q * 2.0 ** 100, d, u)
