"""Bounded waits of the attention kernels.  With a wait budget of 1 ns a wait that does not
succeed at once gives up: the kernels set MOE_DEV_TIMEOUT, let copies and products in flight
finish, return, and leave the context usable.  In a child process, which reads the budget
once."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
sys.path.insert(0, {root!r})
import torch
import sparse_moe_decode_gb300 as moe
dev = torch.device("cuda:0")
bits = dict()
for kv in ("bf16", "int8", "e4m3"):
    for d in (64, 128, 256):
        for seqs, new, length in ((64, 1, 8000), (16, 300, 3000)):
            a = moe.PagedAttention(16, 8, d, 64, kv, device=dev)
            per = length // 64
            cache = a.new_cache(seqs * per)
            table = torch.arange(seqs * per, dtype=torch.int32, device=dev).view(seqs, per)
            lens = torch.full((seqs,), per * 64, dtype=torch.int32, device=dev)
            q = torch.randn((seqs * new, 16, d), device=dev).bfloat16()
            a.attend(cache, q, table, lens)
            torch.cuda.synchronize()
            bits[new] = bits.get(new, 0) | a.status()
y = torch.ones(1 << 20, device=dev).sum().item()  # the context still computes
print("RESULT", int(y), bits[1], bits[300])
"""


def test_wait_budget_expiry_sets_timeout_and_keeps_context():
    import __graft_entry__ as g
    g.build()
    import sparse_moe_decode_gb300 as moe
    env = dict(os.environ, MOE_WAIT_BUDGET_NS="1")
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    line = [l for l in r.stdout.splitlines() if l.startswith("RESULT")][-1].split()
    assert int(line[1]) == 1 << 20
    # (few rows, many rows: which of the calls gives up depends on the memory's load)
    assert int(line[2]) & moe.DEV_TIMEOUT and int(line[3]) & moe.DEV_TIMEOUT, line
