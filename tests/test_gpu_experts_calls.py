"""Calls of the routed-expert operators as a program makes them around other calls: the first of a
process, from several host threads at once, between a capture and its replay, with wrong tables."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Sorts T x 8 choices among E experts and compares with a stable sort on the host.
SORT = """
import numpy as np
import torch
from sparse_mla_decode_front_b200 import experts as G


def check_sort(E, T, K=8):
    idx = torch.randint(0, E, (T, K), generator=torch.Generator(device="cuda").manual_seed(E + T), device="cuda",
                        dtype=torch.int32)
    off, row, src = (torch.full((n,), -7, dtype=torch.int32, device="cuda") for n in (E + 1, T * K, T * K))
    n = G.mla_moe_sort_workspace_bytes(T, K, E)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    G.mla_moe_sort(idx, off, row.view(T, K), src, ws)
    e = idx.cpu().numpy().reshape(-1)
    order = np.argsort(e, kind="stable")
    assert np.array_equal(src.cpu().numpy(), order)
    assert np.array_equal(row.cpu().numpy()[order], np.arange(T * K))
    assert np.array_equal(off.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(e, minlength=E))]))
"""


def run_alone(code):
    r = subprocess.run([sys.executable, "-c", code + "\nprint('fine')"], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("E", [612, 613, 680, 681, 1024])
def test_first_sort_of_a_process(E):
    # a block's shared memory (static and dynamic) is just past what a launch may use without asking at
    # 680 and 681 experts (one launch) and at 612 and 613 (two); no call before raised the limit
    run_alone(SORT + f"check_sort({E}, 4)\ncheck_sort({E}, 1000)")


THREADS = SORT + """
import threading

jobs = []
for E in (700, 1024):
    idx = torch.randint(0, E, (TOKENS, 8), device="cuda", dtype=torch.int32)
    out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, TOKENS * 8, TOKENS * 8)]
    n = G.mla_moe_sort_workspace_bytes(TOKENS, 8, E)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    jobs.append((torch.cuda.Stream(), (idx, out[0], out[1].view(TOKENS, 8), out[2], ws)))
torch.cuda.synchronize()
errors = []


def work(stream, args):
    try:
        for _ in range(3000):
            G.mla_moe_sort(*args, stream=stream)
    except Exception as e:
        errors.append(e)


threads = [threading.Thread(target=work, args=j) for j in jobs]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not errors, errors
for _, (idx, off, row, src, _) in jobs:
    e = idx.cpu().numpy().reshape(-1)
    assert np.array_equal(src.cpu().numpy(), np.argsort(e, kind="stable"))
"""


@pytest.mark.parametrize("tokens", [4, 1000])
def test_two_host_threads_sort_for_different_expert_counts(tokens):
    # each call's shared memory differs, and both are past what a launch may use without asking
    run_alone(THREADS.replace("TOKENS", str(tokens)))


def test_sort_captured_for_many_experts_replays_after_a_call_for_fewer():
    run_alone(SORT + """
E, T = 1024, 1000
idx = torch.randint(0, E, (T, 8), device="cuda", dtype=torch.int32)
off, row, src = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * 8, T * 8))
ws = torch.empty(G.mla_moe_sort_workspace_bytes(T, 8, E), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    G.mla_moe_sort(idx, off, row.view(T, 8), src, ws)
check_sort(700, 1000)
check_sort(640, 4)
g.replay()
torch.cuda.synchronize()
assert np.array_equal(src.cpu().numpy(), np.argsort(idx.cpu().numpy().reshape(-1), kind="stable"))
""")
