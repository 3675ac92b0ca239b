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
