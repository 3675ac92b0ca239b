"""Calls of the routed-expert operators as a program makes them around other calls: the first of a
process, from several host threads at once, between a capture and its replay, with wrong tables."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import test_gpu_experts as base
from sparse_mla_decode_front_b200 import experts as G

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


PRODUCTS = """
import threading
import torch
from sparse_mla_decode_front_b200 import api, experts as G
g = torch.Generator(device="cuda").manual_seed(1)
e4m3 = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
blocks = lambda v: -(-v // 128)
scales = lambda *s: torch.rand(*s, generator=g, device="cuda")


def plain(m, n, k):
    args = (e4m3(m, k), scales(blocks(k), m), e4m3(n, k), scales(blocks(n), blocks(k)))
    return lambda out, stream=None: G.mla_fp8_matmul(*args, out, None, stream), (m, n)


def grouped(rows, n, k):
    m = 2 * rows
    off = torch.tensor([0, rows, m], dtype=torch.int32, device="cuda")
    args = (e4m3(m, k), scales(blocks(k), m), e4m3(2, n, k), scales(2, blocks(n), blocks(k)), off)
    return lambda out, stream=None: G.mla_fp8_grouped_matmul(*args, out, None, stream), (m, n)


def router(t, h):
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    args = (rnd(t, h), rnd(h), rnd(h, 64))
    return lambda out, stream=None: out.copy_(api.rmsnorm_router_topk(*args, top_k=4)[0]), (t, h)


def in_threads(jobs, after=None):
    errors = []

    def work(call, out, stream):
        try:
            if after is not None:
                after.wait()
            call(out, stream)
        except Exception as e:
            errors.append(e)
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors


def job(made):
    return made[0], torch.zeros(made[1], device="cuda"), torch.cuda.Stream()
"""


def test_a_host_threads_first_call_of_cuda():
    # the thread has no context yet, and nothing else in it has asked for one; inputs that no call saw
    run_alone(PRODUCTS + """
for make in (lambda: plain(1, 1536, 1024), lambda: plain(300, 512, 640), lambda: grouped(3, 144, 400),
             lambda: grouped(300, 144, 400), lambda: router(5, 256)):
    first = job(make())                          # this thread's call: what is kept for a device is known now
    first[0](first[1])
    call, out, _ = job(make())
    torch.cuda.synchronize()
    in_threads([(call, out, None)])
    again = torch.zeros_like(out)
    call(again)
    assert torch.equal(out, again) and bool(out.any())
""")


def test_first_products_of_a_process_from_several_host_threads():
    # each sees the same clusters per device, and so the same split and order of the sums
    run_alone(PRODUCTS + """
jobs = [job(plain(*s)) for s in [(1, 1536, 4096), (20, 144, 2064), (64, 2048, 1168), (300, 512, 640)] * 2]
torch.cuda.synchronize()
in_threads(jobs, threading.Barrier(len(jobs)))
for call, out, _ in jobs:
    again = torch.zeros_like(out)
    call(again)
    assert torch.equal(out, again) and bool(out.any())
""")


# ------------------------------------------------------------------ grouped products
def wrong_tables(R):
    return [[0, 9 * R, 10 * R, 20 * R], [-5, R // 10, R // 5, R // 3], [R // 2, R // 10, R // 5, R], [R] * 4,
            [0, 2 ** 31 - 1, -2 ** 31, 7], [R // 3, 0, 2 * R // 3, R // 2], [R, 0, 0, R], [-1, -2, -3, -4]]


@pytest.mark.parametrize("table", range(8))
@pytest.mark.parametrize("R", [24, 60, 100, 700])   # three groups: tiles of 16, 32 and 64 rows, and the many-rows form
def test_grouped_matmul_of_a_wrong_table_gives_the_clamped_groups(R, table):
    N, K = 272, 400
    x, xs = base.make_operand(R, K, R)
    w, ws = base.make_weight(3, N, K, 4)
    buf, status = base.filled(R + 2, N, dtype=torch.float32), torch.zeros(1, dtype=torch.int32, device="cuda")
    out, bad = buf[1:R + 1], wrong_tables(R)[table]
    G.mla_fp8_grouped_matmul(x, xs, w, ws, torch.tensor(bad, dtype=torch.int32, device="cuda"), out, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    ends = np.maximum.accumulate(np.clip(np.array(bad, np.int64), 0, R))   # clamped, and to the running maximum
    assert base.untouched(buf[0]) and base.untouched(buf[-1])
    assert base.untouched(out[:ends[0]]) and base.untouched(out[ends[-1]:])
    for e in range(3):
        part = slice(int(ends[e]), int(ends[e + 1]))
        if part.start < part.stop:
            base.check_product(out[part], x[part], xs[:, part], w[e], ws[e], torch.float32, f"expert {e}")


@pytest.mark.parametrize("N,K", [(16, 16), (272, 1040), (512, 256)])
@pytest.mark.parametrize("name", ["decode", "uneven", "long"])
def test_grouped_matmul_to_fp16(name, N, K):
    counts = base.GROUPS[name]
    ends = np.concatenate([[0], np.cumsum(counts)])
    x, xs = base.make_operand(int(ends[-1]), K, K)
    w, ws = base.make_weight(len(counts), N, K, N)
    out = base.filled(int(ends[-1]), N, dtype=torch.float16)
    G.mla_fp8_grouped_matmul(x, xs, w, ws, torch.tensor(ends, dtype=torch.int32, device="cuda"), out)
    for e, c in enumerate(counts):
        part = slice(ends[e], ends[e + 1])
        if c:
            base.check_product(out[part], x[part], xs[:, part], w[e], ws[e], torch.float16, f"expert {e}")


@pytest.mark.parametrize("dtype", base.DT)
@pytest.mark.parametrize("capacity", [8, 9, 32, 33, 48, 49])   # an expert: both sides of each change of form
def test_grouped_matmul_where_the_form_changes(capacity, dtype):
    E, N, K = 5, 144, 272
    counts = [0, 2 * capacity, 1, 3 * capacity // 2, capacity // 2 - 1]
    ends, R = np.concatenate([[0], np.cumsum(counts)]), E * capacity
    x, xs = base.make_operand(R, K, capacity)
    w, ws = base.make_weight(E, N, K, N)
    out = base.filled(R, N, dtype=dtype)
    G.mla_fp8_grouped_matmul(x, xs, w, ws, torch.tensor(ends, dtype=torch.int32, device="cuda"), out)
    for e, c in enumerate(counts):
        part = slice(ends[e], ends[e + 1])
        if c:
            base.check_product(out[part], x[part], xs[:, part], w[e], ws[e], dtype, f"expert {e}")
    assert base.untouched(out[ends[-1]:])


@pytest.mark.parametrize("rows", [1, 300])   # the few-rows form, and the many-rows one
def test_weights_beyond_32_bits(rows):
    E, N, K = 160, 4096, 7168                          # 4.7e9 bytes
    held, part = [0, 74, 159], 32                      # the second lies past 2^31, the third past 2^32
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda").view(base.E4M3)
    ws = torch.ones(E, N // 128, K // 128, device="cuda")
    for e in held:
        one, scale = base.make_weight(1, N, K, e)
        w.view(torch.uint8)[e], ws[e] = one[0].view(torch.uint8), scale[0]
    counts = np.zeros(E, np.int64)
    counts[held] = rows
    if rows > 1:
        counts[1:60] = 150                             # past 48 rows of capacity an expert
    ends = np.concatenate([[0], np.cumsum(counts)])
    x, xs = base.make_operand(int(ends[-1]), K, rows)
    out = base.filled(int(ends[-1]), N, dtype=torch.float32)
    G.mla_fp8_grouped_matmul(x, xs, w, ws, torch.tensor(ends, dtype=torch.int32, device="cuda"), out)
    for e in held:
        at = slice(int(ends[e]), int(ends[e + 1]))
        for f in (0, N - part):                        # the first features and the last
            base.check_product(out[at, f:f + part], x[at], xs[:, at], w[e, f:f + part], ws[e, f // 128:f // 128 + 1],
                               torch.float32, f"expert {e}")
    assert not out[int(ends[1]):int(ends[74])].any()


def test_more_operands_than_kept_tensor_maps():
    # every call's maps push out the oldest ones, several times round, and none is taken for another's
    M, N, K, count = 5, 48, 144, 150
    x, xs = base.make_operand(M, K, 1)
    w, ws = base.make_weight(count, N, K, 2)
    for _ in range(2):
        out = base.filled(count, M, N, dtype=torch.float32)
        for i in range(count):
            G.mla_fp8_matmul(x, xs, w[i], ws[i], out[i])
        for i in range(0, count, 7):
            base.check_product(out[i], x, xs, w[i], ws[i], torch.float32, f"weight {i}")


# ------------------------------------------------------------------ no rows, no tokens
def test_movers_without_rows_or_tokens():
    # a rank none of whose experts was taken, with buffers of no rows; and a call without tokens
    T, K, H = 3, 2, 64
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    w, row_of = torch.rand(T, K, device="cuda"), torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    rows = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    out, gw = base.filled(T, H, dtype=torch.bfloat16), base.filled(T, K, dtype=torch.float32)
    G.mla_moe_gather(x, row_of, rows)
    G.mla_moe_gather(x, row_of, torch.empty(0, H, dtype=torch.uint8, device="cuda").view(base.E4M3),
                     torch.empty(1, 0, device="cuda"))
    G.mla_moe_combine(rows, row_of, w, out)
    G.mla_moe_combine_backward(x, rows, row_of, w, torch.empty_like(rows), None)
    G.mla_moe_combine_backward(x, None, row_of, w, torch.empty_like(rows), None)
    G.mla_moe_combine_backward(x, rows, row_of, w, torch.empty_like(rows), gw)
    assert not out.any() and not gw.any()
    some = base.filled(4, H, dtype=torch.bfloat16)
    G.mla_moe_gather(x[:0], row_of[:0], some)
    G.mla_moe_combine(some, row_of[:0], w[:0], out[:0])
    G.mla_moe_combine_backward(x[:0], some, row_of[:0], w[:0], some, gw[:0])
    assert base.untouched(some)
