"""The routed-expert operators on the GPU against the fp64 oracle (oracle/moe_experts.py).

Tolerances count roundings (half a step: bf16 2^-8, fp16 2^-11, fp32 2^-24, e4m3 2^-4,
relative to the value):
* sort: whole numbers, equal; weights: one division and one product (2^-23) and the sum's
  K - 1 adds (2^-24 each).
* gather: equal. Quantised: the scale is one division (2^-24); the value before its
  rounding has a reciprocal and a product (2^-23), then half an e4m3 step: 2^-4 of the
  value, 2^-10 below the smallest normal.
* combine: K fused multiply-adds, each 2^-24 of the terms' summed magnitude, and the
  output's half step; the gradient of the weights likewise with H terms.
* product: a block's 128 exact products summed in fp32, at most a step (2^-23) of the terms'
  magnitude for each add (the tensor cores may truncate), a scaled add per block, and the
  output's half step.
"""
import numpy as np
import pytest
import torch

from oracle import moe_experts as X
from sparse_mla_decode_front_b200 import _lib, api, experts as G
from sparse_mla_decode_front_b200.device import ExpertLayer

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}   # half the subnormal step
DT = [torch.bfloat16, torch.float16, torch.float32]
E4M3 = torch.float8_e4m3fn
f64 = lambda t: t.double().cpu().numpy()
SENTINEL = 0x5B


def filled(*shape, dtype):
    """A tensor every byte of which is SENTINEL."""
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    return torch.full((n,), SENTINEL, dtype=torch.uint8, device="cuda").view(dtype).reshape(shape)


def untouched(t):
    return bool((t.contiguous().view(torch.uint8) == SENTINEL).all())


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def within(got, want, tol, what=""):
    """|got - want| <= tol element by element; NaN and infinities in the same places."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~fine & ~np.isnan(want)],
                                                                            want[~fine & ~np.isnan(want)]), what
    bad = np.abs(got - want)[fine] - np.broadcast_to(tol, want.shape)[fine]
    assert bad.size == 0 or bad.max() <= 0, f"{what}: over by {bad.max():.3g}"


def run_sort(idx, first, E, aff=None, normalize=False, scale=1.0, stream=None):
    T, K = idx.shape
    out = dict(expert_offsets=filled(E + 1, dtype=torch.int32), row_of=filled(T, K, dtype=torch.int32),
               source_of=filled(T * K, dtype=torch.int32))
    w = None if aff is None else filled(T, K, dtype=torch.float32)
    n = G.mla_moe_sort_workspace_bytes(T, K, E)
    ws = filled(n, dtype=torch.uint8) if n else None
    G.mla_moe_sort(idx, out["expert_offsets"], out["row_of"], out["source_of"], ws, first, aff, w, normalize, scale,
                   stream)
    return out, w


def random_rows(T, K, R, seed, missing=0.2):
    """row_of [T, K] with distinct rows, some choices without one (-1, or an index past the rows)."""
    g = gen(seed)
    perm = torch.randperm(max(R, T * K), generator=g, device="cuda")[:T * K].to(torch.int32).reshape(T, K)
    perm[torch.rand(T, K, generator=g, device="cuda") < missing] = -1
    return perm


# ------------------------------------------------------------------ sort
SORTS = [(1, 1, 1, 0, 1), (1, 8, 256, 0, 256), (128, 8, 256, 0, 256), (37, 5, 96, 48, 48), (512, 8, 256, 0, 256),
         (513, 8, 256, 0, 256), (300, 32, 1024, 0, 1024), (129, 32, 1024, 0, 1024), (12289, 8, 256, 64, 32),
         (4097, 1, 64, 63, 1), (1, 32, 64, 8, 8), (700, 7, 80, 0, 80),
         (100, 32, 1024, 0, 1024), (128, 32, 1024, 512, 512)]


@pytest.mark.parametrize("T,K,total,first,E", SORTS)
def test_sort_matches_oracle(T, K, total, first, E):
    idx = torch.randint(-1, total + 1, (T, K), generator=gen(T + K), device="cuda", dtype=torch.int32)   # duplicates, strays
    aff = torch.rand(T, total, generator=gen(5), device="cuda").to(torch.bfloat16)
    for normalize in (False, True):
        out, w = run_sort(idx, first, E, aff, normalize, 2.5)
        want = X.sort(idx.cpu().numpy(), first, E)
        for k, v in out.items():
            assert np.array_equal(v.cpu().numpy(), want[k]), k
        ref = X.routing_weights(idx.cpu().numpy(), f64(aff), normalize, 2.5)
        within(f64(w), ref, np.abs(ref) * (K + 2) * 2.0 ** -24, "weights")


@pytest.mark.parametrize("kind", ["none_here", "one_expert", "last_expert", "same_choice_twice", "extremes"])
@pytest.mark.parametrize("T", [3, 2000])
def test_sort_skewed(kind, T):
    idx = torch.randint(0, 64, (T, 4), generator=gen(1), device="cuda", dtype=torch.int32)
    if kind == "none_here":
        idx.fill_(-1)
    elif kind == "one_expert":
        idx.fill_(17)
    elif kind == "last_expert":
        idx.fill_(63)
    elif kind == "extremes":
        idx[:, 0], idx[:, 2] = -2 ** 31, 2 ** 31 - 1
    else:
        idx[:, 1] = idx[:, 0]
    first, E = (40, 16) if kind == "extremes" else (0, 64)
    out, _ = run_sort(idx, first, E)
    want = X.sort(idx.cpu().numpy(), first, E)
    for k, v in out.items():
        assert np.array_equal(v.cpu().numpy(), want[k]), k


def test_sort_many_passes_in_a_chunk():
    # 1.2 million choices: more passes than chunks, so a chunk places several passes
    T, K, E = 150001, 8, 40
    idx = torch.randint(0, 48, (T, K), generator=gen(2), device="cuda", dtype=torch.int32)
    out, _ = run_sort(idx, 4, E)
    e = idx.cpu().numpy().reshape(-1).astype(np.int64) - 4
    here = (e >= 0) & (e < E)
    order = np.argsort(np.where(here, e, E), kind="stable")[:here.sum()]
    src = out["source_of"].cpu().numpy()
    assert np.array_equal(src[:len(order)], order) and (src[len(order):] == -1).all()
    row = out["row_of"].cpu().numpy().reshape(-1)
    assert (row[~here] == -1).all() and np.array_equal(row[order], np.arange(len(order)))
    assert np.array_equal(out["expert_offsets"].cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(e[here], minlength=E))]))


def test_sort_of_no_tokens_zeroes_the_offsets():
    idx = torch.empty(0, 8, dtype=torch.int32, device="cuda")
    out, _ = run_sort(idx, 0, 33)
    assert not out["expert_offsets"].any()


def test_sort_weights_of_zero_affinities():
    idx = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device="cuda")
    aff = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    aff[1, 2] = 0.5
    _, w = run_sort(idx, 0, 64, aff, True, 3.0)
    assert w.tolist() == [[0.0, 0.0], [3.0, 0.0]]


# ------------------------------------------------------------------ gather and quantise
def check_quantized(q, scales, v, slack):
    """q, scales (device) against the values v; `slack`: relative error of the values before the division."""
    want, s = X.quantize(v)
    within(f64(scales), s, np.abs(s) * (2.0 ** -24 + slack), "scales")
    # a value's own error, relative to the block's largest (448 after scaling)
    within(f64(q), np.where(np.isnan(want), np.nan, np.clip(want, -448, 448)),
           np.abs(want) * (2.0 ** -4 + 2.0 ** -23) + 2.0 ** -10 + 448 * 2 * slack * (1 + 2.0 ** -4), "q")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,K,H,R", [(1, 8, 7168, 8), (5, 1, 16, 7), (37, 5, 1040, 185), (130, 10, 272, 1400),
                                     (3, 32, 4096 + 48, 96), (700, 2, 128, 1400)])
def test_gather(T, K, H, R, dtype):
    x = (torch.randn(T, H, generator=gen(H), device="cuda") * 3).to(dtype)
    row_of = random_rows(T, K, R, 3)
    row_of[0, 0] = R if T * K > 1 else 0             # past the rows: no row
    rows = filled(R, H, dtype=dtype)
    G.mla_moe_gather(x, row_of, rows)
    qrows, scales = filled(R, H, dtype=E4M3), filled(G.scale_blocks(H), R, dtype=torch.float32)
    G.mla_moe_gather(x, row_of, qrows, scales)
    r = row_of.reshape(-1).long()
    ok = (r >= 0) & (r < R)
    token = torch.arange(T, device="cuda").repeat_interleave(K)[ok]
    assert torch.equal(rows[r[ok]], x[token])
    check_quantized(qrows[r[ok]].float(), scales[:, r[ok]], f64(x[token]), 0.0)
    free = torch.ones(R, dtype=torch.bool, device="cuda")
    free[r[ok]] = False
    assert untouched(rows[free]) and untouched(qrows.view(torch.uint8)[free]) and untouched(scales[:, free])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("R,C", [(1, 16), (1, 2048), (7, 1040), (333, 272), (64, 7168)])
def test_quantize(R, C, gated, dtype):
    x = (torch.randn(R, 2 * C if gated else C, generator=gen(C + R), device="cuda") * 4).to(dtype)
    q, scales = filled(R, C, dtype=E4M3), filled(G.scale_blocks(C), R, dtype=torch.float32)
    G.mla_fp8_quantize(x, q, scales, gated)
    v = X.gated(f64(x)) if gated else f64(x)
    # |g| < 32: exp within 2 + 1.16 * 32 steps (2^-23), the sum, the division (2 steps) and the product
    check_quantized(q.float(), scales, v, 45 * 2.0 ** -23 if gated else 0.0)


def test_quantize_special_values():
    x = torch.zeros(6, 256, device="cuda")
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    x[3, :128] = 2.0 ** -120
    x[4, 0] = 3e38
    x[5] = torch.tensor([448.0, -448.0], device="cuda").repeat(128)
    q, scales = filled(6, 256, dtype=E4M3), filled(2, 6, dtype=torch.float32)
    G.mla_fp8_quantize(x, q, scales)
    with np.errstate(invalid="ignore"):                # 0 times an infinite scale
        back = f64(q.float()) * np.repeat(f64(scales).T, 128, 1)
    assert not back[0].any() and np.isfinite(f64(scales)[:, 0]).all()
    assert np.isnan(back[1, :128]).all() and not back[1, 128:].any()
    assert np.isnan(back[2, 128:]).all() and not back[2, :128].any()
    assert np.abs(back[3]).max() <= 2.0 ** -100
    assert back[4, 0] == pytest.approx(3e38, rel=2.0 ** -22) and not back[4, 1:].any()
    assert np.array_equal(back[5], f64(x[5]))


def test_quantize_gated_far_gates():
    x = torch.zeros(2, 32, device="cuda", dtype=torch.bfloat16)
    x[0, :16], x[0, 16:] = -300.0, 2.0          # silu of a far negative gate: 0, not NaN
    x[1, :16], x[1, 16:] = 300.0, 2.0
    q, scales = filled(2, 16, dtype=E4M3), filled(1, 2, dtype=torch.float32)
    G.mla_fp8_quantize(x, q, scales, True)
    assert not q.float()[0].any()
    np.testing.assert_allclose(f64(q.float()[1]) * f64(scales)[0, 1], 600.0, rtol=2.0 ** -20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_gated_far_gates_and_large_values(dtype):
    # silu(g) is below fp32's normal range, its product with u is not
    C = 64
    x = torch.empty(3, 2 * C, device="cuda")
    x[0, :C] = -torch.linspace(81, 165, C, device="cuda")
    x[1, :C] = -torch.linspace(86, 90, C, device="cuda")
    x[2, :C] = torch.linspace(-90, 8, C, device="cuda")
    x[:, C:] = torch.linspace(1e38, 3e38, C, device="cuda")
    x[2, C:] = 4e37
    x = x.to(dtype)
    q, scales = filled(3, C, dtype=E4M3), filled(1, 3, dtype=torch.float32)
    G.mla_fp8_quantize(x, q, scales, True)
    # exp of half the gate within 2 + 1.16 * 83 steps (2^-23), taken twice, and three products
    check_quantized(q.float(), scales, X.gated(f64(x)), (2 * (2 + 1.16 * 83) + 3) * 2.0 ** -23)


@pytest.mark.parametrize("valid", [-3, 0, 1, 77, 100, 5000])
def test_quantize_only_the_valid_rows(valid):
    x = torch.randn(100, 144, generator=gen(9), device="cuda").to(torch.bfloat16)
    q, scales = filled(100, 144, dtype=E4M3), filled(2, 100, dtype=torch.float32)
    ends = torch.tensor([7, 8, valid], dtype=torch.int32, device="cuda")
    G.mla_fp8_quantize(x, q, scales, False, ends[2:])
    n = min(max(valid, 0), 100)
    assert untouched(q.view(torch.uint8)[n:]) and untouched(scales[:, n:])
    check_quantized(q[:n].float(), scales[:, :n], f64(x[:n]), 0.0)


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,K,H,R", [(1, 8, 7168, 8), (5, 1, 16, 7), (37, 5, 1040, 185), (130, 10, 272, 1400),
                                     (3, 32, 4096 + 48, 96), (75, 8, 128, 600)])
def test_combine_and_gradient(T, K, H, R, weighted, dtype):
    rows = torch.randn(R, H, generator=gen(H), device="cuda").to(dtype)
    row_of = random_rows(T, K, R, 4)
    row_of[T - 1] = -1                                # a token without rows
    if K > 2:
        row_of[0, 1] = R
    w = torch.randn(T, K, generator=gen(6), device="cuda") if weighted else None
    if weighted:
        w[row_of < 0] = float("nan")                  # weights of absent choices are never used
    r, rn = row_of.cpu().numpy(), f64(rows)
    wn = f64(w) if weighted else None
    out = filled(T, H, dtype=dtype)
    G.mla_moe_combine(rows, row_of, w, out)
    want = X.combine(rn, r, wn)
    mag = X.combine(np.abs(rn), r, None if wn is None else np.abs(wn))
    within(f64(out), want, mag * K * 2.0 ** -24 + np.abs(want) * HALF[dtype] * (1 + 2.0 ** -8) + TINY[dtype], "out")

    dout = torch.randn(T, H, generator=gen(8), device="cuda").to(dtype)
    gr, gw = filled(R, H, dtype=dtype), filled(T, K, dtype=torch.float32)
    G.mla_moe_combine_backward(dout, rows, row_of, w, gr, gw)
    want_r, want_w = X.combine_backward(f64(dout), rn, r, wn)
    used = ~np.isnan(want_r[:, 0])
    at = torch.from_numpy(used).cuda()
    within(f64(gr[at]), want_r[used], np.abs(want_r[used]) * HALF[dtype] * (1 + 2.0 ** -8) + TINY[dtype], "grad_rows")
    assert untouched(gr[~at])
    _, mag_w = X.combine_backward(np.abs(f64(dout)), np.abs(rn), r, None)
    within(f64(gw), want_w, mag_w * H * 2.0 ** -24, "grad_weights")

    # one of the two alone, and the values are the same from run to run
    gr1, gw1 = filled(R, H, dtype=dtype), filled(T, K, dtype=torch.float32)
    G.mla_moe_combine_backward(dout, None, row_of, w, gr1, None)
    G.mla_moe_combine_backward(dout, rows, row_of, w, None, gw1)
    assert torch.equal(gr1.view(torch.uint8), gr.view(torch.uint8)) and torch.equal(gw1, gw)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [296, 297, 592, 593, 1184, 1185])
def test_combine_backward_at_every_team_size(n, dtype):
    T, K, H = n, 1, 16 * 37
    rows, dout = (torch.randn(T, H, generator=gen(n + i), device="cuda").to(dtype) for i in range(2))
    row_of = random_rows(T, K, T, 4)
    gr, gw = filled(T, H, dtype=dtype), filled(T, K, dtype=torch.float32)
    G.mla_moe_combine_backward(dout, rows, row_of, None, gr, gw)
    want_r, want_w = X.combine_backward(f64(dout), f64(rows), row_of.cpu().numpy(), None)
    used = ~np.isnan(want_r[:, 0])
    assert np.array_equal(f64(gr)[used], want_r[used])
    assert untouched(gr[~torch.from_numpy(used).cuda()])
    _, mag_w = X.combine_backward(np.abs(f64(dout)), np.abs(f64(rows)), row_of.cpu().numpy(), None)
    within(f64(gw), want_w, mag_w * H * 2.0 ** -24, "grad_weights")


def test_gather_gradient_is_the_unweighted_combine():
    # <gather(x), g> differentiated by differences in fp64, against combine(g)
    T, K, H, R = 6, 3, 32, 18
    row_of = random_rows(T, K, R, 11)
    g = torch.randn(R, H, generator=gen(12), device="cuda")
    x = torch.randn(T, H, generator=gen(13), device="cuda")
    dx = filled(T, H, dtype=torch.float32)
    G.mla_moe_combine(g, row_of, None, dx)

    def loss(xv):
        rows = torch.zeros(R, H, device="cuda")
        G.mla_moe_gather(xv, row_of, rows)
        return float((rows.double() * g.double()).sum())
    for t, h in [(0, 0), (2, 31), (5, 7)]:
        step = 0.5
        up, down = x.clone(), x.clone()
        up[t, h] += step
        down[t, h] -= step
        width = float(up[t, h].double() - down[t, h].double())
        # linear: the difference quotient is the gradient but for the sums' fp64 rounding
        assert (loss(up) - loss(down)) / width == pytest.approx(float(dx[t, h]), abs=1e-5)


# ------------------------------------------------------------------ products
def make_operand(rows, K, seed):
    g = gen(seed)
    x = (torch.randn(rows, K, generator=g, device="cuda") * 60).clamp(-448, 448).to(E4M3)
    return x, torch.exp(torch.randn(G.scale_blocks(K), rows, generator=g, device="cuda")) * 2.0 ** -7


def make_weight(E, N, K, seed):
    g = gen(seed)
    w = (torch.randn(E, N, K, generator=g, device="cuda") * 60).clamp(-448, 448).to(E4M3)
    return w, torch.exp(torch.randn(E, G.scale_blocks(N), G.scale_blocks(K), generator=g, device="cuda")) * 2.0 ** -9


def check_product(out, x, xs, w, ws, dtype, what=""):
    want, mag = X.product(f64(x.float()), f64(xs), f64(w.float()), f64(ws))
    K = x.shape[1]
    tol = mag * (128 + 2 * G.scale_blocks(K) + 4) * 2.0 ** -23 + np.abs(want) * HALF[dtype] * (1 + 2.0 ** -8) + TINY[dtype]
    within(f64(out), want, tol, what)


PRODUCTS = [(1, 16, 16), (1, 1536, 7168), (16, 128, 128), (17, 576, 1040), (33, 272, 144), (64, 144, 4112),
            (65, 256, 256), (129, 400, 272), (300, 144, 2064), (513, 1040, 528), (1031, 512, 640)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_matmul(M, N, K, dtype):
    x, xs = make_operand(M, K, M + K)
    w, ws = make_weight(1, N, K, N)
    out, status = filled(M, N, dtype=dtype), torch.zeros(1, dtype=torch.int32, device="cuda")
    G.mla_fp8_matmul(x, xs, w[0], ws[0], out, status)
    torch.cuda.synchronize()
    assert api.mla_get_device_status(status) == 0
    check_product(out, x, xs, w[0], ws[0], dtype)


# every width of a feature tile, several tiles a CTA (pair) with an odd count of K blocks, and K
# split over clusters of 2, 4 and 8 CTAs with runs of unequal length
WIDE = [(300, n, 256) for n in range(16, 257, 16)] + [(4100, 1040, 272), (33, 20480, 272), (150, 9600, 400)]
SPLIT = [(m, n, k) for m, n in [(1, 16), (20, 144), (64, 272), (100, 2048)] for k in (512, 640, 1168, 2064, 4112)]


@pytest.mark.parametrize("M,N,K", WIDE + SPLIT)
def test_matmul_tilings(M, N, K):
    x, xs = make_operand(M, K, M + N)
    w, ws = make_weight(1, N, K, N + K)
    buf = filled(M + 2, N, dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    G.mla_fp8_matmul(x, xs, w[0], ws[0], buf[1:M + 1], status)
    torch.cuda.synchronize()
    assert int(status) == 0 and untouched(buf[0]) and untouched(buf[-1])
    check_product(buf[1:M + 1], x, xs, w[0], ws[0], torch.bfloat16)


@pytest.mark.parametrize("N,K", [(n, 272) for n in range(16, 257, 48)] + [(1040, 272)])
def test_grouped_matmul_tilings(N, K):
    counts = [300] * 6 + [1, 127, 128, 129, 515]       # 1040: more tiles than CTAs
    off = np.concatenate([[0], np.cumsum(counts)])
    x, xs = make_operand(int(off[-1]), K, N)
    w, ws = make_weight(len(counts), N, K, K)
    out = filled(int(off[-1]), N, dtype=torch.bfloat16)
    G.mla_fp8_grouped_matmul(x, xs, w, ws, torch.tensor(off, dtype=torch.int32, device="cuda"), out)
    for e, c in enumerate(counts):
        part = slice(off[e], off[e + 1])
        check_product(out[part], x[part], xs[:, part], w[e], ws[e], torch.bfloat16, f"expert {e}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(2560, 2048, 4096), (2500, 2000, 4112), (512, 10240, 4096), (4000, 7152, 2064)])
def test_matmul_a_few_tiles_past_whole_waves(M, N, K, dtype):
    # tiles a few past whole waves of CTA pairs: every tile once, and no row behind the last
    x, xs = make_operand(M, K, M + N)
    w, ws = make_weight(1, N, K, N + K)
    buf = filled(M + 2, N, dtype=dtype)
    G.mla_fp8_matmul(x, xs, w[0], ws[0], buf[1:M + 1])
    torch.cuda.synchronize()
    assert untouched(buf[0]) and untouched(buf[-1])
    rng = np.random.default_rng(M)
    edges = [r for b in range(0, M, 256) for r in (b - 1, b, b + 128) if 0 <= r < M] + [M - 1]
    at = torch.tensor(sorted(set(edges + rng.integers(0, M, 60).tolist())), device="cuda")
    check_product(buf[1:M + 1][at], x[at], xs[:, at].contiguous(), w[0], ws[0], dtype)
    assert bool(torch.isfinite(buf[1:M + 1].float()).all())
    again = filled(M, N, dtype=dtype)
    G.mla_fp8_matmul(x, xs, w[0], ws[0], again)
    assert torch.equal(again, buf[1:M + 1])


def test_offsets_beyond_32_bits():
    # an output of 2.3e9 elements, rows gathered into 2.4e9 bytes, and back
    M, N, K = 70001, 32768, 128
    x, xs = make_operand(M, K, 1)
    w, ws = make_weight(1, N, K, 2)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    G.mla_fp8_matmul(x, xs, w[0], ws[0], out)
    at = [0, 65535, 65536, M - 1]
    check_product(out[at], x[at], xs[:, at].contiguous(), w[0], ws[0], torch.bfloat16)
    del out
    T, H, R = 50, 8192, 300007
    v = torch.randn(T, H, generator=gen(3), device="cuda").to(torch.bfloat16)
    row_of = (R - 1 - 6000 * torch.arange(T, device="cuda", dtype=torch.int32)).reshape(T, 1)
    rows, scales = torch.zeros(R, H, dtype=torch.uint8, device="cuda").view(E4M3), torch.zeros(64, R, device="cuda")
    G.mla_moe_gather(v, row_of, rows, scales)
    r = row_of[:, 0].long()
    check_quantized(rows[r].float(), scales[:, r], f64(v), 0.0)
    wide = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    G.mla_moe_gather(v, row_of, wide)
    back = torch.empty_like(v)
    G.mla_moe_combine(wide, row_of, None, back)
    assert torch.equal(back, v)


GROUPS = {
    "decode": [0, 3, 0, 1, 5, 0, 0, 2],
    "one_row": [0, 0, 1],
    "uneven": [17, 1, 130, 0, 16, 300, 2],
    "one_expert": [0, 0, 400, 0],
    "tiles": [128, 256, 64, 32, 16, 0, 128],
    "empty": [0, 0, 0],
    "long": [700, 900, 1],
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(16, 16), (272, 1040), (512, 256)])
@pytest.mark.parametrize("name", sorted(GROUPS))
def test_grouped_matmul(name, N, K, dtype):
    counts = GROUPS[name]
    E, used = len(counts), sum(counts)
    R = used + 9                                       # rows behind the last expert's
    off = np.concatenate([[0], np.cumsum(counts)])
    x, xs = make_operand(R, K, used + K)
    xs[:, used:] = float("nan")                        # never looked at
    w, ws = make_weight(E, N, K, N)
    out, status = filled(R, N, dtype=dtype), torch.zeros(1, dtype=torch.int32, device="cuda")
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    G.mla_fp8_grouped_matmul(x, xs, w, ws, offsets, out, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for e in range(E):
        part = slice(off[e], off[e + 1])
        if counts[e]:
            check_product(out[part], x[part], xs[:, part], w[e], ws[e], dtype, f"expert {e}")
    assert untouched(out[used:])


def test_grouped_matmul_many_experts():
    E, N, K = 1024, 64, 256
    counts = np.random.default_rng(0).integers(0, 3, E)
    off = np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    x, xs = make_operand(R, K, 1)
    w, ws = make_weight(E, N, K, 2)
    out = filled(R, N, dtype=torch.float32)
    G.mla_fp8_grouped_matmul(x, xs, w, ws, torch.tensor(off, dtype=torch.int32, device="cuda"), out)
    # every expert alone is the same call with the others empty: compare against per-expert products
    for e in list(range(0, E, 37)) + [E - 1]:
        part = slice(off[e], off[e + 1])
        if counts[e]:
            check_product(out[part], x[part], xs[:, part], w[e], ws[e], torch.float32, f"expert {e}")
    assert not untouched(out[R - 1:]) or counts[-1] == 0


@pytest.mark.parametrize("bad", [[0, 900, 1000, 2000], [-5, 10, 20, 30], [40, 10, 20, 100], [100, 100, 100, 100],
                                 [0, 2**31 - 1, -2**31, 7]])
def test_grouped_matmul_clamps_wrong_offsets(bad):
    R, N, K = 100, 144, 256
    x, xs = make_operand(R, K, 3)
    w, ws = make_weight(3, N, K, 4)
    buf = filled(R + 2, N, dtype=torch.float32)
    out = buf[1:R + 1]
    G.mla_fp8_grouped_matmul(x, xs, w, ws, torch.tensor(bad, dtype=torch.int32, device="cuda"), out)
    torch.cuda.synchronize()
    assert untouched(buf[0]) and untouched(buf[-1])


def test_grouped_matmul_overlapping_offsets_stay_bounded():
    R, E, N, K = 500, 1024, 16, 16
    x, xs = make_operand(R, K, 3)
    w, ws = make_weight(E, N, K, 4)
    offsets = torch.tensor([0, R], dtype=torch.int32, device="cuda").repeat(513)[:E + 1].contiguous()
    out = filled(R, N, dtype=torch.float32)
    G.mla_fp8_grouped_matmul(x, xs, w, ws, offsets, out)   # 512 groups claim all rows: the first gets them
    check_product(out, x, xs, w[0], ws[0], torch.float32)


def test_nan_stays_in_its_row_and_column():
    M, N, K = 40, 272, 256
    x, xs = make_operand(M, K, 5)
    w, ws = make_weight(1, N, K, 6)
    x.view(torch.uint8)[7, 3] = 0x7F                   # e4m3 NaN
    w.view(torch.uint8)[0, 130, 200] = 0x7F
    xs[1, 9] = float("inf")
    out = filled(M, N, dtype=torch.float32)
    G.mla_fp8_matmul(x, xs, w[0], ws[0], out)
    nan = torch.isnan(out)
    assert bool(nan[7].all()) and bool(nan[:, 130].all())
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[[7, 9]] = False
    cols = torch.ones(N, dtype=torch.bool, device="cuda")
    cols[130] = False
    assert bool(torch.isfinite(out[keep][:, cols]).all())


# ------------------------------------------------------------------ together
class Layer:
    """The router and its experts, as a decode step or a prompt chunk runs them (device.ExpertLayer),
    with every buffer filled with a sentinel first."""

    def __init__(self, T, H, I, E, K, first, held, seed):
        g = gen(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.T, self.H, self.I, self.E, self.K, self.first, self.held = T, H, I, E, K, first, held
        self.x = rnd(T, H).to(torch.bfloat16)
        gamma = (1 + 0.1 * rnd(H)).to(torch.bfloat16)
        router_w = (rnd(H, E) / H ** 0.5).to(torch.bfloat16)
        self.w1, self.s1 = make_weight(held, 2 * I, H, seed + 1)
        self.w2, self.s2 = make_weight(held, H, I, seed + 2)
        self.s1 *= 2.0 ** -3 * (512 / H) ** 0.5
        self.layer = layer = ExpertLayer(T, gamma, router_w, self.w1, self.s1, self.w2, self.s2, K, first, scale=2.5)
        for name in ("norm", "affinities", "topk_idx", "row_of", "expert_offsets", "source_of", "weights", "x",
                     "x_scales", "gate_up", "h", "h_scales", "y", "out", "router_workspace", "sort_workspace"):
            t = getattr(layer, name)
            if t is not None:
                t.view(torch.uint8).fill_(SENTINEL)
        self.norm, self.idx, self.aff = layer.norm, layer.topk_idx, layer.affinities
        self.off, self.row, self.wt, self.out, self.status = (layer.expert_offsets, layer.row_of, layer.weights,
                                                              layer.out, layer.status)

    def run(self, stream=None):
        return self.layer.run(self.x, stream)

    def check(self):
        """The layer's output against the oracle on the layer's own norm rows and choices, with the
        8-bit roundings of the path (2^-4 an element, averaging out over a product) bounded in norm."""
        torch.cuda.synchronize()
        assert self.layer.device_status() == 0
        idx, x = self.idx.cpu().numpy(), f64(self.norm)
        s = X.sort(idx, self.first, self.held)
        assert np.array_equal(self.off.cpu().numpy(), s["expert_offsets"])
        assert np.array_equal(self.row.cpu().numpy(), s["row_of"])
        n = int(s["expert_offsets"][-1])
        w = X.routing_weights(idx, f64(self.aff), True, 2.5)
        within(f64(self.wt), w, np.abs(w) * (self.K + 2) * 2.0 ** -24, "weights")
        tokens = s["source_of"][:n] // self.K
        qv, qs = X.quantize(x[tokens])
        qv = X.round_e4m3(qv)
        y = np.zeros((n, self.H))
        for e in range(self.held):
            part = slice(s["expert_offsets"][e], s["expert_offsets"][e + 1])
            if part.start == part.stop:
                continue
            h, _ = X.product(qv[part], qs[:, part], f64(self.w1[e].float()), f64(self.s1[e]))
            av, as_ = X.quantize(X.gated(h))
            y[part], _ = X.product(X.round_e4m3(av), as_, f64(self.w2[e].float()), f64(self.s2[e]))
        want = X.combine(y, s["row_of"], w)
        got = f64(self.out)
        # what differs: h and y rounded to bf16 (2^-8 each at most), which moves some activations
        # across an e4m3 border (2^-3 of those at most, of 1 in 2^3 of them): 2^-8 (1 + 1 + 2) + 2^-8
        assert np.linalg.norm(got - want) <= 5 * 2.0 ** -8 * np.linalg.norm(want)
        none = (s["row_of"] < 0).all(1)
        assert not got[none].any()


LAYERS = [(1, 1024, 256, 64, 6, 0, 64), (128, 1024, 256, 256, 8, 64, 32), (37, 1040, 144, 96, 5, 0, 96),
          (601, 512, 128, 64, 8, 0, 64)]


@pytest.mark.parametrize("cfg", LAYERS)
def test_layer(cfg):
    layer = Layer(*cfg, seed=21)
    layer.run()
    layer.check()


def test_layer_in_a_graph_and_on_another_stream():
    layer = Layer(*LAYERS[1], seed=31)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    layer.run(s)
    s.synchronize()
    first = layer.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer.run(s)
    for seed in (41, 42):
        layer.x.copy_(torch.randn(layer.T, layer.H, generator=gen(seed), device="cuda"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = layer.out.clone()
        layer.check()
        layer.run()
        torch.cuda.synchronize()
        assert torch.equal(layer.out, replayed)        # the same from run to run
    assert not torch.equal(first, layer.out)


def test_chunked_sort_and_products_in_a_graph():
    layer = Layer(1201, 512, 128, 64, 8, 0, 64, seed=71)   # 9608 choices: two launches, a workspace
    layer.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        layer.run(s)
    for seed in (72, 73):
        layer.x.copy_(torch.randn(layer.T, layer.H, generator=gen(seed), device="cuda"))
        torch.cuda.synchronize()
        g.replay()
        g.replay()
        layer.check()


def test_first_calls_of_a_process_inside_a_capture():
    code = """
import torch
from sparse_mla_decode_front_b200 import experts as G
idx = torch.randint(0, 64, (600, 8), device="cuda", dtype=torch.int32)
off, row, src = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (65, 4800, 4800))
ws = torch.empty(G.mla_moe_sort_workspace_bytes(600, 8, 64), dtype=torch.uint8, device="cuda")
x = torch.ones(3, 512, device="cuda").to(torch.float8_e4m3fn)
w = torch.ones(64, 512, device="cuda").to(torch.float8_e4m3fn)
xs, wsc, out = torch.ones(4, 3, device="cuda"), torch.ones(1, 4, device="cuda"), torch.zeros(3, 64, device="cuda")
big, bs = torch.ones(600, 512, device="cuda").to(torch.float8_e4m3fn), torch.ones(4, 600, device="cuda")
bout = torch.zeros(600, 64, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    G.mla_moe_sort(idx, off, row.view(600, 8), src, ws)
    G.mla_fp8_matmul(x, xs, w, wsc, out)
    G.mla_fp8_matmul(big, bs, w, wsc, bout)
g.replay()
torch.cuda.synchronize()
assert int(off[-1]) == 4800 and bool((out == 512).all()) and bool((bout == 512).all())
print("fine")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_two_layers_on_two_streams_at_once():
    layers = [Layer(*LAYERS[1], seed=51), Layer(*LAYERS[3], seed=61)]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(4):
        for layer, s in zip(layers, streams):
            layer.run(s)
    for layer in layers:
        layer.check()


def test_calls_refuse_wrong_arguments():
    x, xs = make_operand(4, 128, 1)
    w, ws = make_weight(1, 32, 128, 1)
    out = torch.empty(4, 32, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        G.mla_fp8_matmul(x, xs.t().contiguous(), w[0], ws[0], out)
    with pytest.raises(ValueError, match="contiguous"):
        G.mla_fp8_matmul(x, xs, w[0], ws[0], torch.empty(32, 4, dtype=torch.bfloat16, device="cuda").t())
    with pytest.raises(ValueError, match="float8"):
        G.mla_fp8_matmul(x.float(), xs, w[0], ws[0], out)
    with pytest.raises(ValueError, match="bfloat16"):
        G.mla_fp8_matmul(x, xs, w[0], ws[0], out.double())
    with pytest.raises(_lib.MlaError):
        G.mla_fp8_matmul(x[:, :24].contiguous(), xs, w[0][:, :24].contiguous(), ws[0], out)
    idx = torch.zeros(2000, 8, dtype=torch.int32, device="cuda")
    row, src = torch.empty_like(idx), torch.empty(16000, dtype=torch.int32, device="cuda")
    off = torch.empty(9, dtype=torch.int32, device="cuda")
    with pytest.raises(_lib.MlaError):
        G.mla_moe_sort(idx, off, row, src)              # needs a workspace
    with pytest.raises(ValueError, match="together"):
        G.mla_moe_sort(idx, off, row, src, None, 0, torch.zeros(2000, 8, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="both None"):
        G.mla_moe_combine_backward(out, out, row, None, None, None)
