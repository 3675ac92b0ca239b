"""Run a few block steps of a synthetic workload and exit (for profilers).

    python -m sparse_mla_decode_front_b200.profile_step --workload gather128 --steps 2 [--separate]
    python -m sparse_mla_decode_front_b200.profile_step --router router_ds128 --steps 3
    python -m sparse_mla_decode_front_b200.profile_step --tp-world 1 --steps 3
    python -m sparse_mla_decode_front_b200.profile_step --experts 128 --steps 3
    python -m sparse_mla_decode_front_b200.profile_step --fp8-matmul 2048 7168 4096 --steps 3

Uploads the workload once, runs ``--steps`` calls of the block on cuda:0 (with
``--separate``: the two calls of the separate path, qkv then attention, per step;
with ``--router CASE``: the fused RMSNorm + router top-K on that router case instead;
with ``--tp-world W``: the head split's fused o-projection + reduction on the block's
o-projection shape, every one of W ranks on this GPU; with ``--experts T``: the router and
32 of 256 routed experts, hidden 7168, expert width 2048, top 8, on T tokens; with
``--fp8-matmul M N K``: the block-scaled 8-bit product alone),
synchronises and checks the device status word. Launch count per step is
printed so a profiler's skip/count options can be set (e.g. ncu -s / -c).
"""
from __future__ import annotations

import argparse
import sys

import torch

from . import synth
from .device import DecodeStep


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", default="gather128", choices=[w.name for w in synth.WORKLOADS])
    ap.add_argument("--steps", type=int, default=2)
    ap.add_argument("--separate", action="store_true", help="the separate qkv and attention calls")
    ap.add_argument("--router", default=None, choices=[c.name for c in synth.ROUTER_CASES],
                    help="run the router case instead of the block")
    ap.add_argument("--tp-world", type=int, default=0, help="run the head split's o-projection for W ranks")
    ap.add_argument("--experts", type=int, default=0, metavar="T", help="run the routed experts on T tokens")
    ap.add_argument("--fp8-matmul", type=int, nargs=3, default=None, metavar=("M", "N", "K"))
    args = ap.parse_args(argv)
    if args.experts:
        return _experts(args)
    if args.fp8_matmul:
        return _fp8_matmul(args)
    if args.router:
        return _router(args)
    if args.tp_world:
        return _tp_o_proj(args)
    step = DecodeStep(synth.make_inputs(synth.WORKLOAD_BY_NAME[args.workload].index), device="cuda:0")
    for _ in range(args.steps):
        if args.separate:
            step.run_separate()
        else:
            step.run()
    torch.cuda.synchronize()
    status = step.device_status()
    per_step = "two calls" if args.separate else f"{step.n_launches} kernels"
    print(f"{args.workload}: {args.steps} steps, {per_step} per step, device status {status:#x}")
    return 0 if status == 0 else 1


def _router(args) -> int:
    import numpy as np
    from . import api
    case = synth.ROUTER_CASE_BY_NAME[args.router]
    inp = synth.make_router_inputs(case.index)
    dev = torch.device("cuda:0")
    t16 = lambda bits: torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(dev)
    x, g, w = (t16(inp[k]) for k in ("hidden_states", "gamma", "router_weights"))
    b = None if inp["router_bias"] is None else t16(inp["router_bias"])
    T, H, E, K = case.n_tokens, case.hidden, case.n_experts, case.top_k
    norm = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    aff = torch.empty((T, E), dtype=torch.bfloat16, device=dev)
    ws = torch.empty(api.mla_router_workspace_bytes(T, H, E, K), dtype=torch.uint8, device=dev)
    for _ in range(args.steps):
        api.mla_rmsnorm_router_topk(x, g, w, b, inp["eps"], K, case.act, norm, idx, aff, ws)
    torch.cuda.synchronize()
    status = int(ws[:4].view(torch.int32).item())
    print(f"{case.name}: {args.steps} calls, {api.mla_router_launches(T, H, E, K)} kernels per call, "
          f"device status {status:#x}")
    return 0 if status == 0 else 1


def _fp8_weight(experts_n, n, k, dev):
    from . import experts
    w = torch.empty((experts_n, n, k), dtype=experts.E4M3, device=dev)
    for e in range(experts_n):
        w[e] = (torch.randn(n, k, device=dev) * 100).clamp(-448, 448).to(experts.E4M3)
    return w, torch.full((experts_n, experts.scale_blocks(n), experts.scale_blocks(k)), 0.01 / k ** 0.5, device=dev)


def _experts(args) -> int:
    from .device import ExpertLayer
    dev = torch.device("cuda:0")
    T, H, width, held, n_experts, K = args.experts, 7168, 2048, 32, 256, 8
    torch.manual_seed(7300)
    x = torch.randn(T, H, device=dev).to(torch.bfloat16)
    router = (torch.randn(H, n_experts, device=dev) / H ** 0.5).to(torch.bfloat16)
    layer = ExpertLayer(T, torch.ones(H, dtype=torch.bfloat16, device=dev), router, *_fp8_weight(held, 2 * width, H, dev),
                        *_fp8_weight(held, H, width, dev), K, first_expert=32)
    for _ in range(args.steps):
        layer.run(x)
    torch.cuda.synchronize()
    status = layer.device_status()
    print(f"experts, {T} tokens: {args.steps} steps, {int(layer.expert_offsets[-1])} rows here, device status {status:#x}")
    return 0 if status == 0 else 1


def _fp8_matmul(args) -> int:
    from . import experts
    dev = torch.device("cuda:0")
    M, N, K = args.fp8_matmul
    torch.manual_seed(7400)
    x = (torch.randn(M, K, device=dev) * 100).clamp(-448, 448).to(experts.E4M3)
    xs = torch.full((experts.scale_blocks(K), M), 0.01, device=dev)
    w, ws = _fp8_weight(1, N, K, dev)
    out = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    for _ in range(args.steps):
        experts.mla_fp8_matmul(x, xs, w[0], ws[0], out, status)
    torch.cuda.synchronize()
    print(f"8-bit product {M} x {N} x {K}: {args.steps} calls, device status {int(status):#x}")
    return 0 if int(status) == 0 else 1


def _tp_o_proj(args) -> int:
    from . import api, tp
    from .device import _to_torch
    dev = torch.device("cuda:0")
    T, K, H = 128, 16384, 7168
    x = synth.make_o_proj_inputs(T, K, H, seed=7200)
    o, w = _to_torch(x["o"], True).to(dev), _to_torch(x["o_proj_w"], True).to(dev)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    pb = tp.PeerBuffers.local(args.tp_world, T, H, device=dev)
    for e in range(1, args.steps + 1):
        api.mla_tp_o_proj_allreduce(o, w, pb.table(0, e), args.tp_world, ws, None)
    torch.cuda.synchronize()
    status = int(ws[:4].view(torch.int32).item())
    print(f"head-split o-projection, world {args.tp_world}: {args.steps} calls, device status {status:#x}")
    return 0 if status == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
