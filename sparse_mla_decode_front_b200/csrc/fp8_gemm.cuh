// Block-scaled 8-bit matrix product (include/moe_experts.h: mla_fp8_matmul and
// mla_fp8_grouped_matmul), sm_100a.
//
// out[m, n] = sum_b x_scales[b, m] w_scales[n / 128, b] P_b[m, n], P_b the product of block
// b's 128-deep slices. The scales change with every block, so the tensor cores cannot add
// over blocks: each block's P_b is one short accumulation in TMEM (four K = 32 UMMAs into a
// fresh accumulator), read back by the epilogue warps and added, scaled, in fp32 registers.
// Several accumulators let the UMMAs of the next blocks run while a block is drained.
//
// Groups: expert e's rows are [offsets[e], offsets[e + 1]) of x, its weight is rows
// [e N, (e + 1) N) of w. Every CTA turns the offsets into the tiles before each expert (a
// prefix sum in shared memory) and takes tiles blockIdx.x, + gridDim.x, ...; a tile's rows
// may reach into the next expert's (TMA has no row alignment) and are not stored there. The
// plain product is one group over all rows.
//
// k_fp8_few: few rows per group, where the weights' bytes bound the product: the weight tile
// is the UMMA's A operand (M = 128 features), the rows its B operand (N = BN rows), so a
// group of few rows costs few tensor cycles, and TMEM lane = feature, column = row.
// Warp 0 issues TMA, warp 1 UMMA, warp 2 brings the scales x_scales * w_scales of each block
// into shared memory (every epilogue thread needs all of them), warps 3-6 drain.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace mla {
namespace fp8 {

constexpr int BF = 128;          // features per tile = UMMA M
constexpr int BK = 128;          // K block = scale block = one 128-byte swizzle atom
constexpr int kBufs = 4;         // accumulators in TMEM
constexpr int kMaxGroups = 1024;
constexpr int kFewThreads = 224;

struct Problem {
    const float *xs, *ws;        // x_scales [kb][rows], w_scales [groups][nb][kb]
    const int32_t* offsets;      // [groups + 1], or null: one group of all rows
    int rows, groups, n, k, nb, kb;
    void* out;
    int dtype;
    int32_t* status;
};

// Instruction descriptor, kind::f8f6f4: e4m3 A and B (both K-major), fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The tiles of all groups. start[g] is the first tile of group g, row[g] its first row (both
// with a last entry behind the last group).
struct Groups {
    int start[kMaxGroups + 1];
    int first[kMaxGroups];
    int rows[kMaxGroups];
};
struct Tile {
    int g, row0, rows_left, f0;   // rows_left: rows of the group from row0 on
};

// All threads of the block; ends with a barrier. rows_per_tile x features_per_tile tiles.
__device__ __forceinline__ void build_groups(Groups& G, const Problem& p, int rows_per_tile, int f_tiles) {
    for (int g = threadIdx.x; g < p.groups; g += blockDim.x) {
        int a = 0, b = p.rows;
        if (p.offsets) {
            a = min(max(p.offsets[g], 0), p.rows);
            b = min(max(p.offsets[g + 1], a), p.rows);
        }
        G.first[g] = a;
        G.rows[g] = b - a;
    }
    __syncthreads();
    // One warp, 32 groups at a time. The rows are summed first: groups of a wrong table that
    // overlap are cut where their sum passes the rows there are, so the tiles stay countable.
    if (threadIdx.x < 32) {
        int carry = 0;
        long long rows_before = 0;
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
            const int g = g0 + threadIdx.x;
            int rows = g < p.groups ? G.rows[g] : 0;
            long long sum = rows;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, sum, o);
                if ((int)threadIdx.x >= o) sum += u;
            }
            rows = (int)min((long long)rows, max(0LL, p.rows - (rows_before + sum - rows)));
            rows_before += __shfl_sync(0xffffffffu, sum, 31);
            const int tiles = (rows + rows_per_tile - 1) / rows_per_tile * f_tiles;
            int s = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, s, o);
                if ((int)threadIdx.x >= o) s += u;
            }
            if (g < p.groups) {
                G.rows[g] = rows;
                G.start[g] = carry + s - tiles;
            }
            carry += __shfl_sync(0xffffffffu, s, 31);
        }
        if (threadIdx.x == 0) G.start[p.groups] = carry;
    }
    __syncthreads();
}

// Tile `t` (< start[groups]): its group by bisection, row tiles fastest, so that the CTAs
// which run together share a weight tile.
__device__ __forceinline__ Tile tile_at(const Groups& G, int groups, int t, int rows_per_tile, int bf) {
    int lo = 0, hi = groups;      // start[lo] <= t < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (G.start[mid] <= t) lo = mid; else hi = mid;
    }
    const int l = t - G.start[lo];
    const int row_tiles = (G.rows[lo] + rows_per_tile - 1) / rows_per_tile;
    const int rt = l % row_tiles, ft = l / row_tiles;
    return Tile{lo, G.first[lo] + rt * rows_per_tile, G.rows[lo] - rt * rows_per_tile, ft * bf};
}

template <int BN>
struct FewCfg {
    static constexpr int kWBytes = BF * BK, kXBytes = BN * BK;
    static constexpr int kStageBytes = kWBytes + kXBytes;
    static constexpr int kStages = 196608 / kStageBytes < 12 ? 196608 / kStageBytes : 12;
    static constexpr int kEpiBuf = 16 * 32 * 4;                       // per epilogue warp: [16 rows][32 features]
    static constexpr int kSmem = kStages * kStageBytes + 4 * kEpiBuf + 1024;
    static constexpr uint32_t kTmemCols = kBufs * BN;                 // 64 .. 512
};

template <int BN>
__global__ void __launch_bounds__(kFewThreads, 1)
k_fp8_few(const __grid_constant__ CUtensorMap tma_w, const __grid_constant__ CUtensorMap tma_x, Problem p) {
    using C = FewCfg<BN>;
    constexpr int S = C::kStages;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[S], empty_bar[S], acc_full[kBufs], acc_empty[kBufs], sc_full[kBufs],
        mma_done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ Groups G;
    __shared__ __align__(16) float scale[kBufs][BN];
    griddep_launch();
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            ptx::mbar_init(&full_bar[i], 1);
            ptx::mbar_init(&empty_bar[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            ptx::mbar_init(&acc_full[i], 1);
            ptx::mbar_init(&acc_empty[i], 4);
            ptx::mbar_init(&sc_full[i], 32);
        }
        ptx::mbar_init(&mma_done, 1);
        abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_desc(&tma_w);
        ptx::tma_prefetch_desc(&tma_x);
    }
    if (warp == 2) {
        ptx::tmem_alloc(&tmem_slot, C::kTmemCols);
        ptx::tmem_relinquish();
    }
    griddep_wait();
    build_groups(G, p, BN, (p.n + BF - 1) / BF);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int tiles = G.start[p.groups];

    if (warp == 0 && lane == 0) {
        // ---------------- TMA
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
            const Tile tl = tile_at(G, p.groups, t, BN, BF);
            for (int kb = 0; kb < p.kb; ++kb) {
                if (!ptx::mbar_wait(&empty_bar[stage], phase ^ 1, p.status)) { abort_flag = 1; goto loads_done; }
                if (*(volatile int*)&abort_flag) goto loads_done;
                unsigned char* w_s = smem + stage * C::kStageBytes;
                ptx::mbar_arrive_expect_tx(&full_bar[stage], C::kStageBytes);
                ptx::tma_load_2d(w_s, &tma_w, &full_bar[stage], kb * BK, tl.g * p.n + tl.f0);
                ptx::tma_load_2d(w_s + C::kWBytes, &tma_x, &full_bar[stage], kb * BK, tl.row0);
                ++issued;
                if (++stage == S) { stage = 0; phase ^= 1; }
            }
        }
    loads_done:
        // every load lands before the CTA's shared memory is released
        for (int i = 0; i < S && i < issued; ++i) {
            if (--stage < 0) { stage = S - 1; phase ^= 1; }
            ptx::mbar_wait(&full_bar[stage], phase, p.status);
        }
    } else if (warp == 1 && lane == 0) {
        // ---------------- UMMA
        constexpr uint32_t idesc = idesc_e4m3(BF, BN);
        int stage = 0, buf = 0;
        uint32_t phase = 0, buf_phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            for (int kb = 0; kb < p.kb; ++kb) {
                if (!ptx::mbar_wait(&acc_empty[buf], buf_phase ^ 1, p.status) ||
                    !ptx::mbar_wait(&full_bar[stage], phase, p.status)) {
                    abort_flag = 1;
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t w_addr = ptx::smem_u32(smem + stage * C::kStageBytes);
                const uint32_t x_addr = w_addr + C::kWBytes;
                // past K both operands are zero-filled, so a partial last block needs no other form
#pragma unroll
                for (int kk = 0; kk < BK / 32; ++kk)
                    umma_e4m3(tmem + buf * BN, ptx::sdesc_sw128(w_addr + kk * 32, 16, 1024),
                              ptx::sdesc_sw128(x_addr + kk * 32, 16, 1024), idesc, kk > 0 ? 1u : 0u);
                ptx::umma_commit(&empty_bar[stage]);
                ptx::umma_commit(&acc_full[buf]);
                if (++stage == S) { stage = 0; phase ^= 1; }
                if (++buf == kBufs) { buf = 0; buf_phase ^= 1; }
            }
        }
        ptx::umma_commit(&mma_done);   // all UMMAs complete before TMEM is released
        ptx::mbar_wait(&mma_done, 0, p.status);
    } else if (warp == 2) {
        // ---------------- scales
        constexpr int kPer = (BN + 31) / 32;
        int buf = 0;
        uint32_t buf_phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const Tile tl = tile_at(G, p.groups, t, BN, BF);
            const float* ws = p.ws + ((size_t)tl.g * p.nb + tl.f0 / BF) * p.kb;
            float v[kPer], w;
            auto load = [&](int kb) {
                w = ws[kb];
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int c = lane + 32 * i;
                    v[i] = c < tl.rows_left && c < BN ? p.xs[(size_t)kb * p.rows + tl.row0 + c] : 0.f;
                }
            };
            load(0);
            for (int kb = 0; kb < p.kb; ++kb) {
                if (!ptx::mbar_wait(&acc_empty[buf], buf_phase ^ 1, p.status)) { abort_flag = 1; ok = false; break; }
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (lane + 32 * i < BN) scale[buf][lane + 32 * i] = v[i] * w;   // one fp32 rounding
                ptx::mbar_arrive(&sc_full[buf]);
                if (kb + 1 < p.kb) load(kb + 1);
                if (++buf == kBufs) { buf = 0; buf_phase ^= 1; }
            }
        }
    } else if (warp >= 3) {
        // ---------------- drain: thread = feature of TMEM lane quarter warp & 3
        const int quarter = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        float* ebuf = reinterpret_cast<float*>(smem + S * C::kStageBytes + (warp - 3) * C::kEpiBuf);
        int buf = 0;
        uint32_t buf_phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const Tile tl = tile_at(G, p.groups, t, BN, BF);
            float acc[BN];
#pragma unroll
            for (int c = 0; c < BN; ++c) acc[c] = 0.f;
            for (int kb = 0; kb < p.kb; ++kb) {
                if (!ptx::mbar_wait(&acc_full[buf], buf_phase, p.status) ||
                    !ptx::mbar_wait(&sc_full[buf], buf_phase, p.status)) {
                    abort_flag = 1;
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
#pragma unroll
                for (int c0 = 0; c0 < BN; c0 += 16) {
                    uint32_t d[16];
                    ptx::tmem_ld16_nowait(t_lane + buf * BN + c0, d);
                    ptx::tmem_wait_ld();
                    const float4* s4 = reinterpret_cast<const float4*>(&scale[buf][c0]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 s = s4[j];
                        acc[c0 + 4 * j] = fmaf(__uint_as_float(d[4 * j]), s.x, acc[c0 + 4 * j]);
                        acc[c0 + 4 * j + 1] = fmaf(__uint_as_float(d[4 * j + 1]), s.y, acc[c0 + 4 * j + 1]);
                        acc[c0 + 4 * j + 2] = fmaf(__uint_as_float(d[4 * j + 2]), s.z, acc[c0 + 4 * j + 2]);
                        acc[c0 + 4 * j + 3] = fmaf(__uint_as_float(d[4 * j + 3]), s.w, acc[c0 + 4 * j + 3]);
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&acc_empty[buf]);
                if (++buf == kBufs) { buf = 0; buf_phase ^= 1; }
            }
            if (!ok) break;
            // 16 rows at a time through shared memory: a row's 32 features are stored side by side
            const int f = tl.f0 + quarter * 32;
#pragma unroll
            for (int c0 = 0; c0 < BN; c0 += 16) {
                if (c0 >= tl.rows_left) break;
#pragma unroll
                for (int i = 0; i < 16; ++i) ebuf[i * 32 + lane] = acc[c0 + i];
                __syncwarp();
                if (p.dtype == kDtypeFp32) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int v = lane + 32 * i, c = v >> 3, m = f + 4 * (v & 7);
                        if (c0 + c < tl.rows_left && m < p.n)
                            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + (size_t)(tl.row0 + c0 + c) * p.n + m) =
                                *reinterpret_cast<const float4*>(ebuf + c * 32 + 4 * (v & 7));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int v = lane + 32 * i, c = v >> 2, m = f + 8 * (v & 3);
                        if (c0 + c >= tl.rows_left || m >= p.n) continue;
                        const float* e = ebuf + c * 32 + 8 * (v & 3);
                        uint4 o;
                        if (p.dtype == kDtypeBf16) {
                            __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
                            for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(e[2 * j], e[2 * j + 1]);
                        } else {
                            __half2* h = reinterpret_cast<__half2*>(&o);
#pragma unroll
                            for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(e[2 * j], e[2 * j + 1]);
                        }
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (size_t)(tl.row0 + c0 + c) * p.n + m) = o;
                    }
                }
                __syncwarp();
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::kTmemCols);
    }
}

}  // namespace fp8
}  // namespace mla
