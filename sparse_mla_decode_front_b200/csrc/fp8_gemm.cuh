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

// The tiles of all groups: group g has rows [bound[g], bound[g + 1]) and tiles
// [start[g], start[g + 1]). The bounds are the offsets clamped to the rows there are and to
// their running maximum, so a wrong table still gives disjoint groups.
struct Groups {
    int bound[kMaxGroups + 1];
    int start[kMaxGroups + 1];
};
struct Tile {
    int g, row0, rows_left, f0;   // rows_left: rows of the group from row0 on
};

// All threads of the block; ends with a barrier. rows_per_tile rows x f_tiles feature tiles.
__device__ __forceinline__ void build_groups(Groups& G, const Problem& p, int rows_per_tile, int f_tiles) {
    for (int g = threadIdx.x; g <= p.groups; g += blockDim.x)
        G.bound[g] = p.offsets ? min(max(p.offsets[g], 0), p.rows) : g * p.rows;   // without offsets: one group
    __syncthreads();
    if (threadIdx.x < 32) {   // one warp, 32 groups at a time
        const int lane = threadIdx.x;
        int tiles_before = 0, high = 0;   // of the groups before these 32: tiles, largest bound
        for (int g0 = 0; g0 <= p.groups; g0 += 32) {
            const int g = g0 + lane;
            int b = g <= p.groups ? G.bound[g] : 0;
            b = max(b, high);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, b, o);
                if (lane >= o) b = max(b, u);
            }
            // the tiles of group g - 1, which ends at this bound
            int prev = __shfl_up_sync(0xffffffffu, b, 1);
            if (lane == 0) prev = g0 > 0 ? high : b;
            int s = (b - prev + rows_per_tile - 1) / rows_per_tile * f_tiles;
            high = __shfl_sync(0xffffffffu, b, 31);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += u;
            }
            if (g <= p.groups) {
                G.bound[g] = b;
                G.start[g] = tiles_before + s;
            }
            tiles_before += __shfl_sync(0xffffffffu, s, 31);
        }
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
    const int l = t - G.start[lo], rows = G.bound[lo + 1] - G.bound[lo];
    const int row_tiles = (rows + rows_per_tile - 1) / rows_per_tile;
    const int rt = l % row_tiles, ft = l / row_tiles;
    return Tile{lo, G.bound[lo] + rt * rows_per_tile, rows - rt * rows_per_tile, ft * bf};
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
                    ptx::tmem_wait_ld16(d);
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

// ------------------------------------------------------------------ many rows per group
// k_fp8_many: M = 128 rows x N = bn features (a multiple of 32, 64 .. 256, chosen by the host to
// fill the last wave), the rows as the UMMA's A operand. TMEM lane = row, so an epilogue thread
// needs one scale product per block (two where its columns straddle a 128-feature boundary)
// instead of one per column, and 256-wide tiles let each operand byte in shared memory feed
// enough tensor work. Eight drain warps: two per lane quarter, each with half of the columns and
// its fp32 sums in registers (setmaxnreg moves the other warps' registers to them); two TMEM
// accumulators of 256 columns.
constexpr int kManyThreads = 384;
constexpr int kManyRows = 128;
constexpr int kManyMaxBn = 256;
constexpr int kManyABytes = kManyRows * BK;
constexpr int kManyStageBytes = kManyABytes + kManyMaxBn * BK;
constexpr int kManyStages = 4;
constexpr int kManyEpiBuf = 32 * 64;    // per drain warp: 32 rows x 64 bytes
constexpr int kManySmem = kManyStages * kManyStageBytes + 8 * kManyEpiBuf + 1024;

__device__ __forceinline__ void fma_f32x2(uint64_t& acc, uint32_t d0, uint32_t d1, uint64_t s) {
    asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %0;\n\t}" : "+l"(acc) : "r"(d0), "r"(d1), "l"(s));
}
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

__global__ void __launch_bounds__(kManyThreads, 1)
k_fp8_many(const __grid_constant__ CUtensorMap tma_x, const __grid_constant__ CUtensorMap tma_w, Problem p, int bn) {
    constexpr int S = kManyStages;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[S], empty_bar[S], acc_full[2], acc_empty[2], mma_done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ Groups G;
    griddep_launch();
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            ptx::mbar_init(&full_bar[i], 1);
            ptx::mbar_init(&empty_bar[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&acc_full[i], 1);
            ptx::mbar_init(&acc_empty[i], 8);
        }
        ptx::mbar_init(&mma_done, 1);
        abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_desc(&tma_x);
        ptx::tma_prefetch_desc(&tma_w);
    }
    if (warp == 2) {
        ptx::tmem_alloc(&tmem_slot, 512);
        ptx::tmem_relinquish();
    }
    griddep_wait();
    build_groups(G, p, kManyRows, (p.n + bn - 1) / bn);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int tiles = G.start[p.groups];

    if (warp < 4) {
        // 128 x 72 + 256 x 216 registers = 384 x 168, what the block was launched with
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0 && lane == 0) {
            // ---------------- TMA
            const uint32_t bytes = kManyABytes + bn * BK;
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
                const Tile tl = tile_at(G, p.groups, t, kManyRows, bn);
                for (int kb = 0; kb < p.kb; ++kb) {
                    if (!ptx::mbar_wait(&empty_bar[stage], phase ^ 1, p.status)) { abort_flag = 1; goto loads_done; }
                    if (*(volatile int*)&abort_flag) goto loads_done;
                    unsigned char* x_s = smem + stage * kManyStageBytes;
                    ptx::mbar_arrive_expect_tx(&full_bar[stage], bytes);
                    ptx::tma_load_2d(x_s, &tma_x, &full_bar[stage], kb * BK, tl.row0);
                    ptx::tma_load_2d(x_s + kManyABytes, &tma_w, &full_bar[stage], kb * BK, tl.g * p.n + tl.f0);
                    ++issued;
                    if (++stage == S) { stage = 0; phase ^= 1; }
                }
            }
        loads_done:
            for (int i = 0; i < S && i < issued; ++i) {   // every load lands before shared memory is released
                if (--stage < 0) { stage = S - 1; phase ^= 1; }
                ptx::mbar_wait(&full_bar[stage], phase, p.status);
            }
        } else if (warp == 1 && lane == 0) {
            // ---------------- UMMA
            const uint32_t idesc = idesc_e4m3(kManyRows, bn);
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
                    const uint32_t x_addr = ptx::smem_u32(smem + stage * kManyStageBytes);
                    const uint64_t xd = ptx::sdesc_sw128(x_addr, 16, 1024);
                    const uint64_t wd = ptx::sdesc_sw128(x_addr + kManyABytes, 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < BK / 32; ++kk)   // K = 32 further: 32 bytes, 2 in the descriptor's units
                        umma_e4m3(tmem + buf * 256, xd + 2 * kk, wd + 2 * kk, idesc, kk > 0 ? 1u : 0u);
                    ptx::umma_commit(&empty_bar[stage]);
                    ptx::umma_commit(&acc_full[buf]);
                    if (++stage == S) { stage = 0; phase ^= 1; }
                    buf ^= 1;
                    if (buf == 0) buf_phase ^= 1;
                }
            }
            ptx::umma_commit(&mma_done);
            ptx::mbar_wait(&mma_done, 0, p.status);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ---------------- drain: thread = row of TMEM lane quarter warp & 3, columns [c0, c0 + bn / 2)
        const int quarter = warp & 3, half = bn >> 1, c0 = ((warp - 4) >> 2) * half, chunks = half >> 4;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16) + c0;
        unsigned char* ebuf = smem + S * kManyStageBytes + (warp - 4) * kManyEpiBuf;
        int buf = 0;
        uint32_t buf_phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const Tile tl = tile_at(G, p.groups, t, kManyRows, bn);
            // columns of chunk c belong to scale block b0 while c < cut, to b0 + 1 from there on
            const int f = tl.f0 + c0, b0 = f >> 7, cut = (128 - (f & 127)) >> 4;
            const float* ws0 = p.ws + ((size_t)tl.g * p.nb + min(b0, p.nb - 1)) * p.kb;
            const float* ws1 = p.ws + ((size_t)tl.g * p.nb + min(b0 + 1, p.nb - 1)) * p.kb;
            const int r = quarter * 32 + lane;
            const float* xs = p.xs + tl.row0 + min(r, tl.rows_left - 1);
            uint64_t acc[8][8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[c][i] = 0;
            // scales of the next two blocks, loaded two blocks ahead
            float nx[2], n0[2], n1[2];
            auto fetch = [&](int kb) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int b = min(kb + j, p.kb - 1);
                    nx[j] = xs[(size_t)b * p.rows];
                    n0[j] = ws0[b];
                    n1[j] = ws1[b];
                }
            };
            fetch(0);
            for (int kb2 = 0; ok && kb2 < p.kb; kb2 += 2) {
                const float sa[2] = {nx[0] * n0[0], nx[1] * n0[1]}, sb[2] = {nx[0] * n1[0], nx[1] * n1[1]};
                fetch(kb2 + 2);
#pragma unroll 1
                for (int j = 0; j < 2 && kb2 + j < p.kb; ++j) {
                    const uint64_t lo = j == 0 ? pack_f32x2(sa[0], sa[0]) : pack_f32x2(sa[1], sa[1]);
                    const uint64_t hi = j == 0 ? pack_f32x2(sb[0], sb[0]) : pack_f32x2(sb[1], sb[1]);
                    if (!ptx::mbar_wait(&acc_full[buf], buf_phase, p.status)) {
                        abort_flag = 1;
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    uint32_t d[2][16];
                    ptx::tmem_ld16_nowait(t_lane + buf * 256, d[0]);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        if (c >= chunks) break;
                        ptx::tmem_wait_ld16(d[c & 1]);
                        if (c + 1 < chunks && c + 1 < 8)
                            ptx::tmem_ld16_nowait(t_lane + buf * 256 + 16 * (c + 1), d[(c + 1) & 1]);
                        const uint64_t s = c < cut ? lo : hi;
#pragma unroll
                        for (int i = 0; i < 8; ++i) fma_f32x2(acc[c][i], d[c & 1][2 * i], d[c & 1][2 * i + 1], s);
                    }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&acc_empty[buf]);
                    buf ^= 1;
                    if (buf == 0) buf_phase ^= 1;
                }
            }
            if (!ok) break;
            // Out through shared memory, 64 bytes a row at a time (32 16-bit or 16 fp32 columns):
            // 16-byte pieces, swizzled by the row so that neither side has bank conflicts; four
            // lanes store one row's piece of a line.
            const int rows = min(32, tl.rows_left - quarter * 32);   // this warp's rows (<= 0: none)
            auto store_rows = [&](int col, int cols, int esize) {
                __syncwarp();
                const int piece = lane & 3, pc = col + piece * 16 / esize;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rr = 8 * i + (lane >> 2);
                    if (rr < rows && pc < col + cols && f + pc < p.n)
                        *reinterpret_cast<uint4*>(static_cast<unsigned char*>(p.out) +
                                                  ((size_t)(tl.row0 + quarter * 32 + rr) * p.n + f + pc) * esize) =
                            *reinterpret_cast<const uint4*>(ebuf + rr * 64 + ((piece ^ ((rr >> 1) & 3)) << 4));
                }
                __syncwarp();
            };
            auto piece_at = [&](int piece) {
                return reinterpret_cast<uint4*>(ebuf + lane * 64 + ((piece ^ ((lane >> 1) & 3)) << 4));
            };
            if (p.dtype == kDtypeFp32) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (c >= chunks) break;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 a = unpack_f32x2(acc[c][2 * q]), b = unpack_f32x2(acc[c][2 * q + 1]);
                        *piece_at(q) = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                                                  __float_as_uint(b.y));
                    }
                    store_rows(16 * c, 16, 4);
                }
            } else {
                const bool to_bf16 = p.dtype == kDtypeBf16;
#pragma unroll
                for (int c = 0; c < 8; c += 2) {
                    if (c >= chunks) break;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 a = unpack_f32x2(acc[c + (q >> 1)][4 * (q & 1) + i]);
                            if (to_bf16) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
                                o[i] = *reinterpret_cast<const uint32_t*>(&h);
                            } else {
                                const __half2 h = __floats2half2_rn(a.x, a.y);
                                o[i] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                        }
                        *piece_at(q) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    store_rows(16 * c, min(32, half - 16 * c), 2);
                }
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

}  // namespace fp8
}  // namespace mla
