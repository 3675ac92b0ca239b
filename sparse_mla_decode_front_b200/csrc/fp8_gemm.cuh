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
// Warp 0 issues TMA, warps 1 and 7 UMMA, warp 2 brings the scales x_scales * w_scales of each
// block into shared memory (every drain thread needs all of them), warps 3-6 drain. Where the
// tiles are few, a cluster of `split` CTAs takes one tile, each a run of its K blocks; the
// partial sums meet in distributed shared memory and are added in the order of the ranks.
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
constexpr int kFewThreads = 256;
constexpr int kScales = 8;        // K blocks whose scales are handed over at once
constexpr int kFewIssuer2 = 7;    // warp of the second issuer

struct Problem {
    const float *xs, *ws;        // x_scales [kb][rows], w_scales [groups][nb][kb]
    const int32_t* offsets;      // [groups + 1], or null: one group of all rows
    int rows, groups, n, k, nb, kb;
    void* out;
    int dtype;
    int32_t* status;
    int split_log2;              // k_fp8_few: 2^split_log2 CTAs (a cluster) share a tile's K blocks
};

// Instruction descriptor, kind::f8f6f4: e4m3 A and B (both K-major), fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// PAIR: issued by the leader of a CTA pair, for both.
template <bool PAIR = false>
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
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
    if (!p.offsets) {   // one group
        if (threadIdx.x == 0) {
            G.bound[0] = G.start[0] = 0;
            G.bound[1] = p.rows;
            G.start[1] = (p.rows + rows_per_tile - 1) / rows_per_tile * f_tiles;
        }
        __syncthreads();
        return;
    }
    for (int g = threadIdx.x; g <= p.groups; g += blockDim.x) G.bound[g] = min(max(p.offsets[g], 0), p.rows);
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

// Tiles t0, t0 + step, ... below `tiles`.
__device__ __forceinline__ int my_tiles(int tiles, int t0, int step) {
    return t0 < tiles ? (tiles - 1 - t0) / step + 1 : 0;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// The UMMAs of every second K block, from block `first` on, of `tiles` tiles of `kb` blocks.
// One thread needs about 870 clocks a block (two waits of about 120, four UMMAs, two commits
// of about 75, each of which it sits out; measured on a 128 x 256 tile), more than the 512
// that the tensor cores need. The blocks' accumulators are independent, so two threads of
// different warps take turns: 1.4 to 2 times the rate. idesc_of(i): the instruction
// descriptor of tile i; issue(idesc, stage, buf): one block's UMMAs; commit(bar). Past K both
// operands are zero-filled, so a partial last block has no other form.
template <int S, int BUFS, class D, class F, class C>
__device__ __forceinline__ bool issue_blocks(int first, int tiles, int kb, uint64_t* full_bar, uint64_t* empty_bar,
                                             uint64_t* acc_full, uint64_t* acc_empty, int32_t* status, D idesc_of,
                                             F issue, C commit) {
    static_assert(S >= 2 && BUFS % 2 == 0, "each issuer has its own accumulators");
    int stage = first, buf = first;
    uint32_t phase = 0, buf_phase = 0;
    int next = first;   // block of the tile
    for (int i = 0; i < tiles; ++i) {
        const uint32_t idesc = idesc_of(i);
        for (; next < kb; next += 2) {
            if (!ptx::mbar_wait_spin(&full_bar[stage], phase, status) ||
                !ptx::mbar_wait_spin(&acc_empty[buf], buf_phase ^ 1, status))
                return false;
            ptx::tc_fence_after();
            issue(idesc, stage, buf);
            commit(&acc_full[buf]);
            commit(&empty_bar[stage]);
            stage += 2;
            if (stage >= S) { stage -= S; phase ^= 1; }
            buf += 2;
            if (buf >= BUFS) { buf -= BUFS; buf_phase ^= 1; }
        }
        next -= kb;
    }
    return true;
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
    __shared__ __align__(8) uint64_t full_bar[S], empty_bar[S], acc_full[kBufs], acc_empty[kBufs], sc_full[2],
        sc_empty[2], mma_done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ Groups G;
    __shared__ __align__(16) float scale[2][kScales][BN];
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
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sc_full[i], 32);
            ptx::mbar_init(&sc_empty[i], 4);
        }
        ptx::mbar_init(&mma_done, 2);
        abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_desc(&tma_w);
        ptx::tma_prefetch_desc(&tma_x);
    }
    griddep_wait();
    build_groups(G, p, BN, (p.n + BF - 1) / BF);
    uint32_t tmem = 0;
    if (warp > 0) {   // the first loads are issued while TMEM is allocated
        if (warp == 2) {
            ptx::tmem_alloc(&tmem_slot, C::kTmemCols);
            ptx::tmem_relinquish();
        }
        ptx::tc_fence_before();
        ptx::bar_sync_named(1, kFewThreads - 32);
        ptx::tc_fence_after();
        tmem = tmem_slot;
    }
    const int tiles = G.start[p.groups];
    const int split = 1 << p.split_log2, rank = split > 1 ? (int)ptx::cluster_ctarank() : 0;
    const int t0 = blockIdx.x >> p.split_log2, t_step = gridDim.x >> p.split_log2;   // with a split: one tile at most
    const int kb0 = (p.kb * rank) >> p.split_log2, kb1 = (p.kb * (rank + 1)) >> p.split_log2;

    if (warp == 0 && lane == 0) {
        // ---------------- TMA
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        for (int t = t0; t < tiles; t += t_step) {
            const Tile tl = tile_at(G, p.groups, t, BN, BF);
            for (int kb = kb0; kb < kb1; ++kb) {
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
    } else if ((warp == 1 || warp == kFewIssuer2) && lane == 0) {
        // ---------------- UMMA, two issuers (see issue_blocks)
        constexpr uint32_t idesc = idesc_e4m3(BF, BN);
        const bool ok = issue_blocks<S, kBufs>(
            warp == 1 ? 0 : 1, my_tiles(tiles, t0, t_step), kb1 - kb0, full_bar, empty_bar, acc_full, acc_empty, p.status,
            [&](int) { return idesc; },
            [&](uint32_t, int stage, int buf) {
                const uint32_t w_addr = ptx::smem_u32(smem + stage * C::kStageBytes);
                const uint64_t wd = ptx::sdesc_sw128(w_addr, 16, 1024);
                const uint64_t xd = ptx::sdesc_sw128(w_addr + C::kWBytes, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < BK / 32; ++kk)   // K = 32 further: 32 bytes, 2 in the descriptor's units
                    umma_e4m3(tmem + buf * BN, wd + 2 * kk, xd + 2 * kk, idesc, kk > 0 ? 1u : 0u);
            },
            [](uint64_t* bar) { ptx::umma_commit(bar); });
        if (!ok) abort_flag = 1;
        ptx::umma_commit(&mma_done);   // all UMMAs complete before TMEM is released
        ptx::mbar_wait(&mma_done, 0, p.status);
    } else if (warp == 2) {
        // ---------------- scales: the products x_scales * w_scales of kScales blocks at a time, the
        // next batch's loads under way while the drain works on this one. (One block at a time,
        // the latency of its loads was the bound: 1100 clocks a block.)
        constexpr int kPer = (BN + 31) / 32;
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = t0; ok && t < tiles; t += t_step) {
            const Tile tl = tile_at(G, p.groups, t, BN, BF);
            const float* ws = p.ws + ((size_t)tl.g * p.nb + tl.f0 / BF) * p.kb;
            float v[kScales][kPer], w[kScales];
            auto load = [&](int k0) {
#pragma unroll
                for (int j = 0; j < kScales; ++j) {
                    const int kb = min(k0 + j, kb1 - 1);
                    w[j] = ws[kb];
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {   // rows behind the last: any scale, their sums are not stored
                        const int c = min(lane + 32 * i, tl.rows_left - 1);
                        v[j][i] = p.xs[(size_t)kb * p.rows + tl.row0 + c];
                    }
                }
            };
            load(kb0);
            for (int k0 = kb0; k0 < kb1; k0 += kScales) {
                if (!ptx::mbar_wait(&sc_empty[slot], phase ^ 1, p.status)) { abort_flag = 1; ok = false; break; }
#pragma unroll
                for (int j = 0; j < kScales; ++j)
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        if (lane + 32 * i < BN) scale[slot][j][lane + 32 * i] = v[j][i] * w[j];   // one fp32 rounding
                ptx::mbar_arrive(&sc_full[slot]);
                if (k0 + kScales < kb1) load(k0 + kScales);
                slot ^= 1;
                if (slot == 0) phase ^= 1;
            }
        }
    } else if (warp >= 3 && warp < 7) {
        // ---------------- drain: thread = feature of TMEM lane quarter warp & 3
        const int quarter = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        float* ebuf = reinterpret_cast<float*>(smem + S * C::kStageBytes + (warp - 3) * C::kEpiBuf);
        int buf = 0, slot = 0;
        uint32_t buf_phase = 0, sc_phase = 0;
        bool ok = true;
        for (int t = t0; ok && t < tiles; t += t_step) {
            const Tile tl = tile_at(G, p.groups, t, BN, BF);
            float acc[BN];
#pragma unroll
            for (int c = 0; c < BN; ++c) acc[c] = 0.f;
            for (int kb = kb0; kb < kb1; ++kb) {
                const int j = (kb - kb0) % kScales;
                if ((j == 0 && !ptx::mbar_wait(&sc_full[slot], sc_phase, p.status)) ||
                    !ptx::mbar_wait(&acc_full[buf], buf_phase, p.status)) {
                    abort_flag = 1;
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                // kGroup columns in flight; the accumulator is free once the last are in registers
                constexpr int kGroup = BN < 64 ? BN : 64;
#pragma unroll
                for (int g0 = 0; g0 < BN; g0 += kGroup) {
                    uint32_t d[kGroup / 16][16];
#pragma unroll
                    for (int c = 0; c < kGroup / 16; ++c) ptx::tmem_ld16_nowait(t_lane + buf * BN + g0 + 16 * c, d[c]);
#pragma unroll
                    for (int c = 0; c < kGroup / 16; ++c) ptx::tmem_wait_ld16(d[c]);
                    if (g0 + kGroup == BN) {
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&acc_empty[buf]);
                    }
#pragma unroll
                    for (int c = 0; c < kGroup / 16; ++c) {
                        const float4* s4 = reinterpret_cast<const float4*>(&scale[slot][j][g0 + 16 * c]);
                        float* a16 = acc + g0 + 16 * c;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 s = s4[i];
                            a16[4 * i] = fmaf(__uint_as_float(d[c][4 * i]), s.x, a16[4 * i]);
                            a16[4 * i + 1] = fmaf(__uint_as_float(d[c][4 * i + 1]), s.y, a16[4 * i + 1]);
                            a16[4 * i + 2] = fmaf(__uint_as_float(d[c][4 * i + 2]), s.z, a16[4 * i + 2]);
                            a16[4 * i + 3] = fmaf(__uint_as_float(d[c][4 * i + 3]), s.w, a16[4 * i + 3]);
                        }
                    }
                }
                if (j == kScales - 1 || kb == kb1 - 1) {   // the batch is read
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&sc_empty[slot]);
                    slot ^= 1;
                    if (slot == 0) sc_phase ^= 1;
                }
                if (++buf == kBufs) { buf = 0; buf_phase ^= 1; }
            }
            if (!ok) break;
            if (split > 1) {   // partial sums [row][feature] where the stages were: every load and UMMA is over
                float* part = reinterpret_cast<float*>(smem);
#pragma unroll
                for (int c = 0; c < BN; ++c) part[c * BF + quarter * 32 + lane] = acc[c];
                continue;
            }
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
    if (split > 1) {
        const Tile tl = t0 < tiles ? tile_at(G, p.groups, t0, BN, BF) : Tile{0, 0, 0, 0};
        const int f = threadIdx.x % BF;
        const uint32_t mine = ptx::smem_u32(smem) + 4 * f;
        ptx::cluster_sync_all();   // all ranks' partial sums are there
        for (int c = rank + split * (threadIdx.x / BF); c < min(BN, tl.rows_left); c += split * (kFewThreads / BF)) {
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                v[r] = r < split ? ld_cluster_f32(ptx::mapa_shared(mine, r) + 4 * c * BF) : 0.f;
            float sum = v[0];
#pragma unroll
            for (int r = 1; r < 8; ++r) sum += v[r];
            if (tl.f0 + f < p.n) {
                const size_t at = (size_t)(tl.row0 + c) * p.n + tl.f0 + f;
                if (p.dtype == kDtypeFp32) static_cast<float*>(p.out)[at] = sum;
                else if (p.dtype == kDtypeBf16) static_cast<bf16*>(p.out)[at] = __float2bfloat16_rn(sum);
                else static_cast<__half*>(p.out)[at] = __float2half_rn(sum);
            }
        }
        ptx::cluster_sync_all();   // no rank leaves while its sums are read
    }
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::kTmemCols);
    }
}

// ------------------------------------------------------------------ many rows per group
// k_fp8_many<PAIR>: tiles of 128 rows a CTA x 256 features, the rows as the UMMA's A operand.
// TMEM lane = row, so a drain thread needs one scale per block and not one per column; it holds
// the fp32 sums of 128 columns in registers (setmaxnreg moves the other warps' to it), and two
// accumulators of 256 columns take turns.
//
// PAIR: two CTAs share a tile of 256 rows (cta_group::2, M = 256: each holds 128 rows of x and
// half of the weight rows, and each one's tensor core reads both halves). A block then takes
// 32 KB of operands a CTA instead of 48, and an SM takes in about 64 bytes a clock from L2
// (390 ns a block measured for the single CTA with the drain left out). Measured in a loop (the
// 1000 W cap holds the clock at 1.54 GHz): 4096 x 7168 x 16384 530 - 550 us, 1.8 PFLOP/s, against 579 us
// for single CTAs. But a group's last tile is half empty on average, and of 128 rows that costs less
// than of 256: 8191 rows over 32 experts (3 to 2156 each), 4096 x 7168: 369 - 441 us single, 439 - 480
// us in pairs. Hence pairs for the plain product, single CTAs for groups.
//
// What bounds it: 0.52 us a block of a CTA (1.965 GHz) against 0.26 for the tensor cores alone.
// Loads, products and hand-overs without any drain take 0.44. The drain is a chain: a wait for
// the accumulator (about 75 clocks), TMEM reads of 32 columns overlapped with the additions of
// the 32 before (4 x 90), the hand-back; two warps a scheduler fill each other's gaps. Tried and
// slower: accumulators of 128 columns with four issuing threads (+24%), 16 drain warps of 64
// columns (+22%), packed fp32 pairs (+8%: moves), column counts that are not compile-time (+25%).
//
// Warps 0-3 (72 registers): 0 TMA, 1 and 2 UMMA (every second block each, see issue_blocks; of a
// pair the leader's only), 3 scales and TMEM. Warps 4-11 (216 registers): the drain, four warps
// to 128 columns.
constexpr int kManyThreads = 384;
constexpr int kManyRows = 128;                        // rows of a CTA
constexpr int kManyFeatures = 256;
constexpr int kManyDrain = 8;                         // drain warps
constexpr int kManyEpiBuf = 32 * 64;                  // per drain warp: 32 rows x 64 bytes
template <bool PAIR>
struct ManyCfg {
    static constexpr int kRows = PAIR ? 2 * kManyRows : kManyRows;               // of a tile
    static constexpr int kWRows = PAIR ? kManyFeatures / 2 : kManyFeatures;      // weight rows in a CTA
    static constexpr int kABytes = kManyRows * BK;
    static constexpr int kStageBytes = kABytes + kWRows * BK;
    static constexpr int kStages = PAIR ? 6 : 4;
    static constexpr int kSmem = kStages * kStageBytes + kManyDrain * kManyEpiBuf + 1024;
};

// 4-byte asynchronous copy, counted by cp.async.mbarrier.arrive.
__device__ __forceinline__ void cp_async_4(float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
// One CTA's load of a pair's stage: into its own shared memory, counted on the leader's barrier.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* m, uint32_t bar_cluster, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4}], [%2];" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster), "r"(x), "r"(y)
        : "memory");
}
// Arrive on a barrier of the pair (a shared::cluster address). What it orders are TMEM reads, which the
// tcgen05 fences on both sides cover, so the arrive itself is relaxed: a release (which
// publishes memory writes too) held the warp up, about 250 clocks at CTA and 1300 at cluster scope.
__device__ __forceinline__ void arrive_cluster(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
// Arrive on the barrier at this offset in both CTAs once this thread's earlier UMMAs have completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            ptx::smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// The same on this CTA's barrier alone.
__device__ __forceinline__ void umma_commit_leader(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(ptx::smem_u32(bar))
                 : "memory");
}
// One warp of each CTA of the pair.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

template <bool PAIR>   // PAIR: launched in clusters of two
__global__ void __launch_bounds__(kManyThreads, 1)
k_fp8_many(const __grid_constant__ CUtensorMap tma_x, const __grid_constant__ CUtensorMap tma_w, Problem p) {
    using C = ManyCfg<PAIR>;
    constexpr int S = C::kStages;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[S], empty_bar[S], acc_full[2], acc_empty[2], sc_full[2], sc_empty[2],
        mma_done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ Groups G;
    __shared__ float x_sc[2][kScales][kManyRows];
    __shared__ float w_sc[2][kScales][2];
    griddep_launch();
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)ptx::cluster_ctarank() : 0;
    const int t0 = PAIR ? (int)ptx::cluster_id_x() : blockIdx.x, t_step = PAIR ? (int)ptx::nclusters_x() : gridDim.x;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            ptx::mbar_init(&full_bar[i], 1);     // of a pair the leader's: its producer, and both CTAs' bytes
            ptx::mbar_init(&empty_bar[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&acc_full[i], 1);
            ptx::mbar_init(&acc_empty[i], (PAIR ? 2 : 1) * kManyDrain);   // of a pair the leader's
            ptx::mbar_init(&sc_full[i], 32);
            ptx::mbar_init(&sc_empty[i], kManyDrain);
        }
        ptx::mbar_init(&mma_done, 2);
        abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_desc(&tma_x);
        ptx::tma_prefetch_desc(&tma_w);
    }
    griddep_wait();
    build_groups(G, p, C::kRows, (p.n + kManyFeatures - 1) / kManyFeatures);
    if (warp == 3) {
        if (PAIR) {
            tmem_alloc_pair(&tmem_slot, 512);
        } else {
            ptx::tmem_alloc(&tmem_slot, 512);
            ptx::tmem_relinquish();
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (PAIR) ptx::cluster_sync_all();   // the peer's barriers are set up before anything arrives on them
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int tiles = G.start[p.groups];
    // Features of a tile, the UMMA's N: a multiple of 16, and of 32 in a pair, whose first half are the leader's
    // weight rows (of those behind the last feature, zeros, nothing is stored).
    auto width_of = [&](int f0) { return min(kManyFeatures, PAIR ? (p.n - f0 + 31) & ~31 : p.n - f0); };

    if (warp < 4) {
        // 128 x 72 + 256 x 216 registers = 384 x 168, what the block was launched with
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0 && lane == 0) {
            // ---------------- TMA: this CTA's rows of x and of the weight tile
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int t = t0; t < tiles; t += t_step) {
                const Tile tl = tile_at(G, p.groups, t, C::kRows, kManyFeatures);
                const int x_row = tl.row0 + rank * kManyRows;
                const int w_row = tl.g * p.n + tl.f0 + (PAIR ? rank * (width_of(tl.f0) / 2) : 0);
                for (int kb = 0; kb < p.kb; ++kb) {
                    if (!ptx::mbar_wait_spin(&empty_bar[stage], phase ^ 1, p.status)) { abort_flag = 1; goto loads_done; }
                    if (*(volatile int*)&abort_flag) goto loads_done;
                    unsigned char* x_s = smem + stage * C::kStageBytes;
                    if (PAIR) {
                        const uint32_t bar = ptx::mapa_shared(ptx::smem_u32(&full_bar[stage]), 0);
                        if (rank == 0) ptx::mbar_arrive_expect_tx(&full_bar[stage], 2 * C::kStageBytes);
                        tma_load_2d_pair(x_s, &tma_x, bar, kb * BK, x_row);
                        tma_load_2d_pair(x_s + C::kABytes, &tma_w, bar, kb * BK, w_row);
                    } else {
                        ptx::mbar_arrive_expect_tx(&full_bar[stage], C::kStageBytes);
                        ptx::tma_load_2d(x_s, &tma_x, &full_bar[stage], kb * BK, x_row);
                        ptx::tma_load_2d(x_s + C::kABytes, &tma_w, &full_bar[stage], kb * BK, w_row);
                    }
                    ++issued;
                    if (++stage == S) { stage = 0; phase ^= 1; }
                }
            }
        loads_done:
            if (rank == 0)   // every load lands before shared memory is released (a pair leaves together)
                for (int i = 0; i < S && i < issued; ++i) {
                    if (--stage < 0) { stage = S - 1; phase ^= 1; }
                    ptx::mbar_wait_spin(&full_bar[stage], phase, p.status);
                }
        } else if ((warp == 1 || warp == 2) && lane == 0 && rank == 0) {
            // ---------------- UMMA: every second K block each
            const int q = warp - 1;
            const bool ok = issue_blocks<S, 2>(
                q, my_tiles(tiles, t0, t_step), p.kb, full_bar, empty_bar, acc_full, acc_empty, p.status,
                [&](int i) {
                    const Tile tl = tile_at(G, p.groups, t0 + i * t_step, C::kRows, kManyFeatures);
                    return idesc_e4m3(C::kRows, width_of(tl.f0));
                },
                [&](uint32_t idesc, int stage, int buf) {
                    const uint32_t x_addr = ptx::smem_u32(smem + stage * C::kStageBytes);
                    const uint64_t xd = ptx::sdesc_sw128(x_addr, 16, 1024);
                    const uint64_t wd = ptx::sdesc_sw128(x_addr + C::kABytes, 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < BK / 32; ++kk)
                        umma_e4m3<PAIR>(tmem + buf * kManyFeatures, xd + 2 * kk, wd + 2 * kk, idesc, kk > 0 ? 1u : 0u);
                },
                [](uint64_t* bar) { PAIR ? umma_commit_pair(bar) : ptx::umma_commit(bar); });
            if (!ok) abort_flag = 1;
            PAIR ? umma_commit_leader(&mma_done) : ptx::umma_commit(&mma_done);   // all UMMAs complete before TMEM is released
            ptx::mbar_wait_spin(&mma_done, 0, p.status);
        } else if (warp == 3) {
            // ---------------- scales: 128 row scales and two weight scales a block, kScales blocks
            // at a time and one such batch ahead (a load's latency is longer than a block's product,
            // and each hand-over costs the drain a wait)
            int slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = t0; ok && t < tiles; t += t_step) {
                const Tile tl = tile_at(G, p.groups, t, C::kRows, kManyFeatures);
                const int r0 = tl.row0 + rank * kManyRows + lane;
                const float* ws = p.ws + ((size_t)tl.g * p.nb + min((tl.f0 >> 7) + (lane & 1), p.nb - 1)) * p.kb + (lane >> 1);
                for (int k0 = 0; k0 < p.kb; k0 += kScales) {
                    if (!ptx::mbar_wait_spin(&sc_empty[slot], phase ^ 1, p.status)) { abort_flag = 1; ok = false; break; }
                    const int nk = min(kScales, p.kb - k0);
                    for (int j = 0; j < nk; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i)   // rows behind the last: any scale, their sums are not stored
                            cp_async_4(&x_sc[slot][j][lane + 32 * i],
                                       p.xs + (size_t)(k0 + j) * p.rows + min(r0 + 32 * i, p.rows - 1));
                    if (lane < 2 * nk) cp_async_4(&w_sc[slot][lane >> 1][lane & 1], ws + k0);
                    ptx::cp_async_arrive_noinc(&sc_full[slot]);
                    slot ^= 1;
                    if (slot == 0) phase ^= 1;
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ---------------- drain: thread = row of TMEM lane quarter warp & 3, columns [128 cg, 128 cg + 128)
        const int quarter = warp & 3, cg = (warp - 4) >> 2;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16) + 128 * cg;
        const uint32_t freed = PAIR ? ptx::mapa_shared(ptx::smem_u32(&acc_empty[0]), 0) : 0;   // the leader's
        const float* my_x = &x_sc[0][0][quarter * 32 + lane];
        const float* my_w = &w_sc[0][0][cg];
        int slot = 0, q = 0;
        uint32_t sc_phase = 0, acc_phase = 0;
        bool ok = true;
        for (int t = t0; ok && t < tiles; t += t_step) {
            float acc[4][32];
            uint32_t d[2][32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                acc[0][i] = acc[1][i] = acc[2][i] = acc[3][i] = 0.f;
                d[1][i] = 0;
            }
            auto add = [&](float (&sum)[32], const uint32_t (&v)[32], float by) {
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[i] = fmaf(__uint_as_float(v[i]), by, sum[i]);
            };
            // A block's scale (one fp32 rounding) is fetched while the block before it is drained;
            // 32 columns load while 32 are added, the last 32 of a block while the next one's
            // first load.
            float s = 0.f, s_next = 0.f;
            if (ptx::mbar_wait_spin(&sc_full[slot], sc_phase, p.status))
                s_next = my_x[slot * kScales * kManyRows] * my_w[slot * kScales * 2];
            else
                ok = false;
            for (int kb = 0; ok && kb < p.kb; ++kb) {
                const float s_prev = s;
                s = s_next;
                if (!ptx::mbar_wait_spin(&acc_full[q], acc_phase, p.status)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t src = t_lane + q * kManyFeatures;
                ptx::tmem_ld32_nowait(src, d[0]);
                const int j = (kb + 1) % kScales;
                if (j == 0 || kb + 1 == p.kb) {   // the batch is read
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&sc_empty[slot]);
                    slot ^= 1;
                    if (slot == 0) sc_phase ^= 1;
                    if (kb + 1 < p.kb && !ptx::mbar_wait_spin(&sc_full[slot], sc_phase, p.status)) ok = false;
                }
                if (kb + 1 < p.kb)
                    s_next = my_x[(slot * kScales + j) * kManyRows] * my_w[(slot * kScales + j) * 2];
                add(acc[3], d[1], s_prev);
                ptx::tmem_wait_ld32(d[0]);
                ptx::tmem_ld32_nowait(src + 32, d[1]);
                add(acc[0], d[0], s);
                ptx::tmem_wait_ld32(d[1]);
                ptx::tmem_ld32_nowait(src + 64, d[0]);
                add(acc[1], d[1], s);
                ptx::tmem_wait_ld32(d[0]);
                ptx::tmem_ld32_nowait(src + 96, d[1]);
                add(acc[2], d[0], s);
                ptx::tmem_wait_ld32(d[1]);
                ptx::tc_fence_before();   // all in registers: the accumulator is free
                __syncwarp();
                if (lane == 0) PAIR ? arrive_cluster(freed + 8 * q) : ptx::mbar_arrive(&acc_empty[q]);
                q ^= 1;
                if (q == 0) acc_phase ^= 1;
            }
            if (!ok) {
                abort_flag = 1;
                break;
            }
            add(acc[3], d[1], s);
            const Tile tl = tile_at(G, p.groups, t, C::kRows, kManyFeatures);
            unsigned char* ebuf = smem + S * C::kStageBytes + (warp - 4) * kManyEpiBuf;
            const int f = tl.f0 + 128 * cg, row0 = rank * kManyRows + quarter * 32;
            // Out through shared memory, 64 bytes a row at a time (32 16-bit or 16 fp32 columns):
            // 16-byte pieces, swizzled by the row so that neither side has bank conflicts; four
            // lanes store one row's piece of a line.
            const int rows = min(32, tl.rows_left - row0);   // this warp's rows (<= 0: none)
            auto store_rows = [&](int col, int esize) {
                __syncwarp();
                const int piece = lane & 3, pc = col + piece * 16 / esize;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rr = 8 * i + (lane >> 2);
                    if (rr < rows && f + pc < p.n)
                        *reinterpret_cast<uint4*>(static_cast<unsigned char*>(p.out) +
                                                  ((size_t)(tl.row0 + row0 + rr) * p.n + f + pc) * esize) =
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
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const float* e = &acc[c >> 1][16 * (c & 1) + 4 * v];
                        *reinterpret_cast<float4*>(piece_at(v)) = make_float4(e[0], e[1], e[2], e[3]);
                    }
                    store_rows(16 * c, 4);
                }
            } else {
                const bool to_bf16 = p.dtype == kDtypeBf16;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float ax = acc[c][8 * v + 2 * i], ay = acc[c][8 * v + 2 * i + 1];
                            if (to_bf16) {
                                const __nv_bfloat162 p2 = __floats2bfloat162_rn(ax, ay);
                                o[i] = *reinterpret_cast<const uint32_t*>(&p2);
                            } else {
                                const __half2 p2 = __floats2half2_rn(ax, ay);
                                o[i] = *reinterpret_cast<const uint32_t*>(&p2);
                            }
                        }
                        *piece_at(v) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    store_rows(32 * c, 2);
                }
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (PAIR) ptx::cluster_sync_all();   // no UMMA reads the peer's memory, no arrival is under way any more
    if (warp == 3) {
        ptx::tc_fence_after();
        PAIR ? tmem_dealloc_pair(tmem, 512) : ptx::tmem_dealloc(tmem, 512);
    }
}

}  // namespace fp8
}  // namespace mla
