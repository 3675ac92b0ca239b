// The router's choices sorted by expert (include/moe_experts.h, mla_moe_sort): a stable
// counting sort over E + 1 bins (the held experts, and one for choices without a row here).
//
// With key(i) the bin of choice i (token-major), row(i) = #{j : key(j) < key(i)} +
// #{j < i : key(j) = key(i)}. Each warp takes a run of consecutive choices, 32 at a time:
// equal keys of a group of 32 are found with one match, the choice's place among them is a
// population count, and the warp's own bin counts (shared memory) carry the place from one
// group to the next. The counts are then summed over the warps before, bin by bin. No
// atomics decide a place, so the order is that of the choices.
//
// The data is a few bytes a choice; what costs is the chain of latencies and the launches.
// Up to kSingleItems choices run in one launch, one block for the sort and further blocks
// for the routing weights beside it; more are cut into chunks, a first launch counting each
// chunk's bins and a second placing the chunk behind the chunks before it.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "launch.h"
#include "moe_experts.h"

namespace mla {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kPerLane = 4;                            // choices a lane holds in one pass
constexpr int kPassItems = kThreads * kPerLane;        // choices of one pass of a block
constexpr int kSingleItems = kPassItems;
constexpr int kMaxChunks = 256;                        // chunks (blocks) of the two-launch form
constexpr int kMaxExperts = MLA_MOE_MAX_EXPERTS;
constexpr unsigned kAll = 0xffffffffu;

struct Args {
    const int32_t* idx;
    const bf16* aff;
    int T, K, n_total, first, E, normalize;
    float scale;
    int32_t *offsets, *row_of, *source_of;
    float* weights;
    int32_t* hist;        // [chunks][E + 1] of the two-launch form
    int n, chunks, chunk_items;
};

__device__ __forceinline__ int key_of(const Args& a, int i) {
    const long long e = (long long)a.idx[i] - a.first;   // any int32 may be there
    return e >= 0 && e < a.E ? (int)e : a.E;
}

// Routing weights of the tokens of block `b` of the weight blocks: a lane for each choice, so
// that the choices are read and the weights written side by side, 32 / K whole tokens a warp; a
// token's sum is taken in the order of its choices.
__device__ void token_weights(const Args& a, int b) {
    const int lane = threadIdx.x & 31, per_warp = 32 / a.K, g = lane / a.K;
    const long long t = ((long long)b * kWarps + (threadIdx.x >> 5)) * per_warp + g;
    const bool on = g < per_warp && t < a.T;
    const long long c = t * a.K + (lane - g * a.K);
    const int e = on ? a.idx[c] : -1;
    const float v = (unsigned)e < (unsigned)a.n_total ? bf2f(a.aff[(size_t)t * a.n_total + e]) : 0.f;
    float w = v;
    if (a.normalize) {
        float sum = 0.f;
        for (int j = 0; j < a.K; ++j) sum += __shfl_sync(kAll, v, min(g * a.K + j, 31));
        w = sum == 0.f ? 0.f : v / sum;
    }
    if (on) a.weights[c] = a.scale * w;
}

// Exclusive prefix sum of v over the block's threads; `red` holds kWarps ints.
__device__ int block_exclusive(int v, int* red) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kAll, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) red[wid] = s;
    __syncthreads();
    if (wid == 0) {
        int r = red[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kAll, r, o);
            if (lane >= o) r += u;
        }
        red[lane] = r;
    }
    __syncthreads();
    const int before = wid ? red[wid - 1] : 0;
    __syncthreads();
    return before + s - v;
}

// Exclusive prefix over the E + 1 bins of total[] into base[] (both in shared memory).
__device__ void bin_bases(const int* total, int* base, int bins, int* red) {
    int carry = 0;
    for (int b0 = 0; b0 < bins; b0 += kThreads) {   // one trip up to 1024 bins, a second for bin 1024
        const int b = b0 + threadIdx.x;
        const int v = b < bins ? total[b] : 0;
        const int ex = block_exclusive(v, red);
        if (b < bins) base[b] = carry + ex;
        __shared__ int last;
        if (threadIdx.x == kThreads - 1) last = ex + v;
        __syncthreads();
        carry += last;
        __syncthreads();
    }
}

// Count up to kPassItems choices [i0, i1): each choice's place within its warp, the warps'
// counts turned into those of the warps before (cnt [kWarps][bins]) and the bins' sums (total).
struct Pass {
    int w0, groups;                       // the warp's first choice, its groups of 32
    int key[kPerLane], place[kPerLane];   // bin (-1: none), place among the warp's choices of the bin
};
__device__ void count_pass(const Args& a, Pass& s, int i0, int i1, uint16_t* cnt, int* total) {
    const int bins = a.E + 1, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int (&key)[kPerLane] = s.key, (&place)[kPerLane] = s.place;
    s.groups = min(kPerLane, (i1 - i0 + kThreads - 1) / kThreads);   // a short pass still takes all warps
    s.w0 = i0 + wid * (32 * s.groups);
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
        const int i = s.w0 + 32 * j + lane;
        key[j] = j < s.groups && i < i1 ? key_of(a, i) : -1;
    }
    uint32_t* cw = reinterpret_cast<uint32_t*>(cnt);
    for (int b = threadIdx.x; b < (kWarps * bins + 1) / 2; b += kThreads) cw[b] = 0;
    __syncthreads();
    uint16_t* mine = cnt + wid * bins;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
        if (j >= s.groups) break;
        const unsigned same = __match_any_sync(kAll, key[j]);
        const unsigned before = same & ((1u << lane) - 1);
        place[j] = 0;
        if (key[j] >= 0) place[j] = mine[key[j]] + __popc(before);
        __syncwarp();
        if (key[j] >= 0 && before == 0) mine[key[j]] += (uint16_t)__popc(same);
        __syncwarp();
    }
    __syncthreads();
    // counts -> counts of the warps before; a bin's sum over all warps to total[]
    for (int b = threadIdx.x; b < bins; b += kThreads) {
        int t = 0;
#pragma unroll 8
        for (int w = 0; w < kWarps; ++w) {
            const int c = cnt[w * bins + b];
            cnt[w * bins + b] = (uint16_t)t;
            t += c;
        }
        total[b] = t;
    }
    __syncthreads();
}

// Rows of a counted pass: base[] holds each bin's next row.
__device__ __forceinline__ void write_pass(const Args& a, const Pass& s, const uint16_t* cnt, const int* base) {
    const uint16_t* mine = cnt + (threadIdx.x >> 5) * (a.E + 1);
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
        const int k = s.key[j];
        if (k < 0) continue;
        const int i = s.w0 + 32 * j + (threadIdx.x & 31);
        const int row = base[k] + mine[k] + s.place[j];
        const bool here = k < a.E;
        a.row_of[i] = here ? row : -1;
        a.source_of[row] = here ? i : -1;   // the last bin's rows lie behind the last expert's
    }
}

// Shared memory: `arrays` of [bins] int32, then the warps' counts.
size_t smem_bytes(int arrays, int bins) { return sizeof(int) * arrays * bins + sizeof(uint16_t) * (kWarps * bins + 1) + 4; }

__global__ void __launch_bounds__(kThreads) k_moe_sort_single(Args a) {
    extern __shared__ int sm[];
    __shared__ int red[kWarps];
    griddep_launch();
    griddep_wait();
    if (blockIdx.x > 0) {
        token_weights(a, blockIdx.x - 1);
        return;
    }
    const int bins = a.E + 1;
    int *total = sm, *base = sm + bins;
    uint16_t* cnt = reinterpret_cast<uint16_t*>(sm + 2 * bins);
    Pass s;
    count_pass(a, s, 0, a.n, cnt, total);
    bin_bases(total, base, bins, red);
    for (int b = threadIdx.x; b < bins; b += kThreads) a.offsets[b] = base[b];
    write_pass(a, s, cnt, base);
}

// First launch: blocks [0, chunks) count their chunk's bins, the others weigh tokens. The
// second launch may start once every block here is past its wait (see k_moe_sort_place).
__global__ void __launch_bounds__(kThreads) k_moe_sort_count(Args a) {
    extern __shared__ int sm[];
    griddep_wait();
    griddep_launch();
    if ((int)blockIdx.x >= a.chunks) {
        token_weights(a, blockIdx.x - a.chunks);
        return;
    }
    const int bins = a.E + 1;
    for (int b = threadIdx.x; b < bins; b += kThreads) sm[b] = 0;
    __syncthreads();
    const int i0 = blockIdx.x * a.chunk_items;                   // < n, so no overflow
    const int len = min(a.chunk_items, a.n - i0);
    int none = 0;   // choices without a row here, often most of them: counted apart from the atomics
#pragma unroll 4
    for (int i = threadIdx.x; i < len; i += kThreads) {
        const int k = key_of(a, i0 + i);
        if (k < a.E) atomicAdd(sm + k, 1);   // whole numbers: any order
        else ++none;
    }
    none = __reduce_add_sync(kAll, none);
    if ((threadIdx.x & 31) == 0 && none > 0) atomicAdd(sm + a.E, none);
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kThreads) a.hist[(size_t)blockIdx.x * bins + b] = sm[b];
}

// Second launch: each block's bases are the bins before plus the same bin of the chunks before.
// The first pass is counted before the wait for the first launch: it reads the choices alone,
// which were complete before that launch let this one start.
__global__ void __launch_bounds__(kThreads) k_moe_sort_place(Args a) {
    extern __shared__ int sm[];
    __shared__ int red[kWarps];
    griddep_launch();
    const int bins = a.E + 1;
    int *total = sm, *base = sm + bins, *all = sm + 2 * bins, *before = sm + 3 * bins;
    uint16_t* cnt = reinterpret_cast<uint16_t*>(sm + 4 * bins);
    const int c0 = blockIdx.x * a.chunk_items;
    const int len = min(a.chunk_items, a.n - c0);
    for (int b = threadIdx.x; b < bins; b += kThreads) all[b] = before[b] = 0;
    Pass s;
    count_pass(a, s, c0, c0 + min(len, kPassItems), cnt, total);
    griddep_wait();
    // several threads share a bin where there are few bins
    const int teams = max(1, kThreads / bins);
    const int team = threadIdx.x / bins, b1 = threadIdx.x - team * bins;
    for (int b = bins <= kThreads ? (team < teams ? b1 : bins) : threadIdx.x; b < bins;
         b += bins <= kThreads ? bins : kThreads) {
        int sum = 0, prev = 0;
        const int t0 = bins <= kThreads ? team : 0, step = bins <= kThreads ? teams : 1;
#pragma unroll 4
        for (int c = t0; c < a.chunks; c += step) {
            const int h = a.hist[(size_t)c * bins + b];
            sum += h;
            prev += c < (int)blockIdx.x ? h : 0;
        }
        if (sum) atomicAdd(all + b, sum);
        if (prev) atomicAdd(before + b, prev);
    }
    __syncthreads();
    bin_bases(all, base, bins, red);
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < bins; b += kThreads) a.offsets[b] = base[b];
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kThreads) base[b] += before[b];
    __syncthreads();
    write_pass(a, s, cnt, base);
    for (int o = kPassItems; o < len; o += kPassItems) {
        __syncthreads();
        for (int b = threadIdx.x; b < bins; b += kThreads) base[b] += total[b];
        __syncthreads();
        count_pass(a, s, c0 + o, c0 + min(len, o + kPassItems), cnt, total);
        write_pass(a, s, cnt, base);
    }
}

// Chunks of whole passes, at most kMaxChunks of them.
void chunking(long long n, int* chunks, int* items) {
    const long long passes = (n + kPassItems - 1) / kPassItems;
    const long long per = (passes + kMaxChunks - 1) / kMaxChunks;
    *items = (int)std::min<long long>(per * kPassItems, 1LL << 30);
    *chunks = (int)((n + *items - 1) / *items);
}

// A launch may use 48 KB of shared memory without asking, its static and dynamic parts together, and
// more up to the kernel's limit on the device. The limit is set once, to what the most experts take:
// it belongs to the kernel and not to a launch, so one that followed each call's size would be
// lowered by one host thread between another's request and its launch.
constexpr int kMaxDevices = 64;
template <void (*KERNEL)(Args), int ARRAYS>
cudaError_t allow_smem() {
    static std::atomic<bool> set[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev >= 0 && dev < kMaxDevices;
    if (keep && set[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_bytes(ARRAYS, kMaxExperts + 1));
    if (keep && e == cudaSuccess) set[dev].store(true, std::memory_order_release);
    return e;
}

}  // namespace

size_t moe_sort_workspace_bytes(int T, int K, int E) {
    const long long n = (long long)T * K;
    if (n <= kSingleItems) return 0;
    int chunks, items;
    chunking(n, &chunks, &items);
    return sizeof(int32_t) * (size_t)chunks * (E + 1);
}

cudaError_t launch_moe_sort(const int32_t* idx, const bf16* aff, int T, int K, int n_total, int first, int E,
                            int normalize, float scale, int32_t* offsets, int32_t* row_of, int32_t* source_of,
                            float* weights, void* workspace, cudaStream_t s) {
    if (T == 0) return cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (E + 1), s);
    Args a{idx, aff, T, K, n_total, first, E, normalize, scale, offsets, row_of, source_of, weights,
           static_cast<int32_t*>(workspace), T * K, 1, 0};
    const int weight_tokens = kWarps * (32 / K);   // of one block
    const int weight_blocks = aff ? (T + weight_tokens - 1) / weight_tokens : 0;
    const size_t smem = smem_bytes(2, E + 1), smem_place = smem_bytes(4, E + 1);
    if (a.n <= kSingleItems) {
        const cudaError_t e = allow_smem<k_moe_sort_single, 2>();
        if (e != cudaSuccess) return e;
        return launch_pdl(k_moe_sort_single, dim3(1 + weight_blocks), dim3(kThreads), smem, s, a);
    }
    cudaError_t e = allow_smem<k_moe_sort_place, 4>();
    if (e != cudaSuccess) return e;
    chunking(a.n, &a.chunks, &a.chunk_items);
    e = launch_pdl(k_moe_sort_count, dim3(a.chunks + weight_blocks), dim3(kThreads), sizeof(int) * (E + 1), s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl_mode(true, k_moe_sort_place, dim3(a.chunks), dim3(kThreads), smem_place, s, a);
}

}  // namespace mla
