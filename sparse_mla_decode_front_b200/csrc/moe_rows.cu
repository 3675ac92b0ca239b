// Token rows to the experts' order and back, and rows quantised to e4m3
// (include/moe_experts.h: mla_moe_gather, mla_moe_combine, mla_moe_combine_backward,
// mla_fp8_quantize). All of them read and write each element once and do a few operations
// on it, so they are bound by HBM at large sizes and by one chain of load latencies at small
// ones. Rows are cut into units of 16 elements (every supported width is a multiple of 16),
// one unit a thread, so a single token's row already spreads over several blocks and a
// prompt's fills the GPU many times over.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace mla {
namespace {

constexpr int kUnit = 16;                         // elements a thread holds
constexpr int kScaleBlock = 128;                  // elements that share a scale
constexpr int kLanesPerScale = kScaleBlock / kUnit;
constexpr int kThreads = 128;
constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 7.888609052210118e-31f;   // 2^-100: 448 / amax stays finite, amax / 448 normal

// ------------------------------------------------------------------ 16 elements <-> registers
// Plain loads throughout, not the read-only path: a kernel may start before the one that
// writes its inputs has ended (griddep_wait), and a load that the compiler takes for
// invariant could be moved before that wait.
template <class T>
struct Unit;   // raw 16-byte words of 16 elements
template <>
struct Unit<float> {
    static constexpr int kVecs = 4;
    __device__ static float2 pair(const uint4* v, int i) { return reinterpret_cast<const float2*>(v)[i]; }
    __device__ static void set(uint4* v, int i, float a, float b) { reinterpret_cast<float2*>(v)[i] = make_float2(a, b); }
};
template <>
struct Unit<bf16> {
    static constexpr int kVecs = 2;
    __device__ static float2 pair(const uint4* v, int i) {
        return __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(v)[i]);
    }
    __device__ static void set(uint4* v, int i, float a, float b) {
        reinterpret_cast<__nv_bfloat162*>(v)[i] = __floats2bfloat162_rn(a, b);
    }
};
template <>
struct Unit<__half> {
    static constexpr int kVecs = 2;
    __device__ static float2 pair(const uint4* v, int i) { return __half22float2(reinterpret_cast<const __half2*>(v)[i]); }
    __device__ static void set(uint4* v, int i, float a, float b) {
        reinterpret_cast<__half2*>(v)[i] = __floats2half2_rn(a, b);
    }
};

// ONCE: data that no other thread reads again (evict-first in the caches). Where it pays is
// measured kernel by kernel; it does for the kernels that write most of their bytes.
template <bool ONCE = false, class T>
__device__ __forceinline__ void load_unit(uint4* v, const T* p) {
#pragma unroll
    for (int i = 0; i < Unit<T>::kVecs; ++i)
        v[i] = ONCE ? __ldcs(reinterpret_cast<const uint4*>(p) + i) : reinterpret_cast<const uint4*>(p)[i];
}
template <class T>
__device__ __forceinline__ void store_unit_once(T* p, const uint4* v) {
#pragma unroll
    for (int i = 0; i < Unit<T>::kVecs; ++i) __stcs(reinterpret_cast<uint4*>(p) + i, v[i]);
}
template <class T>
__device__ __forceinline__ void store_unit(T* p, const uint4* v) {
#pragma unroll
    for (int i = 0; i < Unit<T>::kVecs; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
}

// Quantise the 128 values that the 8 lanes of a group hold (v: this lane's 16). The largest
// magnitude is taken on the bit patterns, so a NaN (above infinity there) is not lost.
__device__ __forceinline__ uint4 quantize_unit(const float (&v)[kUnit], float* scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kUnit; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < kLanesPerScale; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float amax = __uint_as_float(max(m, __float_as_uint(kAmaxFloor)));
    *scale = __fdiv_rn(amax, kE4m3Max);
    const float inv = __fdiv_rn(kE4m3Max, amax);
    uint4 q;
    uint16_t* h = reinterpret_cast<uint16_t*>(&q);
#pragma unroll
    for (int i = 0; i < kUnit / 2; ++i)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return q;
}

// ------------------------------------------------------------------ gather
// 4096 x 7168 bf16 to e4m3, 8 rows a token: 51.6 us, 5.8 TB/s (58.6 us with ordinary loads and
// stores; a plain fill of this GPU's memory runs at 3.9 TB/s, a copy at 6.4).
// One thread: one unit of one token, written to the token's rows. With FP8 a token is
// quantised once, not once a copy; the lanes of a scale block past the row's end hold zeros.
template <class T, bool FP8>
__global__ void __launch_bounds__(kThreads)
k_moe_gather(const T* x, const int32_t* row_of, int n_tokens, int K, int H, int R,
             int units, void* rows, float* scales) {
    griddep_launch();
    griddep_wait();
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long t = id / units;
    const int u = (int)(id - t * units);
    const bool inside = t < n_tokens && u * kUnit < H;
    if (!FP8 && !inside) return;
    uint4 raw[Unit<T>::kVecs] = {};
    if (inside) load_unit<true>(raw, x + (size_t)t * H + u * kUnit);
    int to[8];   // rows of the first choices, in flight with the unit
#pragma unroll
    for (int j = 0; j < 8; ++j) to[j] = inside && j < K ? row_of[t * K + j] : -1;
    uint4 q = make_uint4(0, 0, 0, 0);
    float scale = 0.f;
    if (FP8) {
        float v[kUnit];
#pragma unroll
        for (int i = 0; i < kUnit / 2; ++i) {
            const float2 f = Unit<T>::pair(raw, i);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
        q = quantize_unit(v, &scale);
        if (!inside) return;
    }
    for (int k0 = 0; k0 < K; k0 += 8) {
        if (k0 > 0)
#pragma unroll
            for (int j = 0; j < 8; ++j) to[j] = k0 + j < K ? row_of[t * K + k0 + j] : -1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = to[j];
            if ((unsigned)r >= (unsigned)R) continue;
            if (FP8) {
                __stcs(reinterpret_cast<uint4*>(static_cast<uint8_t*>(rows) + (size_t)r * H + u * kUnit), q);
                if (u % kLanesPerScale == 0) scales[(size_t)(u / kLanesPerScale) * R + r] = scale;
            } else {
                store_unit_once(static_cast<T*>(rows) + (size_t)r * H + u * kUnit, raw);
            }
        }
    }
}

// ------------------------------------------------------------------ combine
// 4096 tokens x 8 rows of 7168 bf16: 79 us, 6.7 TB/s (the measured copy rate; with the loads
// evict-first 92 us, with eight choices in flight 120 us). Eight blocks an SM (64 registers): with
// 80 registers 81 us, and 70 us instead of 57 for 8192 tokens of which 8424 choices are here.
// A warp holds 32 units of one token. Its lanes fetch the token's row indices and weights side by
// side, and the choices that have a row are taken from a ballot, kBatch rows in flight at a time:
// a rank that holds an eighth of the experts finds one of eight choices here, and waits for two
// latencies instead of one for each batch of indices and of rows.
template <class T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 6 : 8)
k_moe_combine(const T* rows, const int32_t* row_of, const float* weights, int n_tokens, int K, int H, int R, int units,
              int warps_per_row, T* out) {
    constexpr int kBatch = 8 / Unit<T>::kVecs;   // 128 bytes a lane
    griddep_launch();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const long long wid = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const long long t = wid / warps_per_row;
    const int u = (int)(wid - t * warps_per_row) * 32 + lane;
    if (t >= n_tokens) return;   // uniform over the warp
    const int my_row = lane < K ? row_of[t * K + lane] : -1;
    const float my_w = lane < K && weights ? weights[t * K + lane] : 1.f;
    unsigned left = __ballot_sync(0xffffffffu, (unsigned)my_row < (unsigned)R);
    float acc[kUnit] = {};
    while (left) {
        uint4 raw[kBatch][Unit<T>::kVecs];
        float w[kBatch];
        bool on[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {   // in the order of k
            on[j] = left != 0;
            const int k = on[j] ? __ffs(left) - 1 : 0;
            left &= left - 1;
            const int r = __shfl_sync(0xffffffffu, my_row, k);
            w[j] = __shfl_sync(0xffffffffu, my_w, k);
            on[j] = on[j] && u < units;
            if (on[j]) load_unit(raw[j], rows + (size_t)r * H + u * kUnit);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (!on[j]) continue;
#pragma unroll
            for (int i = 0; i < kUnit / 2; ++i) {
                const float2 f = Unit<T>::pair(raw[j], i);
                acc[2 * i] = fmaf(w[j], f.x, acc[2 * i]);
                acc[2 * i + 1] = fmaf(w[j], f.y, acc[2 * i + 1]);
            }
        }
    }
    if (u >= units) return;
    uint4 o[Unit<T>::kVecs];
#pragma unroll
    for (int i = 0; i < kUnit / 2; ++i) Unit<T>::set(o, i, acc[2 * i], acc[2 * i + 1]);
    store_unit(out + (size_t)t * H + u * kUnit, o);
}

// ------------------------------------------------------------------ combine, backward
// 2999 tokens x 8 rows of 7168 bf16, both gradients: 121 us, 6.0 TB/s (two units in flight 128 us;
// with ordinary loads and stores 134 us).
// A team of `team` warps takes one choice: grad_row = w grad_out[t], and the dot product of
// grad_out[t] with the row. Blocks of 8 warps hold 8 / team neighbouring choices, so the
// choices of a token read its grad_out from L1 / L2. Few choices take
// more warps each, for latency, up to 16 warps an SM (teams of 8 / 4 / 2 / 1, us, rows of 7168: 296
// choices 3.4 / 4.2 / 4.5 / 6.6, 584 5.5 / 4.4 / 6.4 / 10.5, 1024 9.5 / 7.5 / 7.1 / 10.9, 2048 16.9 /
// 13.0 / 12.2 / 11.8, 16384 138 / 98 / 89 / 84; rows of 1024: 1024 choices 6.2 / 3.8 / 2.6 / 2.8).
constexpr int kBackWarps = 8;
constexpr int kBackSmWarps = 16;
template <class T>
__global__ void __launch_bounds__(32 * kBackWarps)
k_moe_combine_backward(const T* dout, const T* rows, const int32_t* row_of,
                       const float* weights, long long n, int K, int H, int R, int units, int team,
                       T* drows, float* dw) {
    __shared__ float part[kBackWarps];
    griddep_launch();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int member = warp % team;
    const long long c = (long long)blockIdx.x * (kBackWarps / team) + warp / team;   // choice t * K + k
    const int r = c < n ? row_of[c] : -1;
    float sum = 0.f;
    if ((unsigned)r < (unsigned)R) {
        const float w = weights ? weights[c] : 1.f;
        const T* d = dout + (size_t)(c / K) * H;
        const T* x = rows + (size_t)r * H;
        T* g = drows + (size_t)r * H;
        constexpr int kBatch = 4;   // units in flight
        for (int u0 = member * 32 + lane; u0 < units; u0 += 32 * team * kBatch) {
            uint4 rd[kBatch][Unit<T>::kVecs], rx[kBatch][Unit<T>::kVecs], ro[Unit<T>::kVecs];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int u = u0 + b * 32 * team;
                if (u >= units) break;
                load_unit<true>(rd[b], d + u * kUnit);
                if (dw) load_unit<true>(rx[b], x + u * kUnit);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int u = u0 + b * 32 * team;
                if (u >= units) break;
                if (dw) {
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < kUnit / 2; ++i) {
                        const float2 p = Unit<T>::pair(rd[b], i), v = Unit<T>::pair(rx[b], i);
                        s = fmaf(p.x, v.x, s);
                        s = fmaf(p.y, v.y, s);
                    }
                    sum += s;
                }
                if (drows) {
#pragma unroll
                    for (int i = 0; i < kUnit / 2; ++i) {
                        const float2 p = Unit<T>::pair(rd[b], i);
                        Unit<T>::set(ro, i, w * p.x, w * p.y);
                    }
                    store_unit_once(g + u * kUnit, ro);
                }
            }
        }
    }
    if (!dw) return;
    sum = warp_sum(sum);
    if (team == 1) {
        if (lane == 0 && c < n) dw[c] = sum;
        return;
    }
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (member == 0 && lane == 0 && c < n) {
        float s = 0.f;
        for (int i = 0; i < team; ++i) s += part[warp + i];   // a fixed order
        dw[c] = s;
    }
}

// ------------------------------------------------------------------ quantise
// 32768 x 2048 of bf16 [g | u]: 62 us, 5.4 TB/s (evict-first loads, two units a thread or blocks of 16
// rows x 128 columns: 4 us more; 3 us of it are the scales' scattered 4-byte stores).
// One thread: one unit of one row. The gated activation in fp32: exp and the division by the
// fast forms (2 ulp and exp's 2 + |1.16 g| ulp), far below e4m3's 2^-4.
// Below a gate of -80, where 1 + exp(-g) is exp(-g) in fp32, the quotient is g exp(g): from about -87
// on the fast division gives 0 for a divisor past 2^126, and a product with a large u still counts.
// In two halves, so that no factor leaves fp32's range before the result does. (Such a unit is rare and
// is read again: 62 us, against 60.5 without it, 64.6 with the unit held and 72 with every gate this way.)
__device__ __forceinline__ float far_gate(float g, float u) {
    const float h = __expf(0.5f * g);
    return (g * h) * (h * u);
}
template <class T, bool GATED>
__device__ __forceinline__ void quantize_row_unit(const T* x, long long r, int u, bool inside, int R, int C, uint8_t* q,
                                                  float* scales) {
    uint4 rg[Unit<T>::kVecs] = {}, ru[Unit<T>::kVecs] = {};
    if (inside) {
        const T* p = x + (size_t)r * (GATED ? 2 * C : C) + u * kUnit;
        load_unit(rg, p);
        if (GATED) load_unit(ru, p + C);
    }
    float v[kUnit], low = 0.f;
#pragma unroll
    for (int i = 0; i < kUnit / 2; ++i) {
        float2 g = Unit<T>::pair(rg, i);
        if (GATED) {
            const float2 m = Unit<T>::pair(ru, i);
            low = fminf(low, fminf(g.x, g.y));
            g.x = __fdividef(g.x, 1.f + __expf(-g.x)) * m.x;
            g.y = __fdividef(g.y, 1.f + __expf(-g.y)) * m.y;
        }
        v[2 * i] = g.x;
        v[2 * i + 1] = g.y;
    }
    if (GATED && low < -80.f) {
        const T* p = x + (size_t)r * (2 * C) + u * kUnit;
        load_unit(rg, p);
        load_unit(ru, p + C);
#pragma unroll
        for (int i = 0; i < kUnit / 2; ++i) {
            const float2 g = Unit<T>::pair(rg, i), m = Unit<T>::pair(ru, i);
            if (g.x < -80.f) v[2 * i] = far_gate(g.x, m.x);
            if (g.y < -80.f) v[2 * i + 1] = far_gate(g.y, m.y);
        }
    }
    float scale;
    const uint4 o = quantize_unit(v, &scale);
    if (!inside) return;
    *reinterpret_cast<uint4*>(q + (size_t)r * C + u * kUnit) = o;
    if (u % kLanesPerScale == 0) scales[(size_t)(u / kLanesPerScale) * R + r] = scale;
}

// All rows: one unit a thread. With a count of valid rows (SOME) the grid is what the GPU holds at
// once and strides over the valid rows: a rank that holds an eighth of the experts has capacity
// for eight times its rows (8424 of 65536 rows x 2048: 20 us, 73 us when a block for every row
// looked whether it was needed).
template <class T, bool GATED, bool SOME>
__global__ void __launch_bounds__(kThreads)
k_fp8_quantize(const T* x, int R, int C, int units, const int32_t* valid_rows, uint8_t* q, float* scales) {
    griddep_launch();
    griddep_wait();
    const int rows = SOME ? min(R, *valid_rows) : R;
    long long first = (long long)blockIdx.x * kThreads;
    do {
        const long long r = (first + threadIdx.x) / units;
        const int u = (int)(first + threadIdx.x - r * units);
        if (SOME && first / units >= rows) return;   // uniform over the block
        quantize_row_unit<T, GATED>(x, r, u, r < rows && u * kUnit < C, R, C, q, scales);
        first += (long long)gridDim.x * kThreads;
    } while (SOME);
}

// Units of a row: whole scale blocks when lanes share a scale, else the row's own.
int row_units(int width, bool whole_blocks) {
    return whole_blocks ? (width + kScaleBlock - 1) / kScaleBlock * kLanesPerScale : width / kUnit;
}
// SMs of the current device.
cudaError_t count_sms(int* sms) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}
unsigned blocks_for(long long rows, int units) { return (unsigned)((rows * units + kThreads - 1) / kThreads); }

template <class T>
cudaError_t gather_as(const void* x, const int32_t* row_of, int T_, int K, int H, int R, void* rows, float* scales,
                      cudaStream_t s) {
    const int units = row_units(H, scales != nullptr);
    const dim3 grid(blocks_for(T_, units));
    const T* xt = static_cast<const T*>(x);
    if (scales)
        return launch_pdl(k_moe_gather<T, true>, grid, dim3(kThreads), 0, s, xt, row_of, T_, K, H, R, units, rows, scales);
    return launch_pdl(k_moe_gather<T, false>, grid, dim3(kThreads), 0, s, xt, row_of, T_, K, H, R, units, rows, scales);
}

template <class T>
cudaError_t combine_as(const void* rows, const int32_t* row_of, const float* w, int T_, int K, int H, int R, void* out,
                       cudaStream_t s) {
    const int units = row_units(H, false), warps = (units + 31) / 32;
    return launch_pdl(k_moe_combine<T>, dim3(blocks_for(T_, 32 * warps)), dim3(kThreads), 0, s,
                      static_cast<const T*>(rows), row_of, w, T_, K, H, R, units, warps, static_cast<T*>(out));
}

template <class T>
cudaError_t combine_backward_as(const void* dout, const void* rows, const int32_t* row_of, const float* w, int T_,
                                int K, int H, int R, void* drows, float* dw, cudaStream_t s) {
    const long long n = (long long)T_ * K;
    const int units = row_units(H, false);
    int team = kBackWarps, sms = 0;
    const cudaError_t e = count_sms(&sms);
    if (e != cudaSuccess) return e;
    while (team > 1 && n * team > (long long)kBackSmWarps * sms) team >>= 1;
    const long long per_block = kBackWarps / team;
    return launch_pdl(k_moe_combine_backward<T>, dim3((unsigned)((n + per_block - 1) / per_block)),
                      dim3(32 * kBackWarps), 0, s, static_cast<const T*>(dout), static_cast<const T*>(rows), row_of, w,
                      n, K, H, R, units, team, static_cast<T*>(drows), dw);
}

template <class T, bool GATED>
cudaError_t quantize_as(const void* x, int R, int C, const int32_t* valid, void* q, float* scales, cudaStream_t s) {
    const int units = row_units(C, true);
    const unsigned blocks = blocks_for(R, units);
    const T* xt = static_cast<const T*>(x);
    uint8_t* qt = static_cast<uint8_t*>(q);
    if (!valid)
        return launch_pdl(k_fp8_quantize<T, GATED, false>, dim3(blocks), dim3(kThreads), 0, s, xt, R, C, units, valid, qt,
                          scales);
    int sms = 0;
    const cudaError_t e = count_sms(&sms);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_fp8_quantize<T, GATED, true>, dim3(std::min(blocks, 16u * sms)), dim3(kThreads), 0, s, xt, R, C,
                      units, valid, qt, scales);
}
template <class T>
cudaError_t quantize_any(const void* x, int R, int C, int gated, const int32_t* valid, void* q, float* scales,
                         cudaStream_t s) {
    return gated ? quantize_as<T, true>(x, R, C, valid, q, scales, s) : quantize_as<T, false>(x, R, C, valid, q, scales, s);
}

}  // namespace

// Blocks of 128 threads over rows x units (of whole warps at most): the grid's x extent holds 2^31 - 1.
bool moe_rows_fit(long long rows, int width) {
    const long long units = (row_units(width, true) + 31) / 32 * 32LL;
    return (rows * units + kThreads - 1) / kThreads < (1LL << 31);
}

cudaError_t launch_moe_gather(const void* x, int dtype, const int32_t* row_of, int T, int K, int H, int R, void* rows,
                              float* scales, cudaStream_t s) {
    switch (dtype) {
        case kDtypeBf16: return gather_as<bf16>(x, row_of, T, K, H, R, rows, scales, s);
        case kDtypeFp16: return gather_as<__half>(x, row_of, T, K, H, R, rows, scales, s);
        default: return gather_as<float>(x, row_of, T, K, H, R, rows, scales, s);
    }
}

cudaError_t launch_moe_combine(const void* rows, int dtype, const int32_t* row_of, const float* w, int T, int K, int H,
                               int R, void* out, cudaStream_t s) {
    switch (dtype) {
        case kDtypeBf16: return combine_as<bf16>(rows, row_of, w, T, K, H, R, out, s);
        case kDtypeFp16: return combine_as<__half>(rows, row_of, w, T, K, H, R, out, s);
        default: return combine_as<float>(rows, row_of, w, T, K, H, R, out, s);
    }
}

cudaError_t launch_moe_combine_backward(const void* dout, const void* rows, int dtype, const int32_t* row_of,
                                        const float* w, int T, int K, int H, int R, void* drows, float* dw,
                                        cudaStream_t s) {
    switch (dtype) {
        case kDtypeBf16: return combine_backward_as<bf16>(dout, rows, row_of, w, T, K, H, R, drows, dw, s);
        case kDtypeFp16: return combine_backward_as<__half>(dout, rows, row_of, w, T, K, H, R, drows, dw, s);
        default: return combine_backward_as<float>(dout, rows, row_of, w, T, K, H, R, drows, dw, s);
    }
}

cudaError_t launch_fp8_quantize(const void* x, int dtype, int R, int C, int gated, const int32_t* valid, void* q,
                                float* scales, cudaStream_t s) {
    switch (dtype) {
        case kDtypeBf16: return quantize_any<bf16>(x, R, C, gated, valid, q, scales, s);
        case kDtypeFp16: return quantize_any<__half>(x, R, C, gated, valid, q, scales, s);
        default: return quantize_any<float>(x, R, C, gated, valid, q, scales, s);
    }
}

}  // namespace mla
