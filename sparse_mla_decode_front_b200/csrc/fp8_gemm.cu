// Host side of the block-scaled 8-bit product: tensor maps, the variant and the launch.
#include "fp8_gemm.cuh"

#include <algorithm>

namespace mla {
namespace {

constexpr int kMaxDevices = 64;

int sms_of(int dev) {
    static int cached[kMaxDevices] = {};
    if (dev >= 0 && dev < kMaxDevices && cached[dev] > 0) return cached[dev];
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    if (dev >= 0 && dev < kMaxDevices) cached[dev] = n;
    return n;
}

// Shared memory of `kern` raised to `bytes`, once per kernel (its flags `set`) and device.
template <class K>
cudaError_t allow_smem(K kern, int bytes, bool* set, int dev) {
    if (dev >= 0 && dev < kMaxDevices && set[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) set[dev] = true;
    return e;
}

template <int BN>
cudaError_t launch_few(const void* x, const void* w, const fp8::Problem& p, cudaStream_t s) {
    using C = fp8::FewCfg<BN>;
    auto kern = fp8::k_fp8_few<BN>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static bool attr_set[kMaxDevices] = {};
    e = allow_smem(kern, C::kSmem, attr_set, dev);
    if (e != cudaSuccess) return e;
    CUtensorMap tw, tx;
    if (!make_tma_2d(&tw, w, (uint64_t)p.k, (uint64_t)p.groups * p.n, (uint64_t)p.k, fp8::BK, fp8::BF, 128, 1) ||
        !make_tma_2d(&tx, x, (uint64_t)p.k, (uint64_t)p.rows, (uint64_t)p.k, fp8::BK, BN, 128, 1))
        return cudaErrorInvalidValue;
    // Tiles there can be: a row tile for every BN rows and one more for each group that has rows.
    const int sms = sms_of(dev), f_tiles = (p.n + fp8::BF - 1) / fp8::BF;
    const long long tiles = ((long long)(p.rows - 1) / BN + std::min(p.groups, p.rows)) * f_tiles;
    // Few tiles leave SMs idle and a long chain of K blocks to each: split K as far as the SMs
    // and at least two blocks a CTA go.
    fp8::Problem q = p;
    while (q.split < 8 && tiles * q.split * 2 <= sms && p.kb >= 4 * q.split) q.split *= 2;
    const int grid = (int)std::min<long long>(tiles, sms) * q.split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(fp8::kFewThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    if (q.split == 1) return launch_pdl(kern, dim3(grid), dim3(fp8::kFewThreads), C::kSmem, s, tw, tx, q);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = q.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tw, tx, q);
}

cudaError_t launch_many(const void* x, const void* w, const fp8::Problem& p, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static bool attr_set[kMaxDevices] = {};
    e = allow_smem(fp8::k_fp8_many, fp8::kManySmem, attr_set, dev);
    if (e != cudaSuccess) return e;
    CUtensorMap tx, tw;
    if (!make_tma_2d(&tx, x, (uint64_t)p.k, (uint64_t)p.rows, (uint64_t)p.k, fp8::BK, fp8::kManyRows, 128, 1) ||
        !make_tma_2d(&tw, w, (uint64_t)p.k, (uint64_t)p.groups * p.n, (uint64_t)p.k, fp8::BK, fp8::kManyFeatures / 2, 128, 1))
        return cudaErrorInvalidValue;
    const int rows = 2 * fp8::kManyRows;
    const long long tiles = (((long long)p.rows + rows - 1) / rows + p.groups - 1) *
                            ((p.n + fp8::kManyFeatures - 1) / fp8::kManyFeatures);
    const int pairs = (int)std::min<long long>(tiles, std::max(1, sms_of(dev) / 2));
    return launch_pdl(fp8::k_fp8_many, dim3(2 * pairs), dim3(fp8::kManyThreads), fp8::kManySmem, s, tx, tw, p);
}

}  // namespace

// Tiles are counted in 32 bits (the smallest row tile is 16).
bool fp8_gemm_fits(int rows, int groups, int n) {
    return ((long long)rows / 16 + groups) * ((n + 127) / 128) < (1LL << 31) && (long long)groups * n < (1LL << 31);
}

cudaError_t launch_fp8_gemm(const void* x, const float* xs, const void* w, const float* ws, const int32_t* offsets,
                            int rows, int groups, int n, int k, void* out, int dtype, int32_t* status,
                            cudaStream_t s) {
    fp8::Problem p{xs, ws, offsets, rows, groups, n, k, (n + 127) / 128, (k + 127) / 128, out, dtype, status, 1};
    const long long per_group = ((long long)rows + groups - 1) / groups;
    if (per_group <= 16) return launch_few<16>(x, w, p, s);
    if (per_group <= 32) return launch_few<32>(x, w, p, s);
    if (per_group <= 64) return launch_few<64>(x, w, p, s);
    if (per_group <= 128) return launch_few<128>(x, w, p, s);
    return launch_many(x, w, p, s);
}

}  // namespace mla
