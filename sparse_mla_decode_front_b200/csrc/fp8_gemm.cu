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

template <int BN>
cudaError_t launch_few(const void* x, const void* w, const fp8::Problem& p, cudaStream_t s) {
    using C = fp8::FewCfg<BN>;
    auto kern = fp8::k_fp8_few<BN>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static bool attr_set[kMaxDevices] = {};   // per instantiation and device
    if (dev < 0 || dev >= kMaxDevices || !attr_set[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) attr_set[dev] = true;
    }
    CUtensorMap tw, tx;
    if (!make_tma_2d(&tw, w, (uint64_t)p.k, (uint64_t)p.groups * p.n, (uint64_t)p.k, fp8::BK, fp8::BF, 128, 1) ||
        !make_tma_2d(&tx, x, (uint64_t)p.k, (uint64_t)p.rows, (uint64_t)p.k, fp8::BK, BN, 128, 1))
        return cudaErrorInvalidValue;
    const long long tiles = ((long long)(p.rows + BN - 1) / BN + p.groups - 1) * ((p.n + fp8::BF - 1) / fp8::BF);
    const int grid = (int)std::min<long long>(tiles, sms_of(dev));
    return launch_pdl(kern, dim3(grid), dim3(fp8::kFewThreads), C::kSmem, s, tw, tx, p);
}

}  // namespace

// Tiles are counted in 32 bits (the smallest row tile is 16).
bool fp8_gemm_fits(int rows, int groups, int n) {
    return ((long long)rows / 16 + groups) * ((n + 127) / 128) < (1LL << 31) && (long long)groups * n < (1LL << 31);
}

cudaError_t launch_fp8_gemm(const void* x, const float* xs, const void* w, const float* ws, const int32_t* offsets,
                            int rows, int groups, int n, int k, void* out, int dtype, int32_t* status,
                            cudaStream_t s) {
    fp8::Problem p{xs, ws, offsets, rows, groups, n, k, (n + 127) / 128, (k + 127) / 128, out, dtype, status};
    const long long per_group = ((long long)rows + groups - 1) / groups;
    if (per_group <= 16) return launch_few<16>(x, w, p, s);
    if (per_group <= 32) return launch_few<32>(x, w, p, s);
    if (per_group <= 64) return launch_few<64>(x, w, p, s);
    return launch_few<128>(x, w, p, s);
}

}  // namespace mla
