// Host side of the block-scaled 8-bit product: tensor maps, the variant and the launch.
#include "fp8_gemm.cuh"

#include <algorithm>
#include <mutex>

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

// launch_pdl (common.cuh) in clusters of `size` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), int size, dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                           Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) cap = cudaStreamCaptureStatusNone;
    cfg.attrs = attr;
    cfg.numAttrs = cap == cudaStreamCaptureStatusNone ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// How k_fp8_few splits `tiles` tiles of kb blocks: as far as every cluster is resident at once
// and each CTA has two blocks or more. clusters[i]: resident clusters of 2^i CTAs. Returns the
// split's logarithm.
int few_split(long long tiles, int kb, const int (&clusters)[4]) {
    int i = 0;
    while (i < 3 && tiles <= clusters[i + 1] && kb >= 4 << i) ++i;
    return i;
}

// What the host knows of one width of k_fp8_few on a device: resident clusters of 1, 2, 4 and 8
// CTAs. Host threads that call for the first time at once see the same values (the split decides
// the order of the sums).
struct FewDevice {
    int clusters[4];
    bool known;
};

template <int BN>
cudaError_t few_device(int dev, FewDevice* out) {
    static std::mutex mu;
    static FewDevice cached[kMaxDevices] = {};
    const bool keep = dev >= 0 && dev < kMaxDevices;
    std::lock_guard<std::mutex> lock(mu);
    if (keep && cached[dev].known) {
        *out = cached[dev];
        return cudaSuccess;
    }
    cudaError_t e = cudaFuncSetAttribute(fp8::k_fp8_few<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         fp8::FewCfg<BN>::kSmem);
    if (e != cudaSuccess) return e;
    FewDevice d{{sms_of(dev), 0, 0, 0}, true};
    for (int i = 1; i < 4; ++i) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(sms_of(dev) / 8 * 8);
        cfg.blockDim = dim3(fp8::kFewThreads);
        cfg.dynamicSmemBytes = fp8::FewCfg<BN>::kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1 << i;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&d.clusters[i], fp8::k_fp8_few<BN>, &cfg);
        if (e != cudaSuccess) return e;
    }
    if (keep) cached[dev] = d;
    *out = d;
    return cudaSuccess;
}

template <int BN>
cudaError_t launch_few(const void* x, const void* w, const fp8::Problem& p, int dev, cudaStream_t s) {
    using C = fp8::FewCfg<BN>;
    FewDevice fd;
    const cudaError_t e = few_device<BN>(dev, &fd);
    if (e != cudaSuccess) return e;
    CUtensorMap tw, tx;
    if (!make_tma_2d(&tw, w, (uint64_t)p.k, (uint64_t)p.groups * p.n, (uint64_t)p.k, fp8::BK, fp8::BF, 128, 1) ||
        !make_tma_2d(&tx, x, (uint64_t)p.k, (uint64_t)p.rows, (uint64_t)p.k, fp8::BK, BN, 128, 1))
        return cudaErrorInvalidValue;
    // Tiles there can be: a row tile for every BN rows and one more for each group that has rows.
    const long long tiles = ((long long)(p.rows - 1) / BN + std::min(p.groups, p.rows)) * ((p.n + fp8::BF - 1) / fp8::BF);
    fp8::Problem q = p;
    q.split_log2 = few_split(tiles, p.kb, fd.clusters);
    const dim3 grid((unsigned)std::min<long long>(tiles, sms_of(dev)) << q.split_log2), block(fp8::kFewThreads);
    if (q.split_log2 == 0) return launch_pdl(fp8::k_fp8_few<BN>, grid, block, C::kSmem, s, tw, tx, q);
    return launch_cluster(fp8::k_fp8_few<BN>, 1 << q.split_log2, grid, block, C::kSmem, s, tw, tx, q);
}

template <bool PAIR>
cudaError_t launch_many(const void* x, const void* w, const fp8::Problem& p, int dev, cudaStream_t s) {
    using C = fp8::ManyCfg<PAIR>;
    static bool attr_set[kMaxDevices] = {};
    if (dev < 0 || dev >= kMaxDevices || !attr_set[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(fp8::k_fp8_many<PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) attr_set[dev] = true;
    }
    CUtensorMap tx, tw;
    if (!make_tma_2d(&tx, x, (uint64_t)p.k, (uint64_t)p.rows, (uint64_t)p.k, fp8::BK, fp8::kManyRows, 128, 1) ||
        !make_tma_2d(&tw, w, (uint64_t)p.k, (uint64_t)p.groups * p.n, (uint64_t)p.k, fp8::BK, C::kWRows, 128, 1))
        return cudaErrorInvalidValue;
    const long long tiles = ((long long)(p.rows - 1) / C::kRows + std::min(p.groups, p.rows)) *
                            ((p.n + fp8::kManyFeatures - 1) / fp8::kManyFeatures);
    if (!PAIR)
        return launch_pdl(fp8::k_fp8_many<PAIR>, dim3((unsigned)std::min<long long>(tiles, sms_of(dev))),
                          dim3(fp8::kManyThreads), C::kSmem, s, tx, tw, p);
    const long long pairs = std::min<long long>(tiles, std::max(1, sms_of(dev) / 2));
    return launch_cluster(fp8::k_fp8_many<PAIR>, 2, dim3((unsigned)(2 * pairs)), dim3(fp8::kManyThreads), C::kSmem, s, tx,
                          tw, p);
}

// Estimated time of the plain product by k_fp8_few<BN>, in 10 ns: `block` for each K block of a
// tile, and 6 us around them.
template <int BN>
cudaError_t few_cost(const fp8::Problem& p, int dev, int block, long long* cost) {
    FewDevice fd;
    const cudaError_t e = few_device<BN>(dev, &fd);
    if (e != cudaSuccess) return e;
    const long long tiles = ((long long)p.rows + BN - 1) / BN * ((p.n + fp8::BF - 1) / fp8::BF);
    const int split = 1 << few_split(tiles, p.kb, fd.clusters), sms = sms_of(dev);
    *cost = 600 + block * ((tiles + sms - 1) / sms) * ((p.kb + split - 1) / split);
    return cudaSuccess;
}

// Which kernel and width (k_fp8_few's rows a tile, or 0 for k_fp8_many). Measured a K block of a
// CTA's tile: 0.30, 0.32, 0.36 and 0.66 us for 128 features x 16, 32, 64 and 128 rows, 0.55 us for
// a pair's 256 x 256. The plain product's tiles are known, so the estimates are compared
// (measured, us, few of 16 / 32 / 64 / 128 / many, K = 7168: 16 x 7168 15.6 / 16.3 / 17.3 / 21.1 /
// 35.2, 128 x 1536 22 / 17 / 13.7 / 12.8 / 34.8, 256 x 7168 120 / 74 / 45 / 34.8 / 33.5,
// 512 x 1536 55 / 40 / 25 / 27 / 33).
// Of groups the host knows only the rows' capacity, so it goes by the capacity an expert, between what
// three kinds of call want (32 experts, N = 4096, K = 7168, us, few of 16 / 32 / 64 / many):
//   equal groups                8: 141 / 143 / 151 / 171, 32: 237 / 146 / 154 / 173, 48: 369 / 261 / 155 / 173,
//                              64: 485 / 256 / 156 / 174, 96: 764 / 383 / 277 / 177
//   a router's (largest 2.5 x)  8: 152 / 141 / 147 / 162, 32: 304 / 201 / 166 / 165, 48: 397 / 240 / 190 / 166,
//                              64: 522 / 319 / 220 / 165, 96: 756 / 426 / 275 / 192
//   a rank with an eighth       8: 80 / 82 / 87 / 93, 32: 111 / 114 / 120 / 123, 48: 124 / 121 / 126 / 134,
//   of the experts             64: 142 / 133 / 140 / 148, 96: 162 / 143 / 146 / 160, 256: 289 / 202 / 167 / 163
// The narrow tiles go as far as a rank with a share gains by them and the others lose little, 64 rows to a
// capacity of 48. Past that many rows, which loses 12 % at most (a share's 96), while 64 rows lose 33 % at
// a router's 64. (Short runs at 1.965 GHz; in a loop under the power cap, 64 / many, at 48 and 64: a
// router's 213 / 208 and 256 / 216, a share's 173 / 190 and 179 / 195, equal groups 189 / 211 and 190 / 209.)
cudaError_t choose(const fp8::Problem& p, int dev, int* width) {
    if (p.offsets) {
        const long long g = p.groups;
        *width = p.rows <= 8 * g ? 16 : p.rows <= 32 * g ? 32 : p.rows <= 48 * g ? 64 : 0;
        return cudaSuccess;
    }
    const long long pairs = std::max(1, sms_of(dev) / 2);
    const long long tiles = ((long long)p.rows + 2 * fp8::kManyRows - 1) / (2 * fp8::kManyRows) *
                            ((p.n + fp8::kManyFeatures - 1) / fp8::kManyFeatures);
    long long best = 400 + 55 * ((tiles + pairs - 1) / pairs) * p.kb, c[4];
    cudaError_t e = few_cost<16>(p, dev, 30, &c[0]);
    if (e == cudaSuccess) e = few_cost<32>(p, dev, 32, &c[1]);
    if (e == cudaSuccess) e = few_cost<64>(p, dev, 36, &c[2]);
    if (e == cudaSuccess) e = few_cost<128>(p, dev, 66, &c[3]);
    *width = 0;
    for (int i = 0; i < 4; ++i)
        if (c[i] < best) {
            best = c[i];
            *width = 16 << i;
        }
    return e;
}

}  // namespace

// Rows, and tiles (the smallest row tile is 16) plus a step of the grid, are counted in 32 bits.
bool fp8_gemm_fits(int rows, int groups, int n) {
    return rows <= (1 << 30) && ((long long)rows / 16 + groups) * ((n + 127) / 128) < (1LL << 30) &&
           (long long)groups * n < (1LL << 31);
}

cudaError_t launch_fp8_gemm(const void* x, const float* xs, const void* w, const float* ws, const int32_t* offsets,
                            int rows, int groups, int n, int k, void* out, int dtype, int32_t* status,
                            cudaStream_t s) {
    fp8::Problem p{xs, ws, offsets, rows, groups, n, k, (n + 127) / 128, (k + 127) / 128, out, dtype, status, 0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int width = 0;
    e = choose(p, dev, &width);
    if (e != cudaSuccess) return e;
    switch (width) {
        case 16: return launch_few<16>(x, w, p, dev, s);
        case 32: return launch_few<32>(x, w, p, dev, s);
        case 64: return launch_few<64>(x, w, p, dev, s);
        case 128: return launch_few<128>(x, w, p, dev, s);
        default: return offsets ? launch_many<false>(x, w, p, dev, s) : launch_many<true>(x, w, p, dev, s);
    }
}

}  // namespace mla
