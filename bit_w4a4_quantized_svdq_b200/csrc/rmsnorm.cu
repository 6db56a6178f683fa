// rmsnorm.cu -- root-mean-square norm with the residual's addition and a
// microscaled output (MXFP8 or MXFP4 codes and scales), one pass over the rows.
//
//   h    = bf16(x + residual)                       (h = x without a residual)
//   rstd = RN32(1 / sqrt(sum_k h^2 / K + eps))       squares, sum and root in fp64
//   y    = RN32(RN32(h * rstd) * weight)             fp32, never rounded to bf16
//   codes, scales = MX of y per 32 channels          (mx.cuh)
//
// The sum is held in fp64 because the codes are decided by comparing y with rounding
// borders: with it rstd is the correctly rounded value in all but about one row in
// 2^18, so equal inputs give equal codes whatever the launch shape.
//
// Bound by HBM: 2 (x) + 2 (residual) + 2 (h) + 1 + 1/32 (or 1/2 + 1/32) bytes per
// element.  A lane takes 16 channels (one 256-bit access per tensor), eight lanes an
// atom; a row of up to 8192 channels stays in registers between the sum and the
// quantisation.  A CTA walks rows of stride gridDim, the next row's loads issued before
// the current one is reduced; the weight is read once per CTA.  Rows from M to the
// layout's 128-row padding only write their zero scales.
//   16384 x 5120 with residual: into MXFP8 95-97 us (6.1 TB/s; a plain copy 6.5), into
//   MXFP4 92; 4096 x 5120 27 us; one row 3.1 us; 16384 x 20480 (two passes) 453-477 us.
//   Without the next row's loads ahead 16384 x 5120 takes 132 us.
#include <algorithm>
#include <cfloat>

#include "mx.cuh"

namespace svdq {
namespace {

struct NormArgs {
    const uint16_t* x;
    const uint16_t* res;
    const void* weight;
    uint16_t* h;
    uint8_t* codes;
    uint8_t* sf;
    int64_t M, K, ldx, ldr, ldh;
    int64_t rows;                  // padded to 128
    double eps, inv_k;
    bool wide_x, wide_r, wide_h;
    int64_t ext_h, ext_codes, ext_sf;
    uint32_t* err;
};

// 1 / sqrt(m) rounded to fp32: one Newton step (in fp64) from the fp32 reciprocal
// root, relative error below 2^-43 before the rounding; arguments outside fp32's
// comfortable range take the fp64 root.
__device__ __forceinline__ float rstd_of(double m) {
    if (!(m > 1e-30 && m < 1e30)) return static_cast<float>(1.0 / sqrt(m));
    const double r = static_cast<double>(rsqrtf(static_cast<float>(m)));
    return static_cast<float>(r * (1.5 - 0.5 * m * r * r));
}

// Two bf16 sums, each rounded once.  (The same bits as an fp32 addition rounded to bf16:
// where the exponents differ by 16 or less the fp32 sum is exact, and beyond that both
// give the larger term.)
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t o;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
    return o;
}

// max(m, |x|), NaN if either is.
__device__ __forceinline__ float absmax_nan(float m, float x) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(x)));
    return m;
}

// Channels 16 t .. 16 t + 15 of the weight as fp32 pairs.
template <bool kW32>
__device__ __forceinline__ void load_weight16(const void* weight, int64_t c, uint64_t (&wv)[8]) {
#pragma unroll
    for (int j = 0; j < (kW32 ? 4 : 2); ++j) {
        const uint4 w = ld_global_v4(static_cast<const uint8_t*>(weight) + c * (kW32 ? 4 : 2) + 16 * j);
        if constexpr (kW32) {
            wv[2 * j] = pack_f32x2(__uint_as_float(w.x), __uint_as_float(w.y));
            wv[2 * j + 1] = pack_f32x2(__uint_as_float(w.z), __uint_as_float(w.w));
        } else {
            wv[4 * j] = bf16x2_to_f32x2(w.x);
            wv[4 * j + 1] = bf16x2_to_f32x2(w.y);
            wv[4 * j + 2] = bf16x2_to_f32x2(w.z);
            wv[4 * j + 3] = bf16x2_to_f32x2(w.w);
        }
    }
}

// The sum of the squares of 16 values.
__device__ __forceinline__ double squares16(const uint32_t (&h)[8], double s) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const double lo = static_cast<double>(bf16_lo(h[j])), hi = static_cast<double>(bf16_hi(h[j]));
        s = fma(lo, lo, s);
        s = fma(hi, hi, s);
    }
    return s;
}

// A lane's 16 channels normalised and quantised (every lane of the warp calls this):
// codes, and the atom's scale word.
template <int kFmt, int kWords>
__device__ __forceinline__ uint32_t norm16(const uint32_t (&h)[8], float rstd, const uint64_t (&wv)[8], int lane,
                                           uint32_t (&q)[kWords]) {
    const uint64_t rstd2 = pack_f32x2(rstd, rstd);
    uint64_t y[8];
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = mul_f32x2(mul_f32x2(bf16x2_to_f32x2(h[j]), rstd2), wv[j]);
        float lo, hi;
        unpack_f32x2(y[j], lo, hi);
        m = absmax_nan(absmax_nan(m, lo), hi);
    }
    return mx_scale_word(mx_quantize16<kFmt>(y, __float_as_uint(m), q), lane);
}

// The sum of `s` over the CTA's warps, in every thread, in a fixed order.  `part`: one of
// two buffers used in turn (a row's partials are read before the next row's barrier).
__device__ __forceinline__ double block_sum(double s, double* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
    const int warps = blockDim.x >> 5;
    for (int w = 0; w < warps; ++w) s += part[w];
    return s;
}

// Rows of up to 8192 channels, held in registers.  kSubLanes: lanes of one row where a
// warp holds several rows (8, 16 or 32), or 0 where a row takes the whole CTA.
template <int kFmt, int kSubLanes, bool kW32>
__global__ void __launch_bounds__(kSubLanes ? 256 : 512, kSubLanes ? 3 : 2)
rmsnorm_mx_kernel(const NormArgs a) {
    constexpr bool kSub = kSubLanes > 0;
    constexpr int kWords = kFmt == kMxFp8 ? 4 : 2;
    __shared__ double part[2][32];
    const int tid = threadIdx.x, lane = tid & 31;
    const int t = kSub ? (tid & (kSubLanes - 1)) : tid;                     // lane within the row
    const int rows_per_cta = kSub ? static_cast<int>(blockDim.x) / kSubLanes : 1;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * rows_per_cta;
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_cta + (kSub ? tid / kSubLanes : 0);
    const int64_t c = static_cast<int64_t>(t) * 16;
    const bool in = c < a.K;

    pdl_launch_dependents();
    pdl_wait();
    uint64_t wv[8] = {};
    if (in) load_weight16<kW32>(a.weight, c, wv);
    uint32_t nx[8], nr[8];                                                  // the next row's loads
    auto fetch = [&](int64_t r) {
        if (in && r < a.M) {
            load16_stream(a.x + r * a.ldx + c, a.wide_x, nx);
            if (a.res) load16_stream(a.res + r * a.ldr + c, a.wide_r, nr);
        }
    };
    fetch(row);
    int it = 0;
    // every lane of a warp runs the same number of rounds (the shuffles need them all)
    for (int64_t r0 = row - (kSub ? tid / kSubLanes : 0); r0 < a.rows; r0 += stride, row += stride, ++it) {
        uint32_t h[8];
        const bool live = row < a.M;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h[j] = (live && in) ? nx[j] : 0u;
            if (a.res && live && in) h[j] = add_bf16x2(h[j], nr[j]);
        }
        fetch(row + stride);
        float rstd = 0.0f;
        // a whole CTA's row past M skips the sums together; a warp's mixed rows run them on zeros
        if (kSub || live) {
            double s = squares16(h, 0.0);
            if (a.res && live && in) {
                const int64_t off = row * a.ldh + c;
                if (store_ok(off, 16, a.ext_h, a.err, kSiteNormH)) store16(a.h + off, a.wide_h, h);
            }
            if constexpr (kSub) {
#pragma unroll
                for (int o = kSubLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            } else {
                s = block_sum(s, part[it & 1]);
            }
            rstd = rstd_of(s * a.inv_k + a.eps);
        }
        uint32_t q[kWords];
        const uint32_t word = norm16<kFmt>(h, rstd, wv, lane, q);
        if (!in) continue;
        if (live) {
            const int64_t off = (row * a.K + c) / (kFmt == kMxFp8 ? 1 : 2);
            if (store_ok(off, 4 * kWords, a.ext_codes, a.err, kSiteMxCodes)) mx_store_codes<kFmt>(a.codes + off, q);
        }
        if ((t & 7) == 0 && row < a.rows) {
            const int64_t off = mx_sf_word(row, c / kMxAtomK, a.K / kMxAtomK);
            if (store_ok(off, 4, a.ext_sf, a.err, kSiteMxSf))
                *reinterpret_cast<uint32_t*>(a.sf + off) = live ? word : 0u;
        }
    }
}

// Longer rows, of any length: the first pass forms h and its squares, the second reads h
// back (each lane its own stores, or x where there is no residual; from L2, the row
// having just passed) and quantises.
template <int kFmt, bool kW32>
__global__ void __launch_bounds__(512, 2)
rmsnorm_mx_long_kernel(const NormArgs a) {
    constexpr int kWords = kFmt == kMxFp8 ? 4 : 2;
    __shared__ double part[2][32];
    const int lane = threadIdx.x & 31;
    const int64_t c0 = static_cast<int64_t>(threadIdx.x) * 16;
    const int64_t step = static_cast<int64_t>(blockDim.x) * 16;
    const uint16_t* hsrc = a.res ? a.h : a.x;
    const int64_t ldh = a.res ? a.ldh : a.ldx;
    const bool wide = a.res ? a.wide_h : a.wide_x;
    pdl_launch_dependents();
    pdl_wait();
    int it = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ++it) {
        const bool live = row < a.M;
        float rstd = 0.0f;
        if (live) {
            double s = 0.0;
#pragma unroll 2
            for (int64_t c = c0; c < a.K; c += step) {
                uint32_t h[8], r[8];
                load16(a.x + row * a.ldx + c, a.wide_x, h);
                if (a.res) {
                    load16_stream(a.res + row * a.ldr + c, a.wide_r, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[j] = add_bf16x2(h[j], r[j]);
                    const int64_t off = row * a.ldh + c;
                    if (store_ok(off, 16, a.ext_h, a.err, kSiteNormH)) store16(a.h + off, a.wide_h, h);
                }
                s = squares16(h, s);
            }
            rstd = rstd_of(block_sum(s, part[it & 1]) * a.inv_k + a.eps);
        }
        // whole warps take each round: the shuffles need every lane
#pragma unroll 2
        for (int64_t c = c0; c - lane * 16 < a.K; c += step) {
            const bool in = c < a.K;
            uint32_t h[8] = {};
            uint64_t wv[8] = {};
            if (in && live) {
                load16(hsrc + row * ldh + c, wide, h);
                load_weight16<kW32>(a.weight, c, wv);
            }
            uint32_t q[kWords];
            const uint32_t word = norm16<kFmt>(h, rstd, wv, lane, q);
            if (!in) continue;
            if (live) {
                const int64_t off = (row * a.K + c) / (kFmt == kMxFp8 ? 1 : 2);
                if (store_ok(off, 4 * kWords, a.ext_codes, a.err, kSiteMxCodes)) mx_store_codes<kFmt>(a.codes + off, q);
            }
            if ((lane & 7) == 0) {
                const int64_t off = mx_sf_word(row, c / kMxAtomK, a.K / kMxAtomK);
                if (store_ok(off, 4, a.ext_sf, a.err, kSiteMxSf))
                    *reinterpret_cast<uint32_t*>(a.sf + off) = live ? word : 0u;
            }
        }
    }
}

// `per_sm`: CTAs resident on an SM (as the kernel's launch bounds allow its registers).
// The grid is whole waves of resident CTAs, as many as leave each CTA about `rounds` rounds
// (0: one wave).  With four, CTAs that start anew fill the gaps that CTAs in step leave in
// the memory's queue: 16384 x 5120 100 -> 95 us; with one round there is no next row to load
// ahead (110 us).
template <typename Kernel>
int norm_launch(Kernel kern, const NormArgs& a, int threads, int rows_per_cta, int per_sm, int rounds,
                cudaStream_t st) {
    const int64_t sms = device_sm_count() > 0 ? device_sm_count() : 148;
    const int64_t groups = (a.rows + rows_per_cta - 1) / rows_per_cta, wave = sms * per_sm;
    const int64_t waves = rounds ? std::max<int64_t>(1, (groups + wave * rounds / 2) / (wave * rounds)) : 1;
    const int64_t grid = std::min(groups, std::min<int64_t>(wave * waves, int64_t(1) << 30));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, kern, a));
}

template <int kFmt, bool kW32>
int norm_dispatch(const NormArgs& a, cudaStream_t st) {
    const int64_t lanes = a.K / 16;
    if (lanes <= 8) return norm_launch(rmsnorm_mx_kernel<kFmt, 8, kW32>, a, 256, 32, 3, 4, st);
    if (lanes <= 16) return norm_launch(rmsnorm_mx_kernel<kFmt, 16, kW32>, a, 256, 16, 3, 4, st);
    if (lanes <= 32) return norm_launch(rmsnorm_mx_kernel<kFmt, 32, kW32>, a, 256, 8, 3, 4, st);
    if (lanes <= 512) {
        const int threads = static_cast<int>((lanes + 31) / 32 * 32);
        return norm_launch(rmsnorm_mx_kernel<kFmt, 0, kW32>, a, threads, 1, 1024 / threads, 4, st);
    }
    // as few rounds of at most 512 threads as the row needs, all of them full
    const int64_t rounds = (lanes + 511) / 512;
    const int threads = static_cast<int>(((lanes + rounds - 1) / rounds + 31) / 32 * 32);
    return norm_launch(rmsnorm_mx_long_kernel<kFmt, kW32>, a, threads, 1, 1024 / threads, 0, st);
}

template <int kFmt>
int rmsnorm_mx(const void* X, int64_t M, int64_t K, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
               int weight_dtype, float eps, void* H, int64_t ldh, uint8_t* codes, uint8_t* sf, void* stream) {
    if (X == nullptr || weight == nullptr || codes == nullptr || sf == nullptr) return SVDQ_ERR_INVALID_ARG;
    if ((residual != nullptr) != (H != nullptr)) return SVDQ_ERR_INVALID_ARG;
    if (M < 1 || K < 1 || ldx < K || (residual && (ldr < K || ldh < K))) return SVDQ_ERR_INVALID_ARG;
    if (weight_dtype != 0 && weight_dtype != 1) return SVDQ_ERR_INVALID_ARG;
    if (!(eps > 0.0f) || eps > FLT_MAX) return SVDQ_ERR_INVALID_ARG;
    if (K % kMxAtomK != 0 || K > (int64_t(1) << 30) || M > (int64_t(1) << 40)) return SVDQ_ERR_UNSUPPORTED;
    if (!aligned16(X) || (ldx * 2) % 16 != 0 || !aligned16(weight) || !aligned16(codes) ||
        (reinterpret_cast<uintptr_t>(sf) & 3u))
        return SVDQ_ERR_MISALIGNED;
    if (residual && (!aligned16(residual) || (ldr * 2) % 16 != 0 || !aligned16(H) || (ldh * 2) % 16 != 0))
        return SVDQ_ERR_MISALIGNED;
    if (!device_is_sm100()) return SVDQ_ERR_NO_DEVICE;
    if (!debug_ptrs_ok({X, residual, weight, H, codes, sf})) return SVDQ_ERR_INVALID_ARG;
    NormArgs a = {};
    a.err = device_error_word();
    if (a.err == nullptr) return SVDQ_ERR_CUDA;
    a.x = static_cast<const uint16_t*>(X);
    a.res = static_cast<const uint16_t*>(residual);
    a.weight = weight;
    a.h = static_cast<uint16_t*>(H);
    a.codes = codes;
    a.sf = sf;
    a.M = M;
    a.K = K;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.rows = (M + 127) / 128 * 128;
    a.eps = static_cast<double>(eps);
    a.inv_k = 1.0 / static_cast<double>(K);
    a.wide_x = aligned32(X) && (ldx * 2) % 32 == 0;
    a.wide_r = aligned32(residual) && (ldr * 2) % 32 == 0;
    a.wide_h = aligned32(H) && (ldh * 2) % 32 == 0;
    a.ext_h = debug_extent(kSiteNormH, (M - 1) * ldh + K);
    a.ext_codes = debug_extent(kSiteMxCodes, kFmt == kMxFp8 ? M * K : M * K / 2);
    a.ext_sf = debug_extent(kSiteMxSf, static_cast<int64_t>(svdq_mxfp8_sf_bytes(M, K)));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return weight_dtype ? norm_dispatch<kFmt, true>(a, st) : norm_dispatch<kFmt, false>(a, st);
}

}  // namespace
}  // namespace svdq

extern "C" int svdq_rmsnorm_mxfp8(const void* X, int64_t M, int64_t K, int64_t ldx, const void* residual, int64_t ldr,
                                  const void* weight, int weight_dtype, float eps, void* H, int64_t ldh, uint8_t* codes,
                                  uint8_t* sf, void* stream) {
    return svdq::rmsnorm_mx<svdq::kMxFp8>(X, M, K, ldx, residual, ldr, weight, weight_dtype, eps, H, ldh, codes, sf,
                                          stream);
}

extern "C" int svdq_rmsnorm_mxfp4(const void* X, int64_t M, int64_t K, int64_t ldx, const void* residual, int64_t ldr,
                                  const void* weight, int weight_dtype, float eps, void* H, int64_t ldh, uint8_t* codes,
                                  uint8_t* sf, void* stream) {
    return svdq::rmsnorm_mx<svdq::kMxFp4>(X, M, K, ldx, residual, ldr, weight, weight_dtype, eps, H, ldh, codes, sf,
                                          stream);
}
