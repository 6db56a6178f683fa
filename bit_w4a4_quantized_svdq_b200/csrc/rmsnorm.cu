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
// 2^20, so equal inputs give equal codes whatever the launch shape.
//
// Bound by HBM: 2 (x) + 2 (residual) + 2 (h) + 1 + 1/32 (or 1/2 + 1/32) bytes per
// element.  A lane takes 16 channels (one 256-bit access per tensor), eight lanes an
// atom; the row stays in registers between the two sums.  CTAs are persistent and walk
// rows of stride gridDim, the next row's loads issued before the current one is
// reduced; the weight is read once per CTA.  Rows from M to the layout's 128-row
// padding only write their zero scales.
#include <algorithm>

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

// kVec: 16-channel pieces per lane (channels 16 t .. of lane t, then 16 (t + T) ..).
// kSubLanes: lanes of one row where a warp holds several rows (8, 16 or 32), or 0
// where a row takes the whole CTA.
template <int kFmt, int kVec, int kSubLanes, bool kW32>
__global__ void __launch_bounds__(kSubLanes ? 256 : 512, kSubLanes ? 3 : (kVec == 1 ? 2 : 1))
rmsnorm_mx_kernel(const NormArgs a) {
    constexpr bool kSub = kSubLanes > 0;
    static_assert(!kSub || kVec == 1, "short rows take one piece a lane");
    constexpr int kWords = kFmt == kMxFp8 ? 4 : 2;
    __shared__ double part[2][32];
    const int tid = threadIdx.x, lane = tid & 31;
    const int t = kSub ? (tid & (kSubLanes - 1)) : tid;                     // lane within the row
    const int T = kSub ? kSubLanes : static_cast<int>(blockDim.x);
    const int rows_per_cta = kSub ? static_cast<int>(blockDim.x) / kSubLanes : 1;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * rows_per_cta;
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_cta + (kSub ? tid / kSubLanes : 0);
    const int64_t atoms = a.K / kMxAtomK;
    bool in[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) in[i] = static_cast<int64_t>(t + i * T) * 16 < a.K;

    pdl_launch_dependents();
    pdl_wait();
    uint64_t wv[kVec][8];                                                   // the lane's weights as fp32 pairs
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int64_t c = static_cast<int64_t>(t + i * T) * 16;
#pragma unroll
        for (int j = 0; j < 8; ++j) wv[i][j] = 0ull;
        if (in[i]) {
#pragma unroll
            for (int j = 0; j < (kW32 ? 4 : 2); ++j) {
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(a.weight) + c / (kW32 ? 4 : 8) + j);
                if constexpr (kW32) {
                    wv[i][2 * j] = pack_f32x2(__uint_as_float(w.x), __uint_as_float(w.y));
                    wv[i][2 * j + 1] = pack_f32x2(__uint_as_float(w.z), __uint_as_float(w.w));
                } else {
                    wv[i][4 * j] = bf16x2_to_f32x2(w.x);
                    wv[i][4 * j + 1] = bf16x2_to_f32x2(w.y);
                    wv[i][4 * j + 2] = bf16x2_to_f32x2(w.z);
                    wv[i][4 * j + 3] = bf16x2_to_f32x2(w.w);
                }
            }
        }
    }
    uint32_t nx[kVec][8], nr[kVec][8];                                      // the next row's loads
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int64_t c = static_cast<int64_t>(t + i * T) * 16;
            if (in[i] && r < a.M) {
                load16_stream(a.x + r * a.ldx + c, a.wide_x, nx[i]);
                if (a.res) load16_stream(a.res + r * a.ldr + c, a.wide_r, nr[i]);
            }
        }
    };
    fetch(row);
    int it = 0;
    // every lane of a warp runs the same number of rounds (the shuffles need them all)
    for (int64_t r0 = row - (kSub ? tid / kSubLanes : 0); r0 < a.rows; r0 += stride, row += stride, ++it) {
        uint32_t h[kVec][8];
        const bool live = row < a.M;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[i][j] = (live && in[i]) ? nx[i][j] : 0u;
                if (a.res && live && in[i]) h[i][j] = add_bf16x2(h[i][j], nr[i][j]);
            }
        }
        fetch(row + stride);
        float rstd = 0.0f;
        // a whole CTA's row past M skips the sums together; a warp's mixed rows run them on zeros
        if (kSub || live) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const double lo = static_cast<double>(bf16_lo(h[i][j])), hi = static_cast<double>(bf16_hi(h[i][j]));
                    s = fma(lo, lo, s);
                    s = fma(hi, hi, s);
                }
                if (a.res && live && in[i]) {
                    const int64_t off = row * a.ldh + static_cast<int64_t>(t + i * T) * 16;
                    if (store_ok(off, 16, a.ext_h, a.err, kSiteNormH)) store16(a.h + off, a.wide_h, h[i]);
                }
            }
#pragma unroll
            for (int o = (kSub ? kSubLanes / 2 : 16); o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if constexpr (!kSub) {
                // two buffers in turn: a row's partials are read before the barrier of the next one's
                if (lane == 0) part[it & 1][tid >> 5] = s;
                __syncthreads();
                s = 0.0;
                const int warps = T >> 5;
                for (int w = 0; w < warps; ++w) s += part[it & 1][w];
            }
            rstd = rstd_of(s * a.inv_k + a.eps);
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const uint64_t rstd2 = pack_f32x2(rstd, rstd);
            uint64_t y[8];
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[j] = mul_f32x2(mul_f32x2(bf16x2_to_f32x2(h[i][j]), rstd2), wv[i][j]);
                float lo, hi;
                unpack_f32x2(y[j], lo, hi);
                m = absmax_nan(absmax_nan(m, lo), hi);
            }
            uint32_t q[kWords];
            const uint32_t byte = mx_quantize16<kFmt>(y, __float_as_uint(m), q);
            const uint32_t word = mx_scale_word(byte, lane);
            const int64_t c = static_cast<int64_t>(t + i * T) * 16;
            if (!in[i]) continue;
            if (live) {
                const int64_t off = (row * a.K + c) / (kFmt == kMxFp8 ? 1 : 2);
                if (store_ok(off, 4 * kWords, a.ext_codes, a.err, kSiteMxCodes)) mx_store_codes<kFmt>(a.codes + off, q);
            }
            if ((t & 7) == 0 && row < a.rows) {
                const int64_t off = mx_sf_word(row, c / kMxAtomK, atoms);
                if (store_ok(off, 4, a.ext_sf, a.err, kSiteMxSf))
                    *reinterpret_cast<uint32_t*>(a.sf + off) = live ? word : 0u;
            }
        }
    }
}

template <int kFmt, int kVec, int kSubLanes, bool kW32>
int norm_launch(const NormArgs& a, int threads, cudaStream_t st) {
    const int rows_per_cta = kSubLanes ? threads / kSubLanes : 1;
    // resident CTAs: 64 registers a thread allow 1024 threads an SM, 80 allow 768, 128 allow 512
    const int64_t sms = device_sm_count() > 0 ? device_sm_count() : 148;
    const int64_t per_sm = std::max(1, (kSubLanes ? 768 : kVec == 1 ? 1024 : 512) / threads);
    const int64_t grid = std::min<int64_t>((a.rows + rows_per_cta - 1) / rows_per_cta, sms * per_sm);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, rmsnorm_mx_kernel<kFmt, kVec, kSubLanes, kW32>, a));
}

template <int kFmt, bool kW32>
int norm_dispatch(const NormArgs& a, cudaStream_t st) {
    const int64_t lanes = a.K / 16;
    if (lanes <= 8) return norm_launch<kFmt, 1, 8, kW32>(a, 256, st);
    if (lanes <= 16) return norm_launch<kFmt, 1, 16, kW32>(a, 256, st);
    if (lanes <= 32) return norm_launch<kFmt, 1, 32, kW32>(a, 256, st);
    if (lanes <= 512) return norm_launch<kFmt, 1, 0, kW32>(a, static_cast<int>((lanes + 31) / 32 * 32), st);
    if (lanes <= 1024) return norm_launch<kFmt, 2, 0, kW32>(a, static_cast<int>((lanes + 63) / 64 * 32), st);
    return norm_launch<kFmt, 4, 0, kW32>(a, static_cast<int>((lanes + 127) / 128 * 32), st);
}

template <int kFmt>
int rmsnorm_mx(const void* X, int64_t M, int64_t K, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
               int weight_dtype, float eps, void* H, int64_t ldh, uint8_t* codes, uint8_t* sf, void* stream) {
    if (X == nullptr || weight == nullptr || codes == nullptr || sf == nullptr) return SVDQ_ERR_INVALID_ARG;
    if ((residual != nullptr) != (H != nullptr)) return SVDQ_ERR_INVALID_ARG;
    if (M < 1 || K < 1 || ldx < K || (residual && (ldr < K || ldh < K))) return SVDQ_ERR_INVALID_ARG;
    if (weight_dtype != 0 && weight_dtype != 1) return SVDQ_ERR_INVALID_ARG;
    if (!(eps > 0.0f) || eps > 3.0e38f) return SVDQ_ERR_INVALID_ARG;
    if (K % kMxAtomK != 0 || K > 32768 || M > (int64_t(1) << 40)) return SVDQ_ERR_UNSUPPORTED;
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
