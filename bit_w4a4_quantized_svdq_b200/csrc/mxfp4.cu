// mxfp4.cu -- MXFP4 quantisation and the read-back of MXFP4 and MXFP8 codes.
//
// OCP microscaling FP4: E2M1 elements (two a byte, element 2i in the low nibble) with
// one E8M0 scale per 32 consecutive elements of a row.  Per block:
//
//   e     = floor(log2 amax) - 2, at least -127; -127 for an all-zero block
//   scale = e + 127;  code = E2M1(v * 2^-e), nearest, ties to even, |.| > 6 saturates
//   a block that holds an infinity or a NaN: scale 255 (the E8M0 NaN), codes 0
//
// bf16 inputs scale exactly, so one E2M1 rounding of an exact value decides each code.
// The read-back is value = code * 2^(scale - 127), exact in fp32 and rounded once to bf16.
//
// Both are bound by HBM: 2 bytes of bf16 against 1/2 (or 1) byte of code and 1/32 of
// scale per element.  Eight lanes take a unit of 128 channels, 16 elements (one
// 256-bit access) a lane; units are consecutive along the rows, so a warp reads 1 KB
// contiguous per step and keeps kUnroll of them in flight.  Each warp does that once:
// with a persistent grid of 8 CTAs an SM the loads and stores of the CTAs ran in step
// (16384 x 20480: quantiser 147 -> 140 us, read-back 146 -> 127 us, which is the copy
// rate).  One lane of eight writes the unit's four scale bytes as one word.  Rows from M
// to the layout's 128-row padding get zero scales.
#include "mx.cuh"

namespace svdq {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 3;
constexpr int kUnitsPerWarp = 4 * kUnroll;

struct MxArgs {
    const uint16_t* x;                          // quantiser input [M, K], row stride ldx
    uint16_t* y;                                // read-back output [M, K], row stride ldx
    uint8_t* codes;
    uint8_t* sf;
    int64_t M, K, ldx;
    uint32_t n_units;                           // 128-channel units: quantiser over padded rows
    FastDiv atoms;                              // units of one row
    bool wide;
    int64_t ext_codes, ext_sf, ext_y;
    uint32_t* err;
};

__global__ void __launch_bounds__(kThreads)
mx4_quantize_kernel(const MxArgs a) {
    const int lane = threadIdx.x & 31, sub = lane & 7;
    const uint32_t u0 = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kUnitsPerWarp;
    pdl_launch_dependents();
    pdl_wait();                                 // the kernel before has written what this one reads
    uint32_t v[kUnroll][8];
    int64_t row[kUnroll];
    uint32_t atom[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const uint32_t u = u0 + 4 * i + (lane >> 3);
        const uint32_t r = fast_div(a.atoms, u);
        row[i] = r;
        atom[i] = u - r * a.atoms.d;
        if (u < a.n_units && row[i] < a.M) {
            load16_stream(a.x + row[i] * a.ldx + static_cast<int64_t>(atom[i]) * kMxAtomK + sub * 16, a.wide, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0u;
        }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        uint32_t m2 = 0u;                   // |bf16| as bits, two at a time: integer order is value order
        uint64_t f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m2 = __vmaxu2(m2, v[i][j] & 0x7FFF7FFFu);
            f[j] = bf16x2_to_f32x2(v[i][j]);
        }
        uint32_t q[2];
        const uint32_t byte = mx_quantize16<kMxFp4>(f, max(m2 << 16, m2 & 0xFFFF0000u), q);
        const uint32_t word = mx_scale_word(byte, lane);
        if (u0 + 4 * i + (lane >> 3) >= a.n_units) continue;
        const int64_t c = (row[i] * a.K + static_cast<int64_t>(atom[i]) * kMxAtomK) / 2 + sub * 8;
        if (row[i] < a.M && store_ok(c, 8, a.ext_codes, a.err, kSiteMxCodes)) mx_store_codes<kMxFp4>(a.codes + c, q);
        const int64_t off = mx_sf_word(row[i], atom[i], a.atoms.d);
        if (sub == 0 && store_ok(off, 4, a.ext_sf, a.err, kSiteMxSf))
            *reinterpret_cast<uint32_t*>(a.sf + off) = word;
    }
}

// Two E2M1 codes (one byte) or two E4M3 codes (two bytes) -> their values as f16 pairs, exactly.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte) {
    uint32_t h;
    asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
    return h;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(pair)));
    return h;
}
__device__ __forceinline__ float f16_bits_to_f32(uint32_t h) {
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(static_cast<uint16_t>(h)));
    return f;
}

template <int kFmt>
__global__ void __launch_bounds__(kThreads)
mx_dequantize_kernel(const MxArgs a) {
    constexpr int kWords = kFmt == kMxFp8 ? 4 : 2;          // 16 codes
    const int lane = threadIdx.x & 31, sub = lane & 7;
    const uint32_t u0 = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kUnitsPerWarp;
    pdl_launch_dependents();
    pdl_wait();                                 // the kernel before has written what this one reads
    uint32_t q[kUnroll][kWords], sb[kUnroll];
    int64_t row[kUnroll], col[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const uint32_t u = u0 + 4 * i + (lane >> 3);
        const uint32_t r = fast_div(a.atoms, u), t = u - r * a.atoms.d;
        row[i] = r;
        col[i] = static_cast<int64_t>(t) * kMxAtomK + sub * 16;
        if (u < a.n_units) {
            sb[i] = ld_global_u8(a.sf + mx_sf_word(row[i], t, a.atoms.d) + (sub >> 1));
            if constexpr (kFmt == kMxFp8) {
                const uint4 w = ld_global_once_v4(a.codes + row[i] * a.K + col[i]);
                q[i][0] = w.x; q[i][1] = w.y; q[i][2] = w.z; q[i][3] = w.w;
            } else {
                const uint2 w = ld_global_v2(a.codes + (row[i] * a.K + col[i]) / 2);
                q[i][0] = w.x; q[i][1] = w.y;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        if (u0 + 4 * i + (lane >> 3) >= a.n_units) continue;
        // 2^(byte - 127): byte 0 is a subnormal fp32, byte 255 is NaN
        const float s = __uint_as_float(sb[i] == 0u ? 0x00400000u : sb[i] == 255u ? 0x7FC00000u : sb[i] << 23);
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t h = kFmt == kMxFp8 ? e4m3x2_to_f16x2(q[i][j >> 1] >> (16 * (j & 1)))
                                              : e2m1x2_to_f16x2((q[i][j >> 2] >> (8 * (j & 3))) & 0xFFu);
            const float lo = __fmul_rn(f16_bits_to_f32(h), s), hi = __fmul_rn(f16_bits_to_f32(h >> 16), s);
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[j]) : "f"(hi), "f"(lo));
        }
        const int64_t off = row[i] * a.ldx + col[i];
        if (store_ok(off, 16, a.ext_y, a.err, kSiteMxValues)) store16(a.y + off, a.wide, o);
    }
}

// Checks shared by both directions; `v` is the bf16 side.
int mx_prepare(const void* v, int64_t M, int64_t K, int64_t ldx, const uint8_t* codes, const uint8_t* sf, bool pad_rows,
               MxArgs* a) {
    if (v == nullptr || codes == nullptr || sf == nullptr) return SVDQ_ERR_INVALID_ARG;
    if (M < 1 || K < 1 || ldx < K) return SVDQ_ERR_INVALID_ARG;
    if (K % kMxAtomK != 0) return SVDQ_ERR_UNSUPPORTED;
    if (M > (int64_t(1) << 40) || K > (int64_t(1) << 30)) return SVDQ_ERR_UNSUPPORTED;
    if (!aligned16(v) || (ldx * 2) % 16 != 0 || !aligned16(codes) || (reinterpret_cast<uintptr_t>(sf) & 3u))
        return SVDQ_ERR_MISALIGNED;
    const int64_t rows = pad_rows ? (M + 127) / 128 * 128 : M;
    if (rows > 0x7FFF0000LL / (K / kMxAtomK)) return SVDQ_ERR_UNSUPPORTED;
    const int64_t units = rows * (K / kMxAtomK);
    if (!device_is_sm100()) return SVDQ_ERR_NO_DEVICE;
    if (!debug_ptrs_ok({v, codes, sf})) return SVDQ_ERR_INVALID_ARG;
    *a = MxArgs{};
    a->err = device_error_word();
    if (a->err == nullptr) return SVDQ_ERR_CUDA;
    a->codes = const_cast<uint8_t*>(codes);
    a->sf = const_cast<uint8_t*>(sf);
    a->M = M;
    a->K = K;
    a->ldx = ldx;
    a->n_units = static_cast<uint32_t>(units);
    a->atoms = make_fast_div(static_cast<uint32_t>(K / kMxAtomK));
    a->wide = aligned32(v) && (ldx * 2) % 32 == 0;
    return SVDQ_OK;
}

template <typename Kernel>
int mx_launch(Kernel kern, const MxArgs& a, void* stream) {
    constexpr uint32_t per_block = (kThreads / 32) * kUnitsPerWarp;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.n_units + per_block - 1) / per_block, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, kern, a));
}

template <int kFmt>
int mx_dequantize(const uint8_t* codes, const uint8_t* sf, int64_t M, int64_t K, void* Y, int64_t ldy, void* stream) {
    MxArgs a;
    const int st = mx_prepare(Y, M, K, ldy, codes, sf, false, &a);
    if (st != SVDQ_OK) return st;
    a.y = static_cast<uint16_t*>(Y);
    a.ext_y = debug_extent(kSiteMxValues, (M - 1) * ldy + K);
    return mx_launch(mx_dequantize_kernel<kFmt>, a, stream);
}

}  // namespace
}  // namespace svdq

extern "C" size_t svdq_mxfp4_sf_bytes(int64_t rows, int64_t K) { return svdq_mxfp8_sf_bytes(rows, K); }

extern "C" int svdq_quantize_mxfp4(const void* X, int64_t M, int64_t K, int64_t ldx, uint8_t* codes, uint8_t* sf,
                                   void* stream) {
    using namespace svdq;
    MxArgs a;
    const int st = mx_prepare(X, M, K, ldx, codes, sf, true, &a);
    if (st != SVDQ_OK) return st;
    a.x = static_cast<const uint16_t*>(X);
    a.ext_codes = debug_extent(kSiteMxCodes, M * K / 2);
    a.ext_sf = debug_extent(kSiteMxSf, static_cast<int64_t>(svdq_mxfp4_sf_bytes(M, K)));
    return mx_launch(mx4_quantize_kernel, a, stream);
}

extern "C" int svdq_dequantize_mxfp4(const uint8_t* codes, const uint8_t* sf, int64_t M, int64_t K, void* Y,
                                     int64_t ldy, void* stream) {
    return svdq::mx_dequantize<svdq::kMxFp4>(codes, sf, M, K, Y, ldy, stream);
}

extern "C" int svdq_dequantize_mxfp8(const uint8_t* codes, const uint8_t* sf, int64_t M, int64_t K, void* Y,
                                     int64_t ldy, void* stream) {
    return svdq::mx_dequantize<svdq::kMxFp8>(codes, sf, M, K, Y, ldy, stream);
}
