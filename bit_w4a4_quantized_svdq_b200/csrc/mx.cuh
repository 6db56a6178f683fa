// mx.cuh -- what the microscaling (MX) kernels share: the scale layout, the two
// element formats, vector loads and stores of 16 bf16 values, and the quantisation
// of one 32-element block by two lanes.
//
// A block is 32 consecutive elements of a row with one E8M0 scale byte.  Eight
// neighbouring lanes take 128 channels, 16 elements each: two lanes a block, four
// blocks an atom row, whose four scale bytes make one 32-bit word of the layout.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace svdq {

enum MxFormat : int { kMxFp8 = 0, kMxFp4 = 1 };

// Channels of one scale atom: 4 blocks of 32.
constexpr int kMxAtomK = 128;

// Byte offset of the scale word of [row, atom] (`atoms` per row): 128-row x 4-block
// atoms of 512 bytes, row r at (r % 32) * 16 + (r / 32 % 4) * 4, atoms along K first.
__device__ __forceinline__ int64_t mx_sf_word(int64_t row, int64_t atom, int64_t atoms) {
    return ((row >> 7) * atoms + atom) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Quotient and remainder by a divisor known on the host, for n < 2^31 (Granlund and
// Montgomery 1994, "Division by invariant integers using multiplication").
struct FastDiv {
    uint32_t d, mul, shift;
};

inline FastDiv make_fast_div(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    const uint64_t m = ((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1;
    return FastDiv{d, static_cast<uint32_t>(m), s};
}

__device__ __forceinline__ uint32_t fast_div(const FastDiv& f, uint32_t n) {
    return (__umulhi(f.mul, n) + n) >> f.shift;
}

// 16 bf16 values (32 bytes) of one lane: one 256-bit access where the address allows it
// (`wide`, the same for a whole launch), two 128-bit ones otherwise.
__device__ __forceinline__ void load16(const uint16_t* p, bool wide, uint32_t (&v)[8]) {
    if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "l"(p) : "memory");
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 8);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

// The same for values read once: they take no room in L1 and leave L2 first.
__device__ __forceinline__ void load16_stream(const uint16_t* p, bool wide, uint32_t (&v)[8]) {
    if (wide) {
        asm volatile("ld.global.L1::no_allocate.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "l"(p) : "memory");
    } else {
        load16(p, false, v);
    }
}

__device__ __forceinline__ void store16(uint16_t* p, bool wide, const uint32_t (&v)[8]) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     :: "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<uint4*>(p + 8) = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

inline bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// Scale byte of a block from the bits of its absolute maximum (an fp32 value with
// the sign cleared; NaN above infinity above every finite value):
//   e = floor(log2 amax) - emax, at least -127; -127 for a zero or subnormal amax.
// emax is the exponent of the format's largest power of two (E4M3: 8, E2M1: 2).
// E2M1 has no NaN and no infinity: a block that holds either gets the E8M0 NaN (255).
template <int kFmt>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    constexpr int kEmax = kFmt == kMxFp8 ? 8 : 2;
    const int field = static_cast<int>(amax_bits >> 23);
    if (kFmt == kMxFp4 && field == 255) return 255u;
    return static_cast<uint32_t>(max(field - kEmax, 0));
}

// 2^-e for scale byte e + 127 <= 253: a normal fp32, so the scaling is exact up to
// fp32 underflow, where both formats round to zero.
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Sixteen scaled values (8 pairs) -> E4M3 codes (16 bytes) or E2M1 codes (8 bytes),
// nearest, ties to even, saturating, sign kept.
__device__ __forceinline__ void mx_encode16(const uint64_t (&v)[8], uint32_t (&q)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a, b, c, d;
        unpack_f32x2(v[2 * j], a, b);
        unpack_f32x2(v[2 * j + 1], c, d);
        q[j] = cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);
    }
}
__device__ __forceinline__ void mx_encode16(const uint64_t (&v)[8], uint32_t (&q)[2]) {
    q[0] = cvt_e2m1x8_pairs(v[0], v[1], v[2], v[3]);
    q[1] = cvt_e2m1x8_pairs(v[4], v[5], v[6], v[7]);
}

// The scale word of an atom row from the scale bytes of its eight lanes (two lanes a
// block hold the same byte): valid in every lane.
__device__ __forceinline__ uint32_t mx_scale_word(uint32_t byte, int lane) {
    uint32_t w = byte << (8 * ((lane >> 1) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    return w | __shfl_xor_sync(0xffffffffu, w, 4);
}

// Quantise a lane's 16 values, whose block's other half is in lane ^ 1 (all 32 lanes
// of the warp call this): codes and the block's scale byte.  `amax_bits`: the maximum
// of |v| over the lane's values, as bits.
template <int kFmt, int kWords>
__device__ __forceinline__ uint32_t mx_quantize16(uint64_t (&v)[8], uint32_t amax_bits, uint32_t (&q)[kWords]) {
    static_assert(kWords == (kFmt == kMxFp8 ? 4 : 2), "16 codes");
    amax_bits = max(amax_bits, __shfl_xor_sync(0xffffffffu, amax_bits, 1));
    const uint32_t byte = mx_scale_byte<kFmt>(amax_bits);
    const float inv = mx_inv_scale(byte);                  // byte 255 (MXFP4): replaced below
    const uint64_t inv2 = pack_f32x2(inv, inv);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = mul_f32x2(v[j], inv2);
    mx_encode16(v, q);
    if (kFmt == kMxFp4 && byte == 255u) q[0] = q[1] = 0u;  // a NaN block's codes are zero
    return byte;
}

template <int kFmt>
__device__ __forceinline__ void mx_store_codes(uint8_t* p, const uint32_t* q) {
    if constexpr (kFmt == kMxFp8)
        *reinterpret_cast<uint4*>(p) = make_uint4(q[0], q[1], q[2], q[3]);
    else
        *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
}

}  // namespace svdq
