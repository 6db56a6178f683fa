// linear_mx4.cu -- the MXFP4 linear: block-scaled E2M1 x E2M1 GEMM on the tcgen05
// tensor cores (kind::mxf4, one E8M0 scale per 32 elements), bias in the epilogue.
//
//   Y[m, n] = bf16( sum_k dec(A)[m, k] dec(W)[n, k] + bias[n] ),  fp32 accumulation
//
// few rows: the weight is what has to be read, (K/2 + K/32) bytes a row of W.  The
// MMA takes 128 rows of W as its M operand and the activation rows (8 to 128) as its N
// operand, so no tensor-core row is spent on rows that are not there.  A CTA owns one
// block of 128 weight rows and a slice of K; the slices of one block are a cluster,
// whose partial sums meet over distributed shared memory in rank order (no workspace,
// no atomics: bitwise repeatable).
#include <algorithm>

#include "mx.cuh"

namespace svdq {
namespace {

constexpr int kStageK = 256;                     // channels per stage (128 code bytes a row)
constexpr uint32_t kSfAtoms = 1024;              // scale bytes of 128 rows per stage: two atoms

struct Mx4Args {
    const uint16_t* bias;
    uint16_t* Y;
    int64_t ldy;
    int64_t M, N, K;
    int k_stages;
    int64_t ext_y;
    uint32_t* err;
};

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
constexpr int kFewThreads = 192;                 // warps: 0 producer, 1 MMA issuer, 2..5 epilogue

// Shared memory per CTA is kept above a third of the SM's, so at most two CTAs share
// an SM and their tensor memory (at most 256 columns each) always fits: an allocation
// that had to wait could otherwise hold up a cluster whose other half waits elsewhere.
template <int kNT>
struct FewLayout {
    static constexpr int kStages = kNT <= 64 ? 4 : 3;
    static constexpr uint32_t kW = 128 * 128, kA = kNT * 128;
    static constexpr uint32_t kStage = kW + kA + 2 * kSfAtoms;
    static constexpr uint32_t kOffBar = kStages * kStage;
    static constexpr uint32_t kBytes = kOffBar + 256;
    static constexpr uint32_t kSmem = kBytes + 1024 < 80 * 1024 ? 80 * 1024 : kBytes + 1024;
    static constexpr uint32_t kAccCols = kNT < 32 ? 32 : kNT;
    static constexpr uint32_t kTmem = kNT <= 64 ? 128 : 256;
    static_assert(kAccCols + 16 * kStages <= kTmem, "accumulator and one scale buffer per stage");
    static_assert(kNT * 128 * 4 <= kStages * kStage, "partial sums reuse the ring");
    static_assert(kSmem <= 112 * 1024, "two CTAs per SM");
};

template <int kNT>
__global__ void __launch_bounds__(kFewThreads)
linear_mx4_few_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a,
                      const __grid_constant__ CUtensorMap tmap_sfw, const __grid_constant__ CUtensorMap tmap_sfa,
                      const Mx4Args args, const int splits) {
    using L = FewLayout<kNT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
    uint64_t* empty = full + L::kStages;
    uint64_t* acc_full = empty + L::kStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int n_blk = static_cast<int>(blockIdx.x) / splits;
    const int m0 = static_cast<int>(blockIdx.y) * kNT;
    const int kb0 = static_cast<int>(static_cast<int64_t>(args.k_stages) * rank / splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(args.k_stages) * (rank + 1) / splits);

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, L::kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tmap(&tmap_w);
            prefetch_tmap(&tmap_a);
            prefetch_tmap(&tmap_sfw);
            prefetch_tmap(&tmap_sfa);
            pdl_wait();
            int s = 0, it = 0;
            uint32_t ph = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                if (!mbar_wait(&empty[s], ph ^ 1, abort_flag, args.err, kErrWaitEmpty)) break;
                uint8_t* st = smem + s * L::kStage;
                mbar_arrive_expect_tx(&full[s], L::kStage);
                tma_load_2d(st, &tmap_w, &full[s], kb * 128, n_blk * 128);
                tma_load_3d(st + L::kW + L::kA, &tmap_sfw, &full[s], 0, kb * 4, n_blk);
                tma_load_2d(st + L::kW, &tmap_a, &full[s], kb * 128, m0);
                tma_load_3d(st + L::kW + L::kA + kSfAtoms, &tmap_sfa, &full[s], 0, kb * 4, m0 / 128);
                if (++s == L::kStages) { s = 0; ph ^= 1u; }
            }
            // Bounded drain of the copies still in flight (an early exit only).
            for (int i = (it > L::kStages ? it - L::kStages : 0); i < it; ++i) {
                const long long t0 = clock64();
                while (!mbar_try_wait(&full[i % L::kStages], (i / L::kStages) & 1) && clock64() - t0 < kWaitLimitCycles) {}
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(&full[s], ph, abort_flag, args.err, kErrWaitFull)) { ok = false; break; }
                tc_fence_after();
                const uint32_t base = smem_u32(smem + s * L::kStage);
                const uint64_t dw = desc_kmajor_sw128(base), da = desc_kmajor_sw128(base + L::kW);
                const uint32_t sfw = tmem + L::kAccCols + s * 16, sfa = sfw + 8;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    tc_cp_32x128b_x4(sfw + 4 * i, desc_sf_block(base + L::kW + L::kA + 512 * i));
                    tc_cp_32x128b_x4(sfa + 4 * i, desc_sf_block(base + L::kW + L::kA + kSfAtoms + 512 * i));
                }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_mxf4(tmem, dw + 2 * kk, da + 2 * kk, idesc_mxf4(128, kNT, 2 * (kk & 1)), sfw + 4 * (kk >> 1),
                             sfa + 4 * (kk >> 1), (kb > kb0 || kk > 0) ? 1u : 0u);
                tc_commit(&empty[s]);
                if (++s == L::kStages) { s = 0; ph ^= 1u; }
            }
            if (ok) tc_commit(acc_full);
        }
    } else {
        // Lane of the accumulator = row of the weight block, column = activation row.
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t tbase = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const bool ok = __all_sync(0xffffffffu, mbar_wait(acc_full, 0, abort_flag, args.err, kErrWaitMma));
        tc_fence_after();
        if (ok) {
            const int64_t n = static_cast<int64_t>(n_blk) * 128 + row;
            const float b = (splits == 1 && args.bias && n < args.N) ? bf16_lo(args.bias[n]) : 0.0f;
            float* part = reinterpret_cast<float*>(smem);
            constexpr int kC = kNT < 32 ? kNT : 32;
#pragma unroll
            for (int c = 0; c < kNT; c += kC) {
                uint32_t v[kC];
                if constexpr (kC == 8) tmem_ld_32x32b_x8(tbase + c, v);
                else if constexpr (kC == 16) tmem_ld_32x32b_x16(tbase + c, v);
                else tmem_ld_32x32b_x32(tbase + c, v);
                tmem_ld_wait(v);
#pragma unroll
                for (int j = 0; j < kC; ++j) {
                    const int64_t m = m0 + c + j;
                    if (splits > 1) {
                        part[(c + j) * 128 + row] = __uint_as_float(v[j]);
                    } else if (m < args.M && n < args.N && store_ok(m * args.ldy + n, 1, args.ext_y, args.err, kSiteLinearMx4)) {
                        args.Y[m * args.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[j]) + b));
                    }
                }
            }
        }
    }
    __syncwarp();
    if (splits > 1) {
        // Every CTA of the cluster sums its share of the activation rows over all ranks,
        // in rank order; a wait that ran out has set the error word and still gets here.
        cluster_sync_all();
        if (warp >= 2) {
            const int row = (warp & 3) * 32 + lane;
            const int64_t n = static_cast<int64_t>(n_blk) * 128 + row;
            const float b = (args.bias && n < args.N) ? bf16_lo(args.bias[n]) : 0.0f;
            for (int t = rank; t < kNT && m0 + t < args.M; t += splits) {
                float s = 0.0f;
                for (int r = 0; r < splits; ++r) s += ld_cluster_f32(cluster_addr(smem, r) + (t * 128 + row) * 4);
                const int64_t off = (m0 + t) * args.ldy + n;
                if (n < args.N && store_ok(off, 1, args.ext_y, args.err, kSiteLinearMx4))
                    args.Y[off] = __bfloat16_as_ushort(__float2bfloat16_rn(s + b));
            }
        }
        cluster_sync_all();                      // no CTA leaves while its partials are being read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmem);
    }
}

template <int kNT>
int launch_few(const uint8_t* a_codes, const uint8_t* a_sf, const uint8_t* w_codes, const uint8_t* w_sf,
               const Mx4Args& a, cudaStream_t st) {
    using L = FewLayout<kNT>;
    static std::atomic<uint64_t> smem_set{0};
    auto kern = linear_mx4_few_kernel<kNT>;
    if (!set_dynamic_smem_once(kern, L::kSmem, smem_set)) return SVDQ_ERR_CUDA;
    const uint64_t halves = static_cast<uint64_t>(a.K / kMxAtomK) * 2;
    CUtensorMap tw, ta, tsw, tsa;
    if (!encode_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w_codes, a.K / 2, a.N, a.K / 2, 128, 128,
                        CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a_codes, a.K / 2, a.M, a.K / 2, 128, kNT,
                        CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_3d_u8(&tsw, w_sf, 256, halves, (a.N + 127) / 128, 256, halves * 256, 256, 4, 1) ||
        !encode_tmap_3d_u8(&tsa, a_sf, 256, halves, (a.M + 127) / 128, 256, halves * 256, 256, 4, 1))
        return SVDQ_ERR_CUDA;
    const int64_t n_blocks = (a.N + 127) / 128, chunks = (a.M + kNT - 1) / kNT;
    // Slices of K: as many as keep every CTA resident (two per SM), at most 8 (a portable cluster).
    const int64_t sms = device_sm_count() > 0 ? device_sm_count() : 148;
    int splits = 1;
    while (splits < 8 && n_blocks * chunks * splits * 2 <= 2 * sms && splits * 2 <= a.k_stages) splits *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n_blocks * splits), static_cast<unsigned>(chunks), 1);
    cfg.blockDim = dim3(kFewThreads, 1, 1);
    cfg.dynamicSmemBytes = L::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launch_status(cudaLaunchKernelEx(&cfg, kern, tw, ta, tsw, tsa, a, splits));
}

}  // namespace
}  // namespace svdq

extern "C" int svdq_linear_mxfp4(const uint8_t* a_codes, const uint8_t* a_sf, const uint8_t* w_codes,
                                 const uint8_t* w_sf, const void* bias, void* Y, int64_t ldy, int64_t M, int64_t N,
                                 int64_t K, void* stream) {
    using namespace svdq;
    if (a_codes == nullptr || a_sf == nullptr || w_codes == nullptr || w_sf == nullptr || Y == nullptr)
        return SVDQ_ERR_INVALID_ARG;
    if (M < 1 || N < 1 || K < 1 || ldy < N) return SVDQ_ERR_INVALID_ARG;
    if (K % kMxAtomK != 0 || N % 8 != 0) return SVDQ_ERR_UNSUPPORTED;
    if (M > (int64_t(1) << 22) || N > (int64_t(1) << 31) - 256 || K > (int64_t(1) << 30)) return SVDQ_ERR_UNSUPPORTED;
    if (!aligned16(a_codes) || !aligned16(a_sf) || !aligned16(w_codes) || !aligned16(w_sf) || !aligned16(Y) ||
        (ldy * 2) % 16 != 0 || (bias && !aligned16(bias)))
        return SVDQ_ERR_MISALIGNED;
    if (!device_is_sm100()) return SVDQ_ERR_NO_DEVICE;
    if (!debug_ptrs_ok({a_codes, a_sf, w_codes, w_sf, bias, Y})) return SVDQ_ERR_INVALID_ARG;
    Mx4Args a = {};
    a.err = device_error_word();
    if (a.err == nullptr) return SVDQ_ERR_CUDA;
    a.bias = static_cast<const uint16_t*>(bias);
    a.Y = static_cast<uint16_t*>(Y);
    a.ldy = ldy;
    a.M = M;
    a.N = N;
    a.K = K;
    a.k_stages = static_cast<int>((K + kStageK - 1) / kStageK);
    a.ext_y = debug_extent(kSiteLinearMx4, (M - 1) * ldy + N);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (M <= 8) return launch_few<8>(a_codes, a_sf, w_codes, w_sf, a, st);
    if (M <= 16) return launch_few<16>(a_codes, a_sf, w_codes, w_sf, a, st);
    if (M <= 32) return launch_few<32>(a_codes, a_sf, w_codes, w_sf, a, st);
    if (M <= 64) return launch_few<64>(a_codes, a_sf, w_codes, w_sf, a, st);
    return launch_few<128>(a_codes, a_sf, w_codes, w_sf, a, st);
}
