// linear_mx4.cu -- the MXFP4 linear: block-scaled E2M1 x E2M1 GEMM on the tcgen05
// tensor cores (kind::mxf4, one E8M0 scale per 32 elements), bias in the epilogue.
//
//   Y[m, n] = bf16( sum_k dec(A)[m, k] dec(W)[n, k] + bias[n] ),  fp32 accumulation
//
// Up to 64 rows, and up to 128 where K is long (linear_mx4_few_kernel): the weight is what
// has to be read, K/2 + K/32 bytes a row of W.  The MMA takes 128 rows of W as its M operand
// and the activation rows (8 to 128) as its N operand, so no tensor-core row is spent on rows
// that are not there.
// A CTA owns one block of 128 weight rows and a slice of K; the slices of one block are a
// cluster, whose partial sums meet over distributed shared memory in rank order (no
// workspace, no atomics: bitwise repeatable).  One row, 5120 -> 5120: 5.5 us (14 MB; 2.1 us
// at the copy rate, and 3.7 us is what the smallest such call takes: launch, set-up, two
// cluster barriers); 29 rows, 5120 -> 15360: 8.9 us, 4.8 TB/s.
//
// More rows (linear_mx4_pair_kernel): persistent pairs of CTAs walk 256 x 256 tiles
// (256 x 128 where that costs no further wave) with cta_group::2 MMAs, each CTA loading half
// of A's and half of W's rows: 32 KB of codes a 256-channel stage and SM, where one CTA of
// 128 x 256 loads 48.  One thread loads, one issues the MMAs, four warps per CTA move block
// scales into tensor memory, eight read the accumulator out.
//   16384 x 20480 -> 5120  570-600 us (6.0-5.7 PFLOP/s), 650 in a loop that runs into the power limit
//   4096 x 5120 -> 15360   117-120 us (5.5-5.4), 4096 x 5120 -> 5120  43 us (5.0; 4.3 waves of tiles)
// What paces a stage of 256 x 256 x 256, in SM cycles on 16384 x 20480 -> 5120 (80 stages a
// tile), launches 50 ms apart: its MMAs alone 526, its copies alone 448, both 588, with the
// scales 606 (a tile 128 columns wide: 355, 402, 572, 593; neither the number of copies nor a
// deeper ring changes that); 800 more at a tile's end, of which the wait for the shared
// accumulator columns is 620.  Back to back for two seconds a stage takes 636; on 4096 x 5120
// -> 15360 (20 stages a tile) 703 apart and 736 back to back.
// The scales do not go by tcgen05.cp: a copy holds the MMA behind it up by about 45 cycles,
// six a stage (805 us on the first shape), and between the MMAs or a stage ahead it is no
// better (876, 838).
#include <algorithm>

#include "mx.cuh"

namespace svdq {
namespace {

constexpr int kStageK = 256;                     // channels per stage (128 code bytes a row)
constexpr uint32_t kSfAtoms = 1024;              // scale bytes of 128 rows per stage: two atoms

__device__ __forceinline__ uint32_t pack_bf16x2_rn(float lo, float hi) {
    uint32_t out;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out) : "f"(hi), "f"(lo));
    return out;
}

// A bounded wait for a commit's arrival.  The loading threads use it for the last commits of every
// ring slot: no arrival may reach a barrier whose CTA has left, and the commit that the epilogue
// waits for is another, unordered with these.
__device__ __forceinline__ void wait_arrival(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity) && *abort_flag == 0u && clock64() - t0 < kWaitLimitCycles) {}
}

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

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int n_blk = static_cast<int>(blockIdx.x) / splits;
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
                tma_load_2d(st + L::kW, &tmap_a, &full[s], kb * 128, 0);
                tma_load_3d(st + L::kW + L::kA + kSfAtoms, &tmap_sfa, &full[s], 0, kb * 4, 0);
                if (++s == L::kStages) { s = 0; ph ^= 1u; }
            }
            // Bounded drain: a copy may still be in flight where a wait ran out, and the last stages'
            // commits have to arrive while this CTA is here (0.2 us of a one-row call).
            for (int i = (it > L::kStages ? it - L::kStages : 0); i < it; ++i) {
                const long long t0 = clock64();
                while (!mbar_try_wait(&full[i % L::kStages], (i / L::kStages) & 1) &&
                       clock64() - t0 < kWaitLimitCycles) {}
                wait_arrival(&empty[i % L::kStages], (i / L::kStages) & 1, abort_flag);
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
        pdl_wait();                                  // bias may come from the kernel before
        const bool ok = __all_sync(0xffffffffu, mbar_wait(acc_full, 0, abort_flag, args.err, kErrWaitMma));
        tc_fence_after();
        if (ok) {
            // [activation row][weight row], over the ring: every copy has landed and been used
            float* part = reinterpret_cast<float*>(smem) + row;
            constexpr int kC = kNT < 32 ? kNT : 32;
#pragma unroll
            for (int c = 0; c < kNT; c += kC) {
                uint32_t v[kC];
                if constexpr (kC == 8) tmem_ld_32x32b_x8(tbase + c, v);
                else if constexpr (kC == 16) tmem_ld_32x32b_x16(tbase + c, v);
                else tmem_ld_32x32b_x32(tbase + c, v);
                tmem_ld_wait(v);
#pragma unroll
                for (int j = 0; j < kC; ++j) part[(c + j) * 128] = __uint_as_float(v[j]);
            }
        }
    }
    __syncwarp();
    // Every CTA of the cluster sums its share of the activation rows over all ranks, in
    // rank order; a wait that ran out has set the error word and still gets here.
    if (splits > 1) cluster_sync_all();
    else __syncthreads();
    if (warp >= 2) {
        // A warp takes activation rows of this rank in turn, a lane four weight rows of one;
        // kAhead rows' loads are in flight at once (a remote load takes most of a microsecond).
        constexpr int kAhead = kNT <= 8 ? 1 : 4;
        constexpr int kWarps = 4;
        const int64_t n = static_cast<int64_t>(n_blk) * 128 + lane * 4;
        uint2 bb = make_uint2(0u, 0u);
        if (args.bias && n < args.N) bb = *reinterpret_cast<const uint2*>(args.bias + n);
        const float b[4] = {bf16_lo(bb.x), bf16_hi(bb.x), bf16_lo(bb.y), bf16_hi(bb.y)};
        const int rows = static_cast<int>(args.M);
        auto store = [&](int t, const float4& v) {
            const int64_t off = t * args.ldy + n;                        // N % 8 == 0: four columns or none
            if (n < args.N && store_ok(off, 4, args.ext_y, args.err, kSiteLinearMx4))
                *reinterpret_cast<uint2*>(args.Y + off) =
                    make_uint2(pack_bf16x2_rn(v.x + b[0], v.y + b[1]), pack_bf16x2_rn(v.z + b[2], v.w + b[3]));
        };
        if (splits == 1) {
            for (int t = warp - 2; t < rows; t += kWarps)
                store(t, *reinterpret_cast<const float4*>(smem + t * 512 + lane * 16));
        } else {
            for (int t0 = rank + splits * (warp - 2); t0 < rows; t0 += splits * kWarps * kAhead) {
                float4 s[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) s[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
                for (int r = 0; r < splits; r += 2) {            // splits is even; added in rank order
                    float4 p[2][kAhead];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t src = cluster_addr(smem, r + q) + lane * 16;
#pragma unroll
                        for (int j = 0; j < kAhead; ++j) {
                            const int t = t0 + j * splits * kWarps;
                            p[q][j] = t < rows ? ld_cluster_f32x4(src + t * 512) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
#pragma unroll
                        for (int j = 0; j < kAhead; ++j) {
                            s[j].x += p[q][j].x; s[j].y += p[q][j].y; s[j].z += p[q][j].z; s[j].w += p[q][j].w;
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int t = t0 + j * splits * kWarps;
                    if (t < rows) store(t, s[j]);
                }
            }
        }
    }
    __syncwarp();                                // lanes past N skipped their stores; the barrier takes whole warps
    if (splits > 1) cluster_sync_all();          // no CTA leaves while its partials are being read
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmem);
    }
}

template <int kNT>
int launch_few(const uint8_t* a_codes, const uint8_t* a_sf, const uint8_t* w_codes, const uint8_t* w_sf,
               const Mx4Args& args, cudaStream_t st) {
    using L = FewLayout<kNT>;
    Mx4Args a = args;
    a.ext_y = debug_extent(kSiteLinearMx4, args.ext_y);
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
    const int64_t n_blocks = (a.N + 127) / 128;
    // Slices of K, at most 8 (a portable cluster): twice as many while every CTA stays resident
    // (two per SM) and the slices are long enough that the halved loads (0.4 us a stage) are
    // worth another set of partial sums, which cost more the more rows they have.  Columns
    // 1280, us: one row, K 512: 2.8 whole, 3.0 in two; K 5120: 10.3, 6.8, 5.0, 4.6 in 1, 2, 4, 8;
    // 32 rows, K 1280: 5.0, 4.4, 4.7 in 1, 2, 4, K 5120: 5.9 in 4, 6.3 in 8; 64 rows, K 20480: 12.9
    // and 10.4.  One row, 5120 -> 5120: 4 slices 5.3, 8 (which do not fit at once) 9.3.
    const int64_t sms = device_sm_count() > 0 ? device_sm_count() : 148;
    int splits = 1;
    while (splits < 8 && n_blocks * splits * 2 <= 2 * sms &&
           a.k_stages >= (splits == 1 ? 4 : splits == 2 ? 8 : kNT == 8 ? 16 : 64))
        splits *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n_blocks * splits), 1, 1);
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

// ---------------------------------------------------------------------------
// Many rows
// ---------------------------------------------------------------------------
constexpr int kPairThreads = 448;    // warps: 0..3 scale writers, 4..11 epilogue, 12 producer, 13 MMA issuer
constexpr int kPairSfWarps = 4;
constexpr int kPairEpiWarp0 = 4;
constexpr int kPairEpiWarps = 8;
constexpr int kPairLoadWarp = 12;
constexpr int kPairMmaWarp = 13;
static_assert(kPairEpiWarp0 % 4 == 0, "four warps cover the four tensor-memory lane quarters (warp % 4)");
constexpr uint32_t kPairTmem = 512;
constexpr int kTileM = 256;                      // rows of a pair's tile; columns kN: 256 or 128

template <int kN>
struct PairLayout {
    static constexpr int kStages = 5;
    static constexpr int kSfbBlocks = kN == 128 ? 1 : 2;                    // 128-row blocks of W scales a tile touches
    static constexpr uint32_t kA = 128 * 128, kB = kN / 2 * 128;            // this CTA's half of each
    static constexpr uint32_t kOffSfa = kA + kB, kOffSfb = kOffSfa + kSfAtoms;
    static constexpr uint32_t kStage = kOffSfb + kSfbBlocks * kSfAtoms;     // 35 or 26 KB
    static constexpr uint32_t kOffOut = kStages * kStage;                   // a box per epilogue warp:
    static constexpr uint32_t kBox = 32 * 128;                              // 32 rows x 64 bf16 columns
    static constexpr uint32_t kOffBar = kOffOut + kPairEpiWarps * kBox;
    static constexpr uint32_t kOffBias = kOffBar + 256;                     // 2 x 256 bf16
    static constexpr uint32_t kBytes = kOffBias + 2 * 256 * 2;
    static_assert(kStage % 1024 == 0 && kBytes + 1024 <= 232448, "swizzle atoms aligned; one CTA per SM");
    // Tensor memory (512 columns): two accumulators, then one scale buffer per ring slot (A
    // 4 columns per atom, W kN / 32 per atom, two atoms).  With 256 columns the accumulators
    // share 120: the epilogue reads the half that holds them first and lets the next tile start.
    static constexpr uint32_t kSfCols = 8 + 2 * (kN / 32);
    static constexpr uint32_t kSf = kPairTmem - kStages * kSfCols;
    static constexpr bool kShared = kN == 256;
    static constexpr uint32_t kAcc1 = kShared ? kSf - kN : kN;
    static_assert(kAcc1 + kN <= kSf && (!kShared || kAcc1 >= 128), "fits; the shared columns lie in one half of each");
    // more than half an SM's shared memory: never two CTAs waiting for one SM's tensor memory
    static_assert(kBytes > 116 * 1024, "one CTA per SM");
};

struct PairArgs {
    Mx4Args g;
    int m_tiles, n_tiles, n_fastest, band;
    int64_t ext_x, ext_yrow;                     // debug: Y's columns and rows for box origins
};

// Tile -> (row block, column block).  The smaller operand's blocks are walked fastest, in
// bands that stay in L2, so the larger one is read once per band.
__device__ __forceinline__ void pair_tile(const PairArgs& a, int tile, int& m_blk, int& n_blk) {
    const int fast_tiles = a.n_fastest ? a.n_tiles : a.m_tiles;
    const int slow_tiles = a.n_fastest ? a.m_tiles : a.n_tiles;
    const int per_band = a.band * slow_tiles;
    const int b = tile / per_band, r = tile - b * per_band;
    const int width = min(a.band, fast_tiles - b * a.band);
    const int fast = b * a.band + r % width, slow = r / width;
    m_blk = a.n_fastest ? slow : fast;
    n_blk = a.n_fastest ? fast : slow;
}

template <int kN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
linear_mx4_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
                       const __grid_constant__ CUtensorMap tmap_sfa, const __grid_constant__ CUtensorMap tmap_sfw,
                       const __grid_constant__ CUtensorMap tmap_y, const PairArgs args) {
    using L = PairLayout<kN>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);        // the first CTA's are used, by both
    uint64_t* empty = full + L::kStages;
    uint64_t* sf_full = empty + L::kStages;                                 // this CTA's scale bytes have landed
    uint64_t* acc_full = sf_full + L::kStages;
    uint64_t* acc_free = acc_full + 2;                                      // the first CTA's
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_free + 2);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int pair = static_cast<int>(blockIdx.x) >> 1, pairs = static_cast<int>(gridDim.x) >> 1;
    const int tiles = args.m_tiles * args.n_tiles;
    const int k_stages = args.g.k_stages;
    uint32_t* err = args.g.err;

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&full[s], 1 + 2 * kPairSfWarps);      // operand bytes, and both CTAs' scales in tensor memory
            mbar_init(&empty[s], 1);
            mbar_init(&sf_full[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_free[i], 2 * kPairEpiWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kPairMmaWarp) {
        tmem_alloc_pair(tmem_slot, kPairTmem);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                          // both CTAs' barriers and tensor memory are ready
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();

    if (warp == kPairLoadWarp) {
        // ------------------------------------------------------------ producer: this CTA's halves
        if (lane == 0) {
            prefetch_tmap(&tmap_a);
            prefetch_tmap(&tmap_w);
            prefetch_tmap(&tmap_sfa);
            prefetch_tmap(&tmap_sfw);
            pdl_wait();
            const uint64_t keep = l2_evict_last_policy(), once = l2_evict_first_policy();
            const uint64_t pol_a = args.n_fastest ? once : keep, pol_w = args.n_fastest ? keep : once;
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += pairs) {
                int m_blk, n_blk;
                pair_tile(args, tile, m_blk, n_blk);
                for (int kb = 0; kb < k_stages; ++kb) {
                    if (!mbar_wait(&empty[s], ph ^ 1, abort_flag, err, kErrWaitEmpty)) { ok = false; break; }
                    uint8_t* st = smem + s * L::kStage;
                    const uint32_t bar = cluster_addr(&full[s], 0);
                    mbar_arrive_expect_tx(&sf_full[s], (1 + L::kSfbBlocks) * kSfAtoms);
                    tma_load_3d_hint(st + L::kOffSfa, &tmap_sfa, &sf_full[s], 0, kb * 4, m_blk * 2 + rank, pol_a);
                    tma_load_3d_hint(st + L::kOffSfb, &tmap_sfw, &sf_full[s], 0, kb * 4, n_blk * kN / 128, pol_w);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (L::kA + L::kB));     // both CTAs' bytes
                    tma_load_2d_pair(st, &tmap_a, bar, kb * 128, m_blk * kTileM + rank * 128, pol_a);
                    tma_load_2d_pair(st + L::kA, &tmap_w, bar, kb * 128, n_blk * kN + rank * (kN / 2), pol_w);
                    if (++s == L::kStages) { s = 0; ph ^= 1u; }
                }
            }
            if (ok) {                                         // the first CTA's commits arrive in both
#pragma unroll 1
                for (int i = 0; i < L::kStages; ++i) {
                    wait_arrival(&empty[s], ph ^ 1, abort_flag);
                    if (++s == L::kStages) { s = 0; ph ^= 1u; }
                }
            }
            if (!ok) {                                        // a wait ran out: let the copies in flight land (~1 ms)
                const long long t0 = clock64();
                while (clock64() - t0 < 2000000) {}
            }
        }
    } else if (warp == kPairMmaWarp) {
        // ------------------------------------------------------------ MMA issuer (first CTA)
        if (rank == 0 && lane == 0) {
            const uint64_t da0 = desc_kmajor_sw128(smem_u32(smem)), db0 = desc_kmajor_sw128(smem_u32(smem + L::kA));
            int s = 0, t = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += pairs, ++t) {
                // the tile before must have left the shared columns, the one before it this accumulator
                const int r = t - (L::kShared ? 1 : 2);
                if (r >= 0 && !mbar_wait(&acc_free[r & 1], (r >> 1) & 1, abort_flag, err, kErrWaitAccum)) break;
                tc_fence_after();
                const uint32_t acc = tmem + ((t & 1) ? L::kAcc1 : 0u);
                for (int kb = 0; kb < k_stages; ++kb) {
                    if (!mbar_wait(&full[s], ph, abort_flag, err, kErrWaitFull)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t da = da0 + s * (L::kStage >> 4), db = db0 + s * (L::kStage >> 4);
                    const uint32_t sfa = tmem + L::kSf + s * L::kSfCols, sfb = sfa + 8;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_mxf4_pair(acc, da + 2 * kk, db + 2 * kk, idesc_mxf4(kTileM, kN, 2 * (kk & 1)),
                                      sfa + 4 * (kk >> 1), sfb + kN / 32 * (kk >> 1), (kb > 0 || kk > 0) ? 1u : 0u);
                    tc_commit_pair(&empty[s]);
                    if (++s == L::kStages) { s = 0; ph ^= 1u; }
                }
                if (ok) tc_commit_pair(&acc_full[t & 1]);
            }
        }
    } else if (warp < kPairSfWarps) {
        // ------------------------------------------------------------ scale writers
        // One warp per lane quarter copies the stage's scales from shared memory into the
        // slot's tensor-memory buffer: lane i's four words of an atom are rows i, 32 + i, 64 + i
        // and 96 + i.  The MMA reads the W scales of all 256 columns in every quarter, and of
        // the A scales of rows 32 j + i (column j) quarter q only column q.  A slot's scales
        // land after its last MMAs have completed (the producer waited for them), so the
        // buffer is free; the shared memory is refilled after the MMAs that wait for the
        // arrival below, which follows the stores that read these registers.
        const uint32_t tq = tmem + (static_cast<uint32_t>(warp * 32) << 16) + L::kSf;
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int tile = pair; tile < tiles && ok; tile += pairs) {
            for (int kb = 0; kb < k_stages; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(&sf_full[s], ph, abort_flag, err, kErrWaitFull))) {
                    ok = false;
                    break;
                }
                const uint8_t* sfa = smem + s * L::kStage + L::kOffSfa;
                const uint8_t* sfb = smem + s * L::kStage + L::kOffSfb;
                const uint32_t base = tq + s * L::kSfCols;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    tmem_st_32x32b_x1(base + 4 * i + warp,
                                      *reinterpret_cast<const uint32_t*>(sfa + i * 512 + lane * 16 + warp * 4));
                    const uint32_t dst = base + 8 + kN / 32 * i;
                    const uint4 x = *reinterpret_cast<const uint4*>(sfb + i * 512 + lane * 16);
                    if constexpr (kN == 128) {
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                        tmem_st_32x32b_x4(dst, w);
                    } else {
                        const uint4 y = *reinterpret_cast<const uint4*>(sfb + kSfAtoms + i * 512 + lane * 16);
                        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                        tmem_st_32x32b_x8(dst, w);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(&full[s], 0));
                if (++s == L::kStages) { s = 0; ph ^= 1u; }
            }
        }
    } else if (warp < kPairEpiWarp0 + kPairEpiWarps) {
        // ------------------------------------------------------------ epilogue: this CTA's 128 rows
        const int ew = warp - kPairEpiWarp0;
        const int quarter = warp & 3, half = ew >> 2;        // lane quarter; which 64 of each 128 columns
        const int etid = ew * 32 + lane;
        uint16_t* bias_s = reinterpret_cast<uint16_t*>(smem + L::kOffBias);
        uint8_t* box = smem + L::kOffOut + ew * L::kBox;
        const uint32_t free_bar = cluster_addr(acc_free, 0);
        const uint64_t pol_y = l2_evict_first_policy();
        pdl_wait();                                          // bias may come from the kernel before
        int t = 0;
        for (int tile = pair; tile < tiles; tile += pairs, ++t) {
            int m_blk, n_blk;
            pair_tile(args, tile, m_blk, n_blk);
            uint16_t* bt = bias_s + (t & 1) * 256;
            const int64_t bn = static_cast<int64_t>(n_blk) * kN + etid;
            bt[etid] = (args.g.bias && etid < kN && bn < args.g.N) ? args.g.bias[bn] : static_cast<uint16_t>(0);
            __syncwarp();                                     // the barrier takes whole warps
            if (bar_sync_or<1, kPairEpiWarps * 32>(*abort_flag != 0u)) break;
            if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[t & 1], (t >> 1) & 1, abort_flag, err, kErrWaitMma)))
                continue;
            tc_fence_after();
            const uint32_t tbase = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + ((t & 1) ? L::kAcc1 : 0u);
            const int32_t row0 = m_blk * kTileM + rank * 128 + quarter * 32;
            // 64 columns at a time.  256 columns: the shared ones lie in the last half of
            // accumulator 0 and in the first of accumulator 1; that half is read first, by
            // all warps, then the next tile may start.
            constexpr int pieces = kN / 128;
#pragma unroll 1
            for (int i = 0; i < pieces; ++i) {
                const int col = (L::kShared ? (((t & 1) ^ i) ? 0 : 128) : 128 * i) + half * 64;
                uint32_t v[2][32];
                tmem_ld_32x32b_x32(tbase + col, v[0]);
                tmem_ld_32x32b_x32(tbase + col + 32, v[1]);
                tmem_ld_wait(v[0]);
                tmem_ld_tie(v[1]);
                if (i == (L::kShared ? 0 : pieces - 1)) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(free_bar + 8 * (t & 1));
                }
                if (lane == 0) bulk_wait_read_all();                 // the previous box has left the buffer
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t bb = *reinterpret_cast<const uint32_t*>(bt + col + 8 * c + 2 * j);
                        const uint32_t* w = v[c >> 2] + 8 * (c & 3) + 2 * j;
                        o[j] = pack_bf16x2_rn(__uint_as_float(w[0]) + bf16_lo(bb), __uint_as_float(w[1]) + bf16_hi(bb));
                    }
                    // 128-byte swizzle: 16-byte piece c of row r sits at c ^ (r % 8)
                    *reinterpret_cast<uint4*>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
                fence_async_shared();
                __syncwarp();
                const int64_t x = static_cast<int64_t>(n_blk) * kN + col;
                if (lane == 0 && row0 < args.g.M && x < args.g.N &&          // boxes wholly past M or N are skipped
                    box_ok(x, row0, args.ext_x, args.ext_yrow, err, kSiteLinearMx4)) {
                    tma_store_2d_hint(&tmap_y, box, static_cast<int32_t>(x), row0, pol_y);
                    bulk_commit_group();
                }
                __syncwarp();                                // the next read of tensor memory takes the whole warp
            }
        }
        if (lane == 0) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                          // no remote arrival, copy or MMA of the pair is left
    if (warp == kPairMmaWarp) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kPairTmem);
    }
}

template <int kN>
int launch_pair(const uint8_t* a_codes, const uint8_t* a_sf, const uint8_t* w_codes, const uint8_t* w_sf,
                const Mx4Args& g, cudaStream_t st) {
    using L = PairLayout<kN>;
    static std::atomic<uint64_t> smem_set{0};
    constexpr uint32_t smem = L::kBytes + 1024;
    if (!set_dynamic_smem_once(linear_mx4_pair_kernel<kN>, smem, smem_set)) return SVDQ_ERR_CUDA;
    const uint64_t halves = static_cast<uint64_t>(g.K / kMxAtomK) * 2;
    CUtensorMap ta, tw, tsa, tsw, ty;
    if (!encode_tmap_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a_codes, g.K / 2, g.M, g.K / 2, 128, 128,
                        CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w_codes, g.K / 2, g.N, g.K / 2, 128, kN / 2,
                        CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_3d_u8(&tsa, a_sf, 256, halves, (g.M + 127) / 128, 256, halves * 256, 256, 4, 1) ||
        !encode_tmap_3d_u8(&tsw, w_sf, 256, halves, (g.N + 127) / 128, 256, halves * 256, 256, 4, L::kSfbBlocks) ||
        !encode_tmap_2d(&ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.Y, g.N, g.M, g.ldy * 2, 64, 32,
                        CU_TENSOR_MAP_SWIZZLE_128B))
        return SVDQ_ERR_CUDA;
    PairArgs a = {};
    a.g = g;
    a.m_tiles = static_cast<int>((g.M + kTileM - 1) / kTileM);
    a.n_tiles = static_cast<int>((g.N + kN - 1) / kN);
    a.n_fastest = g.N <= g.M ? 1 : 0;
    {
        // A band of at most 40 MB of the operand walked fastest: each die's half of the L2
        // holds it beside the other operand's blocks in flight.
        constexpr int64_t kBandBytes = int64_t(40) << 20;
        const int64_t fast = a.n_fastest ? a.n_tiles : a.m_tiles;
        const int64_t bands = (fast * (a.n_fastest ? kN : kTileM) * (g.K / 2) + kBandBytes - 1) / kBandBytes;
        a.band = static_cast<int>((fast + bands - 1) / bands);
    }
    a.ext_x = debug_extent(kSiteLinearMx4, g.N);
    a.ext_yrow = g.M;
    const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    if (tiles > 0x3FFFFFFF) return SVDQ_ERR_UNSUPPORTED;
    const int64_t sms = device_sm_count() > 1 ? device_sm_count() : 148;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(tiles, sms / 2)), 1, 1);
    cfg.blockDim = dim3(kPairThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, linear_mx4_pair_kernel<kN>, ta, tw, tsa, tsw, ty, a));
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
    a.ext_y = (M - 1) * ldy + N;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // The MMA's N operand is the rows themselves up to 64 of them, and up to 128 where K is
    // long: a pair's 256-row tile has no partial sums to add but reads K unsliced (128 rows,
    // 1280 -> 1280: 6.7 us sliced, 5.1 in a pair; 115 rows, 5120 -> 5120: 10.8 and 10.2, 20480 -> 5120:
    // 17.8 and 29; 64 rows, 5120 -> 5120: 8.4 and 9.9).
    if (M <= 8) return launch_few<8>(a_codes, a_sf, w_codes, w_sf, a, st);
    if (M <= 16) return launch_few<16>(a_codes, a_sf, w_codes, w_sf, a, st);
    if (M <= 32) return launch_few<32>(a_codes, a_sf, w_codes, w_sf, a, st);
    if (M <= 64) return launch_few<64>(a_codes, a_sf, w_codes, w_sf, a, st);
    if (M <= 128 && a.k_stages > 16) return launch_few<128>(a_codes, a_sf, w_codes, w_sf, a, st);
    // A stage takes about 600 cycles whatever the tile's width, so the narrow tile pays only
    // where it costs no further wave: there it has half the epilogue and twice the pairs at
    // work (256 x 5120 -> 5120: 10.4 against 11.9 us, 515 x 1920 -> 1160: 6.2 against 8.3;
    // 4096 x 5120 -> 5120: 69 against 43).
    const int64_t pairs = std::max(device_sm_count() / 2, 1), m_tiles = (M + kTileM - 1) / kTileM;
    const int64_t waves = (m_tiles * ((N + 255) / 256) + pairs - 1) / pairs;
    const int64_t waves128 = (m_tiles * ((N + 127) / 128) + pairs - 1) / pairs;
    if (waves < waves128) return launch_pair<256>(a_codes, a_sf, w_codes, w_sf, a, st);
    return launch_pair<128>(a_codes, a_sf, w_codes, w_sf, a, st);
}
