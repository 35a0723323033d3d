// mx_gemm.cu - grouped product of microscaled 4-bit operands on the block-scaled
// tensor cores (sm_100a tcgen05 kind::mxf4 and kind::mxf4nvf4).
//
//   out[r][n] = act( alpha_g 2^e sum_k A[r][k] W[g][n][k] + bias[g][n] ),  g = group of row r,
//
// A and W being 4-bit codes times their blocks' scales; the sum is held in
// fp32 and rounded once, to the output's type.
//
// Operand roles. The MMA's M side is 128 output features (rows of W[g]) and its
// N side a token tile of up to TILE rows of one group, so a group of a few rows
// costs an MMA of a few columns.
// Unit = (token tile, feature tile); every CTA builds the groups' tile prefix in
// shared memory and takes units cta, cta + grid, ...
//
// Per CTA (192 threads): warp 0 loads codes (TMA, 128B swizzle, 256 elements
// of K a stage) and scale tiles (bulk copies), warp 1 owns TMEM, copies the
// scale tiles of a stage into TMEM (tcgen05.cp) and issues its MMAs, warps 2..5
// drain the accumulator (lane = feature, column = token).
//
// TMEM (512 columns): two accumulators of up to 192 columns, and two buffers of
// scale columns. A scale buffer is filled again once the MMAs two stages back
// have completed (their stage's commit), so no copy passes an MMA that reads it.
// A token tile starts at a multiple of 64 rows of the 128-row scale tiles, so
// its first scale column is 0 or 2.
//
// Every wait is bounded; a role that gives up sets the block's status word, the
// others stop, and the block ends after its copies and MMAs have drained.
#include <algorithm>

#include "mx_common.cuh"

namespace moe {
namespace {

constexpr int kEpiWarps = 4;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kFeat = 128;                // features per unit (MMA M)
constexpr int kStageK = 256;              // elements of K per stage: 128 bytes of codes
constexpr int kWBytes = kFeat * 128;      // weight codes per stage
constexpr int kMaxGroups = 1024;
constexpr int kTmemCols = 512;
constexpr int kAccStride = 192;           // columns between the two accumulators
constexpr int kScaleCol = 2 * kAccStride; // first scale column

template <int FMT, int TILE>
struct Cfg {
    static constexpr int kSfTiles = kStageK / MxFormat<FMT>::kTileK;  // scale tiles along K per stage
    static constexpr int kRowBlocks = TILE > 64 ? 2 : 1;              // 128-row scale tiles under a token tile
    static constexpr int kSfA = kSfTiles * 512;                       // weight scales
    static constexpr int kSfB = kRowBlocks * kSfTiles * 512;          // token scales
    static constexpr int kB = TILE * 128;
    static constexpr int kStage = kWBytes + kB + kSfA + kSfB;
    static constexpr int kFixed = 1024 + 512 + (kMaxGroups + 1) * 4 + 64;
    static constexpr int kStages = (232448 - kFixed) / kStage < 12 ? (232448 - kFixed) / kStage : 12;
    static constexpr int kSmem = kFixed + kStages * kStage;
    static constexpr int kSfColsA = kSfTiles * 4, kSfColsB = kSfTiles * 4 * kRowBlocks;
    static constexpr int kSfCols = kSfColsA + kSfColsB;               // scale columns of one buffer
    static_assert(kScaleCol + 2 * kSfCols <= kTmemCols, "scale columns");
    static_assert(kStage % 1024 == 0 || kStage % 512 == 0, "stage alignment");
    static_assert(kB % 1024 == 0, "operand tiles keep the 1024-byte swizzle alignment");
};

struct Unit {
    int g, row0, ntok, feat0;
};

template <int FMT, int TILE>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                   const MxGemmArgs a) {
    using C = Cfg<FMT, TILE>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sW = base, *sT = sW + kStages * kWBytes;
    uint8_t *sSfW = sT + kStages * C::kB, *sSfT = sSfW + kStages * C::kSfA;
    uint64_t *full = reinterpret_cast<uint64_t *>(sSfT + kStages * C::kSfB);
    uint64_t *empty = full + kStages, *tfull = empty + kStages, *tempty = tfull + 2, *mma_done = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    uint32_t *status = tmem_slot + 1;
    int32_t *scan = reinterpret_cast<int32_t *>(tmem_slot + 2);    // [8]
    int32_t *prefix = scan + 8;                                    // [G + 1] token tiles before each group
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_a);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], kEpiWarps);
        }
        mbar_init(mma_done, 1);
        *status = kDevOk;
        prefix[0] = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    // Token tiles before each group: a scan over the groups, kThreads at a time.
    for (int g0 = 0, carry = 0; g0 < a.G; g0 += kThreads) {
        const int g = g0 + threadIdx.x;
        int v = 0;
        if (g < a.G) {
            const int start = a.group_start ? a.group_start[g] : 0;
            const int rows = a.group_rows ? a.group_rows[g] : a.rows;
            // A segment that is not where the layout allows it is not computed.
            const bool fits = rows >= 0 && start >= 0 && start % 128 == 0 && start <= a.rows && rows <= a.rows - start;
            if (!fits && rows != 0) atomicOr(status, kDevBadGroup);
            v = fits ? (rows + TILE - 1) / TILE : 0;
        }
        int s = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += o;
        }
        if (lane == 31) scan[warp] = s;
        __syncthreads();
        int before = carry, total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += scan[w];
            total += scan[w];
        }
        if (g < a.G) prefix[g + 1] = before + s;
        carry += total;
        __syncthreads();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    // A bad group is reported and skipped; it does not stop the roles.
    const uint32_t bad = *status & kDevBadGroup;
    __syncthreads();
    if (threadIdx.x == 0) *status = kDevOk;
    __syncthreads();

    const int n_ft = (a.N + kFeat - 1) / kFeat;
    const int64_t total = (int64_t)prefix[a.G] * n_ft;
    const int kblocks = (a.K + kStageK - 1) / kStageK;
    const int SB = mx_scale_tiles(a.K, MxFormat<FMT>::kBlock);
    auto unit_of = [&](int64_t u) {
        const int tt = static_cast<int>(u / n_ft);
        int lo = 0, hi = a.G - 1;  // the last group whose prefix is <= tt
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= tt) lo = mid;
            else hi = mid - 1;
        }
        const int start = a.group_start ? a.group_start[lo] : 0;
        const int rows = a.group_rows ? a.group_rows[lo] : a.rows;
        const int off = (tt - prefix[lo]) * TILE;
        return Unit{lo, start + off, min(TILE, rows - off), static_cast<int>(u - (int64_t)tt * n_ft) * kFeat};
    };
    bool ok = true;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        const int NB = (a.N + 127) / 128;
        uint32_t it = 0;
        for (int64_t u = blockIdx.x; u < total && ok; u += gridDim.x) {
            const Unit w = unit_of(u);
            const int n16 = (w.ntok + 15) / 16;
            const int rb0 = w.row0 / 128, nrb = (w.row0 % 128 + w.ntok + 127) / 128;
            const int64_t wrow = (int64_t)w.g * a.N + w.feat0;
            const uint8_t *sfw = a.w_scales + ((int64_t)w.g * NB + w.feat0 / 128) * SB * 512;
            const uint8_t *sft = a.a_scales + (int64_t)rb0 * SB * 512;
            for (int kb = 0; kb < kblocks; ++kb, ++it) {
                const int st = it % kStages;
                const uint32_t ph = (it / kStages) & 1u;
                int got = 1;
                if (lane == 0) got = mbar_wait(&empty[st], ph ^ 1u, status) ? 1 : 0;
                if (!__shfl_sync(0xffffffffu, got, 0)) {
                    ok = false;
                    break;
                }
                const int sft_n = min(C::kSfTiles, SB - kb * C::kSfTiles);
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[st], kWBytes + n16 * 2048 + (1 + nrb) * sft_n * 512);
                __syncwarp();
                if (lane == 0) tma_load_2d(&map_w, &full[st], sW + st * kWBytes, kb * 128, static_cast<int>(wrow));
                if (lane < n16)
                    tma_load_2d(&map_a, &full[st], sT + st * C::kB + lane * 2048, kb * 128, w.row0 + lane * 16);
                const int64_t so = (int64_t)kb * C::kSfTiles * 512;
                if (lane == 16) bulk_load(sSfW + st * C::kSfA, sfw + so, sft_n * 512, &full[st]);
                if (lane >= 17 && lane - 17 < nrb) {
                    const int b = lane - 17;
                    bulk_load(sSfT + st * C::kSfB + b * C::kSfTiles * 512, sft + (int64_t)b * SB * 512 + so,
                              sft_n * 512, &full[st]);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        if (lane == 0) {
            uint32_t it = 0, tcount = 0;
            for (int64_t u = blockIdx.x; u < total && ok; u += gridDim.x, ++tcount) {
                const Unit w = unit_of(u);
                const int nrb = (w.row0 % 128 + w.ntok + 127) / 128;
                const uint32_t idesc = mx_idesc<FMT>(kFeat, (w.ntok + 15) / 16 * 16);
                const uint32_t shift = (w.row0 % 128) / 32;  // first scale column of the tile
                const uint32_t acc = tcount & 1u, use = tcount >> 1;
                if (!mbar_wait(&tempty[acc], (use & 1u) ^ 1u, status)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d = tmem_base + acc * kAccStride;
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const int st = it % kStages;
                    if (!mbar_wait(&full[st], (it / kStages) & 1u, status)) {
                        ok = false;
                        break;
                    }
                    // The scale buffer's previous MMAs (two stages back) are done.
                    if (it >= 2 && !mbar_wait(&empty[(it - 2) % kStages], ((it - 2) / kStages) & 1u, status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t sfa = tmem_base + kScaleCol + (it & 1u) * C::kSfCols, sfb = sfa + C::kSfColsA;
                    const int sft_n = min(C::kSfTiles, SB - kb * C::kSfTiles);
                    for (int j = 0; j < sft_n; ++j) {
                        tc_cp_scales<1>(sfa + 4 * j, scale_tile_desc(smem_u32(sSfW + st * C::kSfA + j * 512)));
                        for (int b = 0; b < nrb; ++b)
                            tc_cp_scales<1>(sfb + (j * C::kRowBlocks + b) * 4,
                                            scale_tile_desc(smem_u32(sSfT + st * C::kSfB +
                                                                     (b * C::kSfTiles + j) * 512)));
                    }
                    const uint64_t ad = sw128_kmajor_desc(smem_u32(sW + st * kWBytes));
                    const uint64_t bd = sw128_kmajor_desc(smem_u32(sT + st * C::kB));
                    const int steps = (min(kStageK, a.K - kb * kStageK) + 63) / 64;
                    for (int kk = 0; kk < steps; ++kk) {
                        // 64 elements: half of an MXFP4 scale tile's 4 scales, a whole NVFP4 one's.
                        const int j = FMT == kMxFp4 ? kk / 2 : kk;
                        const uint32_t id = FMT == kMxFp4 ? 2u * (kk & 1) : 0u;
                        tc_mma_mx<FMT, 1>(d, ad + 2u * kk, bd + 2u * kk, idesc | mx_idesc_sf(id), sfa + 4 * j,
                                          sfb + j * C::kRowBlocks * 4 + shift, (kb | kk) != 0 ? 1u : 0u);
                    }
                    tc_commit(&empty[st]);
                }
                if (ok) tc_commit(&tfull[acc]);
            }
            tc_commit(mma_done);
            mbar_wait_drain(mma_done, 0u);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;  // the TMEM lane quarter this warp may read
        uint32_t tcount = 0;
        for (int64_t u = blockIdx.x; u < total; u += gridDim.x, ++tcount) {
            const Unit w = unit_of(u);
            const uint32_t acc = tcount & 1u, use = tcount >> 1;
            int got = 1;
            if (lane == 0) got = mbar_wait_idle(&tfull[acc], use & 1u, status) ? 1 : 0;
            if (!__shfl_sync(0xffffffffu, got, 0)) break;
            tc_fence_after_sync();
            const int f = w.feat0 + q * 32 + lane;
            const bool fok = f < a.N;
            const float mul = a.post * (a.alpha ? __ldg(a.alpha + w.g) : 1.f);
            const float bv = fok && a.bias ? __ldg(a.bias + (int64_t)w.g * a.N + f) : 0.f;
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * kAccStride;
            const uint32_t odd = lane & 1u;
            for (int c = 0; c < w.ntok; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(taddr + c, r);
                tmem_ld_wait();
                float z[16];
#pragma unroll
                for (int t = 0; t < 16; ++t) z[t] = activate(a.act, fmaf(__uint_as_float(r[t]), mul, bv));
                if (a.out_f32) {
                    float *o = static_cast<float *>(a.out) + (int64_t)(w.row0 + c) * a.out_ld + f;
#pragma unroll
                    for (int t = 0; t < 16; ++t)
                        if (fok && c + t < w.ntok) o[t * a.out_ld] = z[t];
                } else if (!a.wide_ok) {
                    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.out) + (int64_t)(w.row0 + c) * a.out_ld + f;
#pragma unroll
                    for (int t = 0; t < 16; ++t)
                        if (fok && c + t < w.ntok) o[t * a.out_ld] = __float2bfloat16_rn(z[t]);
                } else {
                    // Neighbouring lanes trade values: the even lane stores features (f, f + 1) of
                    // token t, the odd lane those (f - 1, f) of token t + 1.
                    __nv_bfloat16 *o =
                        static_cast<__nv_bfloat16 *>(a.out) + (int64_t)(w.row0 + c + odd) * a.out_ld + (f & ~1);
#pragma unroll
                    for (int t = 0; t < 16; t += 2) {
                        const float other = __shfl_xor_sync(0xffffffffu, odd ? z[t] : z[t + 1], 1);
                        const __nv_bfloat162 p =
                            odd ? __floats2bfloat162_rn(other, z[t + 1]) : __floats2bfloat162_rn(z[t], other);
                        if (c + t + static_cast<int>(odd) < w.ntok) {
                            if ((f | 1) < a.N) *reinterpret_cast<__nv_bfloat162 *>(o + t * a.out_ld) = p;
                            else if ((f & ~1) < a.N) o[t * a.out_ld] = p.x;
                        }
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[acc]);
        }
    }

    // A role that gave up may leave loads in flight: let them land.
    if (!ok || *reinterpret_cast<volatile uint32_t *>(status) != kDevOk) spin_ns(1000000ull);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem_base, kTmemCols);
    if (threadIdx.x == 0 && a.status) {
        const uint32_t v = *status | bad;
        if (v) atomicOr(a.status, v);
    }
}

template <int FMT, int TILE>
cudaError_t launch(const CUtensorMap &mw, const CUtensorMap &ma, const MxGemmArgs &a, int num_sms, cudaStream_t s) {
    using C = Cfg<FMT, TILE>;
    cudaError_t e = set_smem_limit_once<mx_gemm_kernel<FMT, TILE>>(C::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t most = ((int64_t)a.rows / TILE + a.G) * ((a.N + kFeat - 1) / kFeat);
    const int grid = static_cast<int>(std::min<int64_t>(most, num_sms));
    mx_gemm_kernel<FMT, TILE><<<grid, kThreads, C::kSmem, s>>>(mw, ma, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_gemm(const CUtensorMap &map_w, const CUtensorMap &map_a, const MxGemmArgs &a, int format,
                           int num_sms, cudaStream_t s) {
    // Short segments: rows beyond the 127 that each group's start may leave unused.
    const int64_t filled = (int64_t)a.rows - (a.G > 1 ? (int64_t)a.G * 127 : 0);
    const bool narrow = filled <= (int64_t)64 * a.G;
    if (format == kMxFp4)
        return narrow ? launch<kMxFp4, 64>(map_w, map_a, a, num_sms, s) : launch<kMxFp4, 192>(map_w, map_a, a, num_sms, s);
    return narrow ? launch<kNvFp4, 64>(map_w, map_a, a, num_sms, s) : launch<kNvFp4, 192>(map_w, map_a, a, num_sms, s);
}

}  // namespace moe
