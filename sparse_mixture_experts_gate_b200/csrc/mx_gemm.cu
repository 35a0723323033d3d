// mx_gemm.cu - grouped product of microscaled 4-bit operands on the block-scaled
// tensor cores (sm_100a tcgen05 kind::mxf4 and kind::mxf4nvf4).
//
//   out[r][n] = act( alpha_g 2^e sum_k A[r][k] W[g][n][k] + bias[g][n] ),  g = group of row r,
//
// A and W being 4-bit codes times their blocks' scales; the sum is held in
// fp32 and rounded once, to the output's type.
//
// Operand roles. The MMA's M side is the output features (rows of W[g]) and its
// N side a token tile of up to TILE rows of one group, so a group of a few rows
// costs an MMA of a few columns. Unit = (token tile, feature tile); every CTA
// builds the groups' tile prefix in shared memory and takes its share of the
// units in steps of the grid.
//
// Two forms. Long segments run on CTA pairs (cta_group::2): 256 features x 192
// tokens, each CTA staging its 128 weight rows and half of the tokens, because
// the operands' way from L2 is what bounds them. Short segments (a few tokens for
// each expert: the weights' bytes bound them) run on single CTAs with 128
// features x up to 64 tokens and a deeper pipeline.
//
// Per CTA (320 threads): warp 0 loads codes (TMA, 128B swizzle, 256 elements
// of K a stage) and scale tiles, signalling the (leader's) stage barrier; warp
// 1 owns TMEM and, in the leader, copies a stage's scale tiles into TMEM
// (tcgen05.cp, both CTAs') and issues its MMAs; warps 2..9 drain this CTA's 128
// features of the accumulator, two warps for each quarter of the TMEM lanes.
//
// TMEM (512 columns): two accumulators of TILE columns and, in the rest, as many
// buffers of scale columns as there are stages, or fit: then a buffer is
// filled again only once the MMAs that read it have completed (their stage's
// commit), so no copy passes an MMA. A token tile starts at a multiple of 64 rows
// of the 128-row scale tiles, so its first scale column is 0 or 2.
//
// Epilogue of bf16 outputs: TMEM is read in 16 x 256-bit pieces, whose register
// layout (a lane holds two neighbouring tokens of one feature) is the one that
// stmatrix.trans takes, so a warp turns 32 tokens x 32 features around through a
// shared buffer of its own without shuffles, and stores each token's 64 bytes
// with 16-byte stores. fp32 outputs are stored from lane = feature directly.
//
// Every wait is bounded; a role that gives up sets the block's status word, the
// others stop, and the block ends after its copies and MMAs have drained.
#include <algorithm>

#include "mx_common.cuh"

namespace moe {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kFeat = 128;                // features per CTA
constexpr int kStageK = 256;              // elements of K per stage: 128 bytes of codes
constexpr int kWBytes = kFeat * 128;      // weight codes per stage
constexpr int kMaxGroups = 1024;
constexpr int kTmemCols = 512;
constexpr int kPitch = 80;                // bytes of a staged token row (64 used): conflict-free stmatrix
constexpr int kStageOut = 32 * kPitch;    // one warp's output buffer
constexpr int kActRuntime = -2;           // fp32 outputs: the activation is looked up at run time

template <int FMT, int TILE, int CG>
struct Cfg {
    static constexpr int kSfTiles = kStageK / MxFormat<FMT>::kTileK;  // scale tiles along K per stage
    static constexpr int kRowBlocks = TILE > 64 ? 2 : 1;              // 128-row scale tiles under a token tile
    static constexpr int kSfA = kSfTiles * 512;                       // weight scales
    static constexpr int kSfB = kRowBlocks * kSfTiles * 512;          // token scales
    static constexpr int kB = TILE / CG * 128;
    static constexpr int kStage = kWBytes + kB + kSfA + kSfB;
    static constexpr int kFixed = 1024 + kEpiWarps * kStageOut + 512 + (kMaxGroups + 1) * 4 + 128;
    static constexpr int kFit = (232448 - kFixed) / kStage;
    static constexpr int kStages = kFit < 12 ? kFit : 12;
    static constexpr int kSmem = kFixed + kStages * kStage;
    static constexpr int kSfColsA = kSfTiles * 4, kSfColsB = kSfTiles * 4 * kRowBlocks;
    static constexpr int kSfCols = kSfColsA + kSfColsB;               // scale columns of one buffer
    static constexpr int kScaleCol = 2 * TILE;                        // first scale column
    static constexpr int kSfFit = (kTmemCols - kScaleCol) / kSfCols;
    static constexpr int kSfBufs = kSfFit < kStages ? kSfFit : kStages;
    static constexpr int kStep = 16 * CG;                             // token rows: a TMA box per CTA
    static_assert(kStages >= 4 && kSfBufs >= 2, "pipeline depth");
    static_assert(kB % 1024 == 0, "operand tiles keep the 1024-byte swizzle alignment");
};

struct Unit {
    int g, row0, ntok, feat0;
};

__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Four 8 x 8 matrices of 16-bit values, transposed: lane 8 m + i gives the address of row i of matrix m.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

template <int FMT, int TILE, int CG, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ MxMaps m, const MxGemmArgs a) {
    using C = Cfg<FMT, TILE, CG>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sW = base, *sT = sW + kStages * kWBytes;
    uint8_t *sSfW = sT + kStages * C::kB, *sSfT = sSfW + kStages * C::kSfA;
    uint8_t *sOut = sSfT + kStages * C::kSfB;
    uint64_t *full = reinterpret_cast<uint64_t *>(sOut + kEpiWarps * kStageOut);
    uint64_t *empty = full + kStages, *tfull = empty + kStages, *tempty = tfull + 2, *mma_done = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    uint32_t *status = tmem_slot + 1;
    int32_t *scan = reinterpret_cast<int32_t *>(tmem_slot + 2);    // [16]
    int32_t *prefix = scan + 16;                                   // [G + 1] token tiles before each group
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&m.w);
        tma_prefetch_desc(&m.a);
        tma_prefetch_desc(&m.sw);
        tma_prefetch_desc(&m.sa);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], CG * kEpiWarps);
        }
        mbar_init(mma_done, 1);
        *status = kDevOk;
        prefix[0] = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (warp == 1) {
        if constexpr (CG == 2) {
            tmem_alloc_pair(tmem_slot, kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, kTmemCols);
            tmem_relinquish();
        }
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
    // A bad group is reported and skipped; it does not stop the roles.
    const uint32_t bad = *status & kDevBadGroup;
    __syncthreads();
    if (threadIdx.x == 0) *status = kDevOk;
    tc_fence_before_sync();
    if constexpr (CG == 2) cluster_sync_all();  // both CTAs' barriers and TMEM are ready
    else __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;

    const int n_ft = (a.N + kFeat * CG - 1) / (kFeat * CG);
    const int total = prefix[a.G] * n_ft;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;
    const int kblocks = (a.K + kStageK - 1) / kStageK;
    auto unit_of = [&](int u) {
        const int tt = u / n_ft;
        int lo = 0, hi = a.G - 1;  // the last group whose prefix is <= tt
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= tt) lo = mid;
            else hi = mid - 1;
        }
        const int start = a.group_start ? a.group_start[lo] : 0;
        const int rows = a.group_rows ? a.group_rows[lo] : a.rows;
        const int off = (tt - prefix[lo]) * TILE;
        return Unit{lo, start + off, min(TILE, rows - off), (u - tt * n_ft) * kFeat * CG};
    };
    auto commit_all = [&](uint64_t *bar) {
        if constexpr (CG == 2) tc_commit_pair_mc(bar, 0x3);
        else tc_commit(bar);
    };
    bool ok = true;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        const int NB = (a.N + 127) / 128;
        uint32_t it = 0;
        for (int u = first; u < total && ok; u += step) {
            const Unit w = unit_of(u);
            const int boxes = (w.ntok + C::kStep - 1) / C::kStep;  // 16-row boxes of this CTA
            const int nrb = (w.row0 % 128 + w.ntok + 127) / 128;
            const int feat = w.feat0 + static_cast<int>(rank) * kFeat;
            const int wrow = w.g * a.N + feat, trow = w.row0 + static_cast<int>(rank) * boxes * 16;
            // The second CTA of a last feature tile may have no weight scales: it reads the group's last ones.
            const int wblk = w.g * NB + min(feat / 128, NB - 1), tblk = w.row0 / 128;
            const uint32_t bytes = CG * (kWBytes + boxes * 2048 + C::kSfA + nrb * C::kSfTiles * 512);
            for (int kb = 0; kb < kblocks; ++kb, ++it) {
                const int st = it % kStages;
                const uint32_t ph = (it / kStages) & 1u;
                int got = 1;
                if (lane == 0) got = mbar_wait(&empty[st], ph ^ 1u, status) ? 1 : 0;
                if (!__shfl_sync(0xffffffffu, got, 0)) {
                    ok = false;
                    break;
                }
                if (lane == 0 && leader) mbar_arrive_expect_tx(&full[st], bytes);
                __syncwarp();
                auto load = [&](const CUtensorMap *map, void *dst, int x, int y) {
                    if constexpr (CG == 2) tma_load_2d_pair(map, mapa_shared(smem_u32(&full[st]), 0), dst, x, y);
                    else tma_load_2d(map, &full[st], dst, x, y);
                };
                if (lane == 0) load(&m.w, sW + st * kWBytes, kb * 128, wrow);
                if (lane < boxes) load(&m.a, sT + st * C::kB + lane * 2048, kb * 128, trow + lane * 16);
                if (lane == 16) load(&m.sw, sSfW + st * C::kSfA, kb * C::kSfTiles * 64, wblk);
                if (lane >= 17 && lane - 17 < nrb)
                    load(&m.sa, sSfT + st * C::kSfB + (lane - 17) * C::kSfTiles * 512, kb * C::kSfTiles * 64,
                         tblk + lane - 17);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA (leader)
        if (leader && lane == 0) {
            uint32_t it = 0, tcount = 0;
            for (int u = first; u < total && ok; u += step, ++tcount) {
                const Unit w = unit_of(u);
                const int nrb = (w.row0 % 128 + w.ntok + 127) / 128;
                const uint32_t idesc = mx_idesc<FMT>(kFeat * CG, (w.ntok + C::kStep - 1) / C::kStep * C::kStep);
                const uint32_t shift = (w.row0 % 128) / 32;  // first scale column of the tile
                const uint32_t acc = tcount & 1u, use = tcount >> 1;
                if (!mbar_wait(&tempty[acc], (use & 1u) ^ 1u, status)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d = tmem_base + acc * TILE;
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const int st = it % kStages;
                    // The MMAs that read this scale buffer before are done.
                    if (C::kSfBufs < kStages && it >= C::kSfBufs &&
                        !mbar_wait(&empty[(it - C::kSfBufs) % kStages], ((it - C::kSfBufs) / kStages) & 1u, status)) {
                        ok = false;
                        break;
                    }
                    if (!mbar_wait(&full[st], (it / kStages) & 1u, status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t sfa = tmem_base + C::kScaleCol + (it % C::kSfBufs) * C::kSfCols;
                    const uint32_t sfb = sfa + C::kSfColsA;
                    const uint64_t ad = sw128_kmajor_desc(smem_u32(sW + st * kWBytes));
                    const uint64_t bd = sw128_kmajor_desc(smem_u32(sT + st * C::kB));
                    const uint64_t da = scale_tile_desc(smem_u32(sSfW + st * C::kSfA));
                    const uint64_t db = scale_tile_desc(smem_u32(sSfT + st * C::kSfB));
                    const int steps = (min(kStageK, a.K - kb * kStageK) + 63) / 64;
#pragma unroll
                    for (int j = 0; j < C::kSfTiles; ++j) {
                        tc_cp_scales<CG>(sfa + 4 * j, da + 32u * j);
                        tc_cp_scales<CG>(sfb + j * C::kRowBlocks * 4, db + 32u * j);
                        if (nrb > 1)
                            tc_cp_scales<CG>(sfb + j * C::kRowBlocks * 4 + 4, db + 32u * (C::kSfTiles + j));
                    }
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk >= steps) break;
                        // 64 elements: half of an MXFP4 scale tile's 4 scales, a whole NVFP4 one's.
                        const int j = FMT == kMxFp4 ? kk / 2 : kk;
                        const uint32_t id = FMT == kMxFp4 ? 2u * (kk & 1) : 0u;
                        tc_mma_mx<FMT, CG>(d, ad + 2u * kk, bd + 2u * kk, idesc | mx_idesc_sf(id), sfa + 4 * j,
                                           sfb + j * C::kRowBlocks * 4 + shift, (kb | kk) != 0 ? 1u : 0u);
                    }
                    commit_all(&empty[st]);
                }
                if (ok) commit_all(&tfull[acc]);
            }
            if constexpr (CG == 2) tc_commit_pair(mma_done);
            else tc_commit(mma_done);
            mbar_wait_drain(mma_done, 0u);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;             // the TMEM lane quarter this warp may read
        const int half = (warp - 2) >> 2;   // which of the quarter's two warps: every other 32 tokens
        const uint32_t buf = smem_u32(sOut + (warp - 2) * kStageOut);
        uint32_t tcount = 0;
        for (int u = first; u < total; u += step, ++tcount) {
            const Unit w = unit_of(u);
            const uint32_t acc = tcount & 1u, use = tcount >> 1;
            const int f0 = w.feat0 + static_cast<int>(rank) * kFeat + q * 32;
            const float mul = a.post * (a.alpha ? __ldg(a.alpha + w.g) : 1.f);
            auto bias_of = [&](int f) { return a.bias && f < a.N ? __ldg(a.bias + (int64_t)w.g * a.N + f) : 0.f; };
            int got = 1;
            if constexpr (ACT != kActRuntime) {
                float bv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) bv[i] = bias_of(f0 + lane / 4 + 8 * i);
                if (lane == 0) got = mbar_wait_idle(&tfull[acc], use & 1u, status) ? 1 : 0;
                if (!__shfl_sync(0xffffffffu, got, 0)) break;
                tc_fence_after_sync();
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * TILE;
                for (int c = half * 32; c < w.ntok; c += 64) {
                    uint32_t lo[16], hi[16];  // features 0..15 and 16..31 of the quarter
                    tmem_ld_16x256b_x4(taddr + c, lo);
                    tmem_ld_16x256b_x4(taddr + (16u << 16) + c, hi);
                    tmem_ld_wait();
                    auto pack = [&](uint32_t x, uint32_t y, float b) {
                        const __nv_bfloat162 p =
                            __floats2bfloat162_rn(activate_t<ACT>(fmaf(__uint_as_float(x), mul, b)),
                                                  activate_t<ACT>(fmaf(__uint_as_float(y), mul, b)));
                        return *reinterpret_cast<const uint32_t *>(&p);
                    };
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        stmatrix_x4_trans(buf + (8 * j + lane % 8) * kPitch + lane / 8 * 16,
                                          pack(lo[4 * j], lo[4 * j + 1], bv[0]), pack(lo[4 * j + 2], lo[4 * j + 3], bv[1]),
                                          pack(hi[4 * j], hi[4 * j + 1], bv[2]),
                                          pack(hi[4 * j + 2], hi[4 * j + 3], bv[3]));
                    __syncwarp();
                    const int f = f0 + lane % 4 * 8;
                    const uint8_t *src = sOut + (warp - 2) * kStageOut + lane % 4 * 16;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = c + 8 * i + lane / 4;
                        const uint4 v = *reinterpret_cast<const uint4 *>(src + (8 * i + lane / 4) * kPitch);
                        if (t < w.ntok && f < a.N) {
                            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.out) + (int64_t)(w.row0 + t) * a.out_ld + f;
                            if (a.vec_ok && f + 8 <= a.N) {
                                *reinterpret_cast<uint4 *>(o) = v;
                            } else {
                                const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    if (f + k < a.N)
                                        o[k] = __ushort_as_bfloat16(static_cast<unsigned short>(words[k / 2] >> (16 * (k & 1))));
                            }
                        }
                    }
                    __syncwarp();
                }
            } else {
                const int f = f0 + lane;
                const float bv = bias_of(f);
                if (lane == 0) got = mbar_wait_idle(&tfull[acc], use & 1u, status) ? 1 : 0;
                if (!__shfl_sync(0xffffffffu, got, 0)) break;
                tc_fence_after_sync();
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * TILE;
                for (int c = half * 16; c < w.ntok; c += 32) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(taddr + c, r);
                    tmem_ld_wait();
                    float *o = static_cast<float *>(a.out) + (int64_t)(w.row0 + c) * a.out_ld + f;
#pragma unroll
                    for (int t = 0; t < 16; ++t)
                        if (f < a.N && c + t < w.ntok)
                            o[t * a.out_ld] = activate(a.act, fmaf(__uint_as_float(r[t]), mul, bv));
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
                else mbar_arrive(&tempty[acc]);
            }
        }
    }

    // A role that gave up may leave loads in flight: let them land.
    if (!ok || *reinterpret_cast<volatile uint32_t *>(status) != kDevOk) spin_ns(1000000ull);
    tc_fence_before_sync();
    if constexpr (CG == 2) cluster_sync_all();
    else __syncthreads();
    tc_fence_after_sync();
    if (warp == 1) {
        if constexpr (CG == 2) tmem_dealloc_pair(tmem_base, kTmemCols);
        else tmem_dealloc(tmem_base, kTmemCols);
    }
    if (threadIdx.x == 0 && a.status) {
        const uint32_t v = *status | bad;
        if (v) atomicOr(a.status, v);
    }
}

template <int FMT, int TILE, int CG, int ACT>
cudaError_t launch(const MxMaps &m, const MxGemmArgs &a, int num_sms, cudaStream_t s) {
    using C = Cfg<FMT, TILE, CG>;
    cudaError_t e = set_smem_limit_once<mx_gemm_kernel<FMT, TILE, CG, ACT>>(C::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t most = ((int64_t)a.rows / TILE + a.G) * ((a.N + kFeat * CG - 1) / (kFeat * CG));
    if (most > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CG * static_cast<unsigned>(std::min<int64_t>(most, num_sms / CG)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<FMT, TILE, CG, ACT>, m, a);
}

template <int FMT, int TILE, int CG>
cudaError_t launch_act(const MxMaps &m, const MxGemmArgs &a, int num_sms, cudaStream_t s) {
    if (a.out_f32) return launch<FMT, TILE, CG, kActRuntime>(m, a, num_sms, s);
    switch (a.act) {
        case 0: return launch<FMT, TILE, CG, 0>(m, a, num_sms, s);
        case 1: return launch<FMT, TILE, CG, 1>(m, a, num_sms, s);
        case 2: return launch<FMT, TILE, CG, 2>(m, a, num_sms, s);
        default: return launch<FMT, TILE, CG, -1>(m, a, num_sms, s);
    }
}

}  // namespace

cudaError_t launch_mx_gemm(const MxMaps &m, const MxGemmArgs &a, int format, int num_sms, cudaStream_t s) {
    // Short segments: rows beyond the 127 that each group's start may leave unused.
    const int64_t filled = (int64_t)a.rows - (a.G > 1 ? (int64_t)a.G * 127 : 0);
    const bool narrow = filled <= (int64_t)64 * a.G;
    if (format == kMxFp4)
        return narrow ? launch_act<kMxFp4, 64, 1>(m, a, num_sms, s) : launch_act<kMxFp4, 192, 2>(m, a, num_sms, s);
    return narrow ? launch_act<kNvFp4, 64, 1>(m, a, num_sms, s) : launch_act<kNvFp4, 192, 2>(m, a, num_sms, s);
}

}  // namespace moe
