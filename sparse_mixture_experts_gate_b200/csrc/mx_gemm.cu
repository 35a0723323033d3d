// mx_gemm.cu - grouped product of microscaled 4-bit operands on the block-scaled
// tensor cores (sm_100a tcgen05 kind::mxf4 and kind::mxf4nvf4).
//
//   out[r][n] = act( alpha_g 2^e sum_k A[r][k] W[g][n][k] + bias[g][n] ),  g = group of row r,
//
// A and W being 4-bit codes times their blocks' scales; the sum is held in
// fp32 and rounded once, to the output's type.
//
// Operand roles. The MMA's M side is the output features (rows of W[g]) and its
// N side a token tile of one group, so a group of a few rows costs an MMA of a few
// columns. Unit = (token tile, feature tile); every CTA builds the groups' tile
// prefix in shared memory and takes its share of the units in steps of the grid.
//
// Three forms (launch_mx_gemm has the rule). Long segments run on CTA pairs
// (cta_group::2), 256 features x 192 tokens an accumulator, each CTA staging its
// 128 weight rows and half of the tokens: either a unit fills both accumulators (384
// tokens: the weights' way through L2 and shared memory is shared by twice the
// tokens, but the next unit waits for the epilogue), or units take the two in turn
// (the epilogue is hidden). Short segments (a few tokens for each expert) are bound
// by the weights' bytes: single CTAs, 128 features x up to 64 tokens, a deeper
// pipeline, two accumulators in turn.
//
// Per CTA (576 threads): warp 0 loads codes (TMA, 128B swizzle, 256 elements
// of K a stage) and scale tiles, signalling the (leader's) stage barrier; warp
// 1 owns TMEM and, in the leader, copies a stage's scale tiles into TMEM
// (tcgen05.cp, both CTAs') and issues its MMAs; warps 2..17 drain this CTA's 128
// features of the accumulators, four warps for each quarter of the TMEM lanes. The
// loading and issuing warps run their loops with all lanes and elect one only for
// the instructions themselves: descriptors then stay in uniform registers (with
// one lane in the loop, issuing took longer than the products: 121 us instead of
// 91 for 128 experts of 1536 x 4096 with a row or a few each).
//
// TMEM (512 columns): two accumulators and, in the rest, as many buffers of scale
// columns as there are stages, or fit: a buffer is filled again only once the MMAs
// that read it have completed (their stage's commit), so no copy passes an MMA. A
// token tile starts at a multiple of 64 rows of the 128-row scale tiles, so its
// first scale column is even.
//
// Epilogue of bf16 outputs: TMEM is read in 16 x 256-bit pieces, whose register
// layout (a lane holds two neighbouring tokens of one feature) is the one that
// stmatrix.trans takes, so a warp turns 16 tokens x 32 features around through a
// shared buffer of its own without shuffles, and stores each token's 64 bytes
// with 16-byte stores. A warp takes all of its part of an accumulator into
// registers and hands the accumulator back before it computes. fp32 outputs are
// stored from lane = feature directly.
//
// Every wait is bounded; a role that gives up sets the block's status word, the
// others stop, and the block ends after its copies and MMAs have drained.
#include <algorithm>

#include "mx_common.cuh"

namespace moe {
namespace {

constexpr int kEpiWarps = 16;               // four for each quarter of the TMEM lanes
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kFeat = 128;                // features per CTA
constexpr int kStageK = 256;              // elements of K per stage: 128 bytes of codes
constexpr int kWBytes = kFeat * 128;      // weight codes per stage
constexpr int kMaxGroups = 1024;
constexpr int kTmemCols = 512;
constexpr int kStageOut = 16 * 64;        // one warp's output buffer: 16 tokens x 32 bf16 features
constexpr int kActRuntime = -2;           // fp32 outputs: the activation is looked up at run time

// TILE tokens per accumulator, SUB accumulators per unit.
template <int FMT, int TILE, int SUB, int CG>
struct Cfg {
    static constexpr int kUnitTok = TILE * SUB;
    static constexpr int kSfTiles = kStageK / MxFormat<FMT>::kTileK;  // scale tiles along K per stage
    static constexpr int kRowBlocks = (kUnitTok + 127) / 128;         // 128-row scale tiles under a unit's tokens
    static constexpr int kSfA = kSfTiles * 512;                       // weight scales
    static constexpr int kSfB = kRowBlocks * kSfTiles * 512;          // token scales
    static constexpr int kSub = TILE / CG * 128;                      // token codes of one accumulator
    static constexpr int kB = SUB * kSub;
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
    static_assert(TILE % 64 == 0 && kEpiWarps == 16, "the epilogue warps share an accumulator evenly");
    static_assert(SUB == 1 || kUnitTok % 128 == 0, "units start on a scale tile");
    static_assert(kSub % 1024 == 0, "operand tiles keep the 1024-byte swizzle alignment");
};

// Status bits of the products that were given no word of their own, until mx_take_status reads them.
__device__ uint32_t g_unclaimed_status;

struct Unit {
    int g, row0, ntok, feat0;
};

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0u;
}

__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// Byte of 16-byte piece p (0..3) of token row r in a warp's output buffer: pieces
// trade places by row, so that eight rows' pieces p (stmatrix) as well as two
// rows' four pieces (the loads that follow) lie in different banks.
__device__ __forceinline__ int staged(int r, int p) { return r * 64 + ((p ^ (r >> 1 & 3)) << 4); }

// Arrives on an mbarrier of either CTA of the pair with CTA-scope release. What
// it hands over is the accumulator, whose loads have completed (wait::ld, then the
// tcgen05 fence); a cluster-scope release would also wait for this thread's
// earlier output stores to land (with it, 147 instead of 131 us for 64 experts,
// 49152 rows, 1408 x 2048, NVFP4, swish, when this was changed).
__device__ __forceinline__ void arrive_pair(uint32_t bar_cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster_addr) : "memory");
}

// Four 8 x 8 matrices of 16-bit values, transposed: lane 8 m + i gives the address of row i of matrix m.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

template <int FMT, int TILE, int SUB, int CG, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ MxMaps m, const MxGemmArgs a) {
    using C = Cfg<FMT, TILE, SUB, CG>;
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
    int32_t *scan = reinterpret_cast<int32_t *>(tmem_slot + 2);    // [32]
    int32_t *prefix = scan + 32;                                   // [G + 1] token tiles before each group
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&m.w);
        tma_prefetch_desc(&m.a);
        if (CG == 2) tma_prefetch_desc(&m.a96);
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
    // All of this may run while the rows are still being quantised.
    wait_for_previous();
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
            v = fits ? (rows + C::kUnitTok - 1) / C::kUnitTok : 0;
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
        const int off = (tt - prefix[lo]) * C::kUnitTok;
        return Unit{lo, start + off, min(C::kUnitTok, rows - off), (u - tt * n_ft) * kFeat * CG};
    };
    auto commit_all = [&](uint64_t *bar) {
        if constexpr (CG == 2) tc_commit_pair_mc(bar, 0x3);
        else tc_commit(bar);
    };
    bool ok = true;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        const bool one = elect_one();
        const int NB = (a.N + 127) / 128;
        uint32_t it = 0;
        for (int u = first; u < total && ok; u += step) {
            const Unit w = unit_of(u);
            const int nrb = (w.row0 % 128 + w.ntok + 127) / 128;
            const int feat = w.feat0 + static_cast<int>(rank) * kFeat;
            const int wrow = w.g * a.N + feat;
            // The second CTA of a last feature tile may have no weight scales: it reads the group's last ones.
            const int wblk = w.g * NB + min(feat / 128, NB - 1), tblk = w.row0 / 128;
            int boxes[SUB], rows = 0;  // 16-row boxes of this CTA's part of each accumulator's tokens
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
                boxes[s] = (min(TILE, max(w.ntok - s * TILE, 0)) + C::kStep - 1) / C::kStep;
                rows += boxes[s] * 16;
            }
            const uint32_t bytes = CG * (kWBytes + rows * 128 + C::kSfA + nrb * C::kSfTiles * 512);
            for (int kb = 0; kb < kblocks; ++kb, ++it) {
                const int st = it % kStages;
                if (!__all_sync(0xffffffffu, mbar_wait(&empty[st], ((it / kStages) & 1u) ^ 1u, status))) {
                    ok = false;
                    break;
                }
                if (one) {
                    const uint32_t bar = CG == 2 ? mapa_shared(smem_u32(&full[st]), 0) : 0u;
                    auto load = [&](const CUtensorMap *map, void *dst, int x, int y) {
                        if constexpr (CG == 2) tma_load_2d_pair(map, bar, dst, x, y);
                        else tma_load_2d(map, &full[st], dst, x, y);
                    };
                    if (leader) mbar_arrive_expect_tx(&full[st], bytes);
                    load(&m.w, sW + st * kWBytes, kb * 128, wrow);
                    load(&m.sw, sSfW + st * C::kSfA, kb * C::kSfTiles * 64, wblk);
#pragma unroll
                    for (int s = 0; s < SUB; ++s) {
                        uint8_t *dst = sT + st * C::kB + s * C::kSub;
                        const int row = w.row0 + s * TILE + static_cast<int>(rank) * boxes[s] * 16;
                        if (CG == 2 && boxes[s] == TILE / C::kStep) {
                            load(&m.a96, dst, kb * 128, row);
                        } else {
                            for (int b = 0; b < boxes[s]; ++b) load(&m.a, dst + b * 2048, kb * 128, row + b * 16);
                        }
                    }
                    for (int b = 0; b < nrb; ++b)
                        load(&m.sa, sSfT + st * C::kSfB + b * C::kSfTiles * 512, kb * C::kSfTiles * 64, tblk + b);
                }
                __syncwarp();
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA (leader)
        if (leader) {
            const bool one = elect_one();
            const uint32_t w_lo = operand_desc_lo(smem_u32(sW)), t_lo = operand_desc_lo(smem_u32(sT));
            const uint32_t sw_lo = scale_desc_lo(smem_u32(sSfW)), st_lo = scale_desc_lo(smem_u32(sSfT));
            uint32_t uses[SUB] = {}, tcount = 0;
            uint32_t st = 0, ph = 0;              // stage and its parity
            uint32_t buf = 0, old = 0, old_ph = 0;  // scale buffer; the stage that used it last, and its parity
            bool reused = false;
            for (int u = first; u < total && ok; u += step, ++tcount) {
                const Unit w = unit_of(u);
                const int nrb = (w.row0 % 128 + w.ntok + 127) / 128;
                const uint32_t shift = (w.row0 % 128) / 32;  // first scale column of the unit's tokens
                uint32_t idesc[SUB];  // 0: no tokens
#pragma unroll
                for (int s = 0; s < SUB; ++s) {
                    const int cols = (min(TILE, max(w.ntok - s * TILE, 0)) + C::kStep - 1) / C::kStep * C::kStep;
                    idesc[s] = cols ? mx_idesc<FMT>(kFeat * CG, cols) : 0u;
                }
                for (int kb = 0; kb < kblocks; ++kb) {
                    if constexpr (C::kSfBufs < kStages) {  // the MMAs that read this scale buffer before are done
                        if (reused) ok = mbar_wait(&empty[old], old_ph, status);
                    }
                    if (ok) ok = mbar_wait(&full[st], ph, status);
                    if (kb == 0 && ok) {  // the (first) accumulator has been drained
                        const uint32_t use = SUB == 2 ? uses[0] : tcount >> 1;
                        ok = mbar_wait(&tempty[SUB == 2 ? 0 : tcount & 1u], (use & 1u) ^ 1u, status);
                        ++uses[0];
                    }
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t sfa = tmem_base + C::kScaleCol + buf * C::kSfCols, sfb = sfa + C::kSfColsA;
                    const bool last = kb == kblocks - 1;
                    const int steps = last ? (a.K - kb * kStageK + 63) / 64 : 4;
                    auto products = [&](int s) {
                        const uint32_t acc = SUB == 2 ? s : tcount & 1u;
                        const uint32_t al = w_lo + st * (kWBytes >> 4), bl = t_lo + st * (C::kB >> 4) + s * (C::kSub >> 4);
                        const uint32_t d = tmem_base + acc * TILE, sb = sfb + shift + s * (TILE / 32);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if (kk >= steps) break;
                            // 64 elements: half of an MXFP4 scale tile's 4 scales, a whole NVFP4 one's.
                            const int j = FMT == kMxFp4 ? kk / 2 : kk;
                            const uint32_t id = FMT == kMxFp4 ? 2u * (kk & 1) : 0u;
                            tc_mma_mx<FMT, CG>(d, al + 2u * kk, bl + 2u * kk, idesc[s] | mx_idesc_sf(id), sfa + 4 * j,
                                               sb + j * C::kRowBlocks * 4, kk > 0 ? 1u : (kb > 0 ? 1u : 0u));
                        }
                        if (last) commit_all(&tfull[acc]);
                    };
                    if (one) {
                        const uint32_t da = sw_lo + st * (C::kSfA >> 4), db = st_lo + st * (C::kSfB >> 4);
#pragma unroll
                        for (int j = 0; j < C::kSfTiles; ++j) {
                            tc_cp_scales<CG>(sfa + 4 * j, da + 32u * j);
#pragma unroll
                            for (int b = 0; b < C::kRowBlocks; ++b)
                                if (b < nrb)
                                    tc_cp_scales<CG>(sfb + (j * C::kRowBlocks + b) * 4, db + 32u * (b * C::kSfTiles + j));
                        }
                        products(0);
                    }
                    if (SUB == 2 && idesc[SUB - 1]) {
                        if (kb == 0) {
                            if (!__all_sync(0xffffffffu, mbar_wait(&tempty[SUB - 1], (uses[SUB - 1] & 1u) ^ 1u, status))) {
                                ok = false;
                                break;
                            }
                            ++uses[SUB - 1];
                            tc_fence_after_sync();
                        }
                        if (one) products(SUB - 1);
                    }
                    if (one) commit_all(&empty[st]);
                    if constexpr (C::kSfBufs < kStages) {
                        if (reused && ++old == kStages) {
                            old = 0;
                            old_ph ^= 1u;
                        }
                        if (++buf == C::kSfBufs) {
                            buf = 0;
                            reused = true;
                        }
                    } else {
                        buf = st + 1 == kStages ? 0 : st + 1;
                    }
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                    __syncwarp();
                }
            }
            if (one) {
                if constexpr (CG == 2) tc_commit_pair(mma_done);
                else tc_commit(mma_done);
            }
            __syncwarp();
            mbar_wait_drain(mma_done, 0u);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;             // the TMEM lane quarter this warp may read
        const int part = (warp - 2) >> 2;   // which of the quarter's four warps: every fourth 16 tokens
        const uint8_t *own = sOut + (warp - 2) * kStageOut;
        const uint32_t buf = smem_u32(own);
        auto release = [&](uint32_t acc) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) arrive_pair(mapa_shared(smem_u32(&tempty[acc]), 0));
                else mbar_arrive(&tempty[acc]);
            }
        };
        uint32_t uses[SUB] = {}, tcount = 0;
        for (int u = first; u < total && ok; u += step, ++tcount) {
            const Unit w = unit_of(u);
            const int f0 = w.feat0 + static_cast<int>(rank) * kFeat + q * 32;
            const float mul = a.post * (a.alpha ? a.alpha[w.g] : 1.f);
            auto bias_of = [&](int f) { return a.bias && f < a.N ? a.bias[(int64_t)w.g * a.N + f] : 0.f; };
            float bv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) bv[i] = bias_of(ACT == kActRuntime ? f0 + lane : f0 + lane / 4 + 8 * i);
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
                const int ntok = min(TILE, w.ntok - s * TILE), row0 = w.row0 + s * TILE;
                if (ntok <= 0) break;
                const uint32_t acc = SUB == 2 ? s : tcount & 1u;
                const uint32_t use = SUB == 2 ? uses[s] : tcount >> 1;
                int got = 1;
                if (lane == 0) got = mbar_wait_idle(&tfull[acc], use & 1u, status) ? 1 : 0;
                ++uses[s];
                if (!__shfl_sync(0xffffffffu, got, 0)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * TILE;
                if constexpr (ACT != kActRuntime) {
                    constexpr int kChunks = TILE / 64;
                    uint32_t lo[kChunks][8], hi[kChunks][8];  // features 0..15 and 16..31 of the quarter
#pragma unroll
                    for (int i = 0; i < kChunks; ++i) {
                        const int c = part * 16 + 64 * i;
                        if (c < ntok) {
                            tmem_ld_16x256b_x2(taddr + c, lo[i]);
                            tmem_ld_16x256b_x2(taddr + (16u << 16) + c, hi[i]);
                        }
                    }
                    tmem_ld_wait();
                    release(acc);
                    auto pack = [&](uint32_t x, uint32_t y, float b) {
                        const __nv_bfloat162 p =
                            __floats2bfloat162_rn(activate_t<ACT>(fmaf(__uint_as_float(x), mul, b)),
                                                  activate_t<ACT>(fmaf(__uint_as_float(y), mul, b)));
                        return *reinterpret_cast<const uint32_t *>(&p);
                    };
                    const int f = f0 + lane % 4 * 8;
                    __nv_bfloat16 *orow = static_cast<__nv_bfloat16 *>(a.out) +
                                          (int64_t)(row0 + part * 16 + lane / 4) * a.out_ld + f;
                    const bool whole = a.vec_ok && f + 8 <= a.N;
#pragma unroll
                    for (int i = 0; i < kChunks; ++i) {
                        const int c = part * 16 + 64 * i;
                        if (c >= ntok) break;
                        uint32_t pk[8];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            pk[4 * j] = pack(lo[i][4 * j], lo[i][4 * j + 1], bv[0]);
                            pk[4 * j + 1] = pack(lo[i][4 * j + 2], lo[i][4 * j + 3], bv[1]);
                            pk[4 * j + 2] = pack(hi[i][4 * j], hi[i][4 * j + 1], bv[2]);
                            pk[4 * j + 3] = pack(hi[i][4 * j + 2], hi[i][4 * j + 3], bv[3]);
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            stmatrix_x4_trans(buf + staged(8 * j + lane % 8, lane / 8), pk[4 * j], pk[4 * j + 1],
                                              pk[4 * j + 2], pk[4 * j + 3]);
                        __syncwarp();
                        uint4 v[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            v[k] = *reinterpret_cast<const uint4 *>(own + staged(8 * k + lane / 4, lane % 4));
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (c + 8 * k + lane / 4 >= ntok) continue;
                            __nv_bfloat16 *o = orow + (64 * i + 8 * k) * a.out_ld;
                            if (whole) {
                                *reinterpret_cast<uint4 *>(o) = v[k];
                            } else {
                                const uint32_t words[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (f + e < a.N)
                                        o[e] = __ushort_as_bfloat16(
                                            static_cast<unsigned short>(words[e / 2] >> (16 * (e & 1))));
                            }
                        }
                    }
                } else {
                    const int f = f0 + lane;
                    for (int c = part * 16; c < ntok; c += 64) {
                        uint32_t r[16];
                        tmem_ld_32x32b_x16(taddr + c, r);
                        tmem_ld_wait();
                        float *o = static_cast<float *>(a.out) + (int64_t)(row0 + c) * a.out_ld + f;
#pragma unroll
                        for (int t = 0; t < 16; ++t)
                            if (f < a.N && c + t < ntok)
                                o[t * a.out_ld] = activate(a.act, fmaf(__uint_as_float(r[t]), mul, bv[0]));
                    }
                    release(acc);
                }
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
    if (threadIdx.x == 0) {
        const uint32_t v = *status | bad;
        if (v) atomicOr(a.status ? a.status : &g_unclaimed_status, v);
    }
}

__global__ void clear_status_kernel(uint32_t bits) { atomicAnd(&g_unclaimed_status, ~bits); }

template <int FMT, int TILE, int SUB, int CG, int ACT>
cudaError_t launch(const MxMaps &m, const MxGemmArgs &a, int num_sms, cudaStream_t s) {
    using C = Cfg<FMT, TILE, SUB, CG>;
    cudaError_t e = set_smem_limit_once<mx_gemm_kernel<FMT, TILE, SUB, CG, ACT>>(C::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t most = ((int64_t)a.rows / C::kUnitTok + a.G) * ((a.N + kFeat * CG - 1) / (kFeat * CG));
    if (most > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CG * static_cast<unsigned>(std::min<int64_t>(most, num_sms / CG)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0] = early_start_attribute();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<FMT, TILE, SUB, CG, ACT>, m, a);
}

template <int FMT, int TILE, int SUB, int CG>
cudaError_t launch_act(const MxMaps &m, const MxGemmArgs &a, int num_sms, cudaStream_t s) {
    if (a.out_f32) return launch<FMT, TILE, SUB, CG, kActRuntime>(m, a, num_sms, s);
    switch (a.act) {
        case 0: return launch<FMT, TILE, SUB, CG, 0>(m, a, num_sms, s);
        case 1: return launch<FMT, TILE, SUB, CG, 1>(m, a, num_sms, s);
        case 2: return launch<FMT, TILE, SUB, CG, 2>(m, a, num_sms, s);
        default: return launch<FMT, TILE, SUB, CG, -1>(m, a, num_sms, s);
    }
}

}  // namespace

// Short segments: with few rows a group the narrow form is ahead (128 experts, 1024 rows, K 4096, N 1536:
// 81 us against 95). The border is one of its tiles for each group; between 8 rows a group and that the two
// were not compared. `filled` is a lower bound where there are several groups: segments that leave little unused
// count as fewer rows than they have.
bool mx_gemm_narrow(const MxGemmArgs &a) { return a.filled <= (int64_t)64 * a.G; }

cudaError_t mx_take_status(uint32_t *bits, cudaStream_t s) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(bits, g_unclaimed_status, sizeof *bits, 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess || !*bits) return e;
    clear_status_kernel<<<1, 1, 0, s>>>(*bits);
    return cudaGetLastError();
}

cudaError_t launch_mx_gemm(const MxMaps &m, const MxGemmArgs &a, int format, int num_sms, cudaStream_t s) {
    const bool narrow = mx_gemm_narrow(a);
    // Both accumulators a unit from K = 4096 on: 218 us instead of 251 at K = 7168 (32 experts, 32768
    // rows, N 2048, MXFP4), where the epilogue is short beside the products; 123 instead of 113 at K = 2048
    // (64 experts, 49152 rows, N 1408, NVFP4). Between the two the border was not measured, nor with segments of
    // at most 192 rows, which leave the second accumulator empty.
    const bool deep = a.K >= 4096;
    if (format == kMxFp4)
        return narrow ? launch_act<kMxFp4, 64, 1, 1>(m, a, num_sms, s)
                      : deep ? launch_act<kMxFp4, 192, 2, 2>(m, a, num_sms, s) : launch_act<kMxFp4, 192, 1, 2>(m, a, num_sms, s);
    return narrow ? launch_act<kNvFp4, 64, 1, 1>(m, a, num_sms, s)
                  : deep ? launch_act<kNvFp4, 192, 2, 2>(m, a, num_sms, s) : launch_act<kNvFp4, 192, 1, 2>(m, a, num_sms, s);
}

}  // namespace moe
