// mx_quant.cu - rows to and from microscaled 4-bit floating point.
//
// For every block of 32 (MXFP4) or 16 (NVFP4) elements of u = x 2^-e:
//   MXFP4: scale = 2^(floor(log2 max|u|) - 2), held as E8M0 between 2^-127 and 2^127;
//   NVFP4: scale = max|u| / 6, rounded to nearest even E4M3, at most 448;
//   code = u / scale rounded to nearest even E2M1, at most 6 in magnitude.
// A block with an infinity or a NaN gets the NaN scale and zero codes. Where
// an NVFP4 scale rounds to 0 the codes are 0.
//
// Every rounding is the one of the exact quotient. MXFP4 quotients are exact: x / scale 2^-e, in this
// order, as u itself may be below fp32's normal numbers.
// NVFP4 divides fp32 elements (correctly rounded: a quotient that is not one of
// the rounding borders cannot round onto one, as border times scale has at most
// 7 significant bits). For bf16 elements the quotient times 1 / scale is off by
// less than 2^-19, and is rounded to a multiple of 2^-12: borders (multiples of
// 1/4) come out exactly, and every other quotient is at least 2^-10 away from
// one, since element and border times scale differ by 2^-8 of themselves.
//
// 2 (bf16) or 4 bytes are read and 0.5 + 1 / block written per element; the
// instructions per element are what stands between that and HBM's rate, so a
// thread takes 16 neighbouring elements (32-byte loads): one NVFP4 block or half
// an MXFP4 one, whose scale it works out once; the lanes of 4 blocks put their
// scale bytes together into the one 32-bit word that the scale tile holds of them.
#include <algorithm>
#include <cfloat>

#include "mx_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Eight E2M1 codes, the first in the low four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float *v) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

__device__ __forceinline__ float2 f16x2_values(uint32_t h) {
    float lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return make_float2(lo, hi);
}

// The values of two codes (fp16 holds them exactly), `x` the low one's.
__device__ __forceinline__ float2 e2m1x2_values(uint32_t b) {
    uint32_t h;
    asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(b));
    return f16x2_values(h);
}

// E4M3 byte of v >= 0, to nearest even, at most 448.
__device__ __forceinline__ uint32_t e4m3_of(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
    return r & 0xffu;
}

// The value of an E4M3 byte that is not NaN (fp16 holds it exactly).
__device__ __forceinline__ float e4m3_finite(uint32_t b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
    return f16x2_values(h).x;
}

__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ void load32(const void *p, uint32_t *w) {
    asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(p));
}

__device__ __forceinline__ void store32(void *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

constexpr int kLaneElems = 16;              // neighbouring elements of a row that a thread takes
constexpr int kStep = 32 * kLaneElems;      // and a warp

// Sixteen elements of a row as they lie in memory.
template <typename XT>
struct Raw {
    static constexpr int kWords = kLaneElems * sizeof(XT) / 4;
    uint32_t w[kWords];
};

template <typename XT>
__device__ __forceinline__ Raw<XT> load16(const XT *p, bool vec) {
    Raw<XT> r;
    if (vec) {
#pragma unroll
        for (int i = 0; i < Raw<XT>::kWords; i += 8) load32(reinterpret_cast<const uint32_t *>(p) + i, r.w + i);
        return r;
    }
#pragma unroll
    for (int i = 0; i < kLaneElems; ++i) {
        if constexpr (sizeof(XT) == 2) {
            const uint32_t h = __bfloat16_as_ushort(p[i]);
            r.w[i / 2] = i % 2 ? r.w[i / 2] | (h << 16) : h;
        } else {
            r.w[i] = __float_as_uint(p[i]);
        }
    }
    return r;
}

// The bits of the largest magnitude, as an fp32's (a NaN is the largest).
template <typename XT>
__device__ __forceinline__ uint32_t top_bits(const Raw<XT> &r) {
    constexpr uint32_t kMask = sizeof(XT) == 2 ? 0x7fff7fffu : 0x7fffffffu;
    uint32_t m = r.w[0] & kMask;
#pragma unroll
    for (int i = 1; i < Raw<XT>::kWords; ++i) {
        if constexpr (sizeof(XT) == 2) m = __vmaxu2(m, r.w[i] & kMask);
        else m = max(m, r.w[i] & kMask);
    }
    return sizeof(XT) == 2 ? max(m << 16, m & 0xffff0000u) : m;
}

template <typename XT>
__device__ __forceinline__ float element(const Raw<XT> &r, int i) {
    if constexpr (sizeof(XT) == 2) return __uint_as_float(i % 2 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
    else return __uint_as_float(r.w[i]);
}

template <typename XT>
__device__ __forceinline__ void store8(XT *p, bool vec, const float *v) {
    if (!vec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = from_f32<XT>(v[i]);
        return;
    }
    if constexpr (sizeof(XT) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

template <typename XT>
__device__ __forceinline__ void store16(XT *p, bool vec, const float *v) {
    if (!vec) {
#pragma unroll
        for (int i = 0; i < kLaneElems; ++i) p[i] = from_f32<XT>(v[i]);
        return;
    }
    uint32_t w[Raw<XT>::kWords];
#pragma unroll
    for (int i = 0; i < Raw<XT>::kWords; ++i) {
        if constexpr (sizeof(XT) == 2) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        } else {
            w[i] = __float_as_uint(v[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < Raw<XT>::kWords; i += 8) store32(reinterpret_cast<uint32_t *>(p) + i, w + i);
}

// Codes, scale byte and scale of the lane's 16 elements (see the head of this file).
template <int FMT, typename XT, bool PRE>
__device__ __forceinline__ uint2 quantize16(const Raw<XT> &v, float pre, uint32_t &byte, float &scale) {
    uint32_t top = top_bits<XT>(v);
    if constexpr (FMT == kMxFp4) top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const bool finite = top < 0x7f800000u;
    const float most = PRE ? __uint_as_float(top) * pre : __uint_as_float(top);
    float u[kLaneElems];
    if constexpr (FMT == kMxFp4) {
        int e = static_cast<int>(__float_as_uint(most) >> 23) - 2;
        // Where 2^-e takes a finite maximum out of fp32's range its exponent is known all the same.
        if (PRE && most == INFINITY) e = min(static_cast<int>((top >> 23) + (__float_as_uint(pre) >> 23)) - 129, 254);
        byte = finite ? static_cast<uint32_t>(e > 0 ? e : 0) : 255u;
        scale = e8m0_value(byte);
        const float inv = __uint_as_float(byte > 253u ? 1u << 22 : (254u - byte) << 23);
        // The scale first: what 2^-e alone would make too small for fp32's normal numbers keeps its digits.
#pragma unroll
        for (int i = 0; i < kLaneElems; ++i) u[i] = PRE ? element<XT>(v, i) * inv * pre : element<XT>(v, i) * inv;
    } else {
        byte = finite ? e4m3_of(__fdiv_rn(PRE ? fminf(most, FLT_MAX) : most, 6.f)) : 0u;
        scale = e4m3_finite(byte);
        if constexpr (sizeof(XT) == 2) {
            const float inv = scale > 0.f ? rcp_approx(scale) : 0.f;
            constexpr float kSnap = 0x1.8p11f;  // adding it rounds to multiples of 2^-12
#pragma unroll
            for (int i = 0; i < kLaneElems; ++i) {  // a quotient that becomes 0 keeps its sign
                const float e = PRE ? element<XT>(v, i) * pre : element<XT>(v, i);
                u[i] = copysignf(__fsub_rn(__fmaf_rn(e, inv, kSnap), kSnap), e);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kLaneElems; ++i)
                u[i] = __fdiv_rn(PRE ? element<XT>(v, i) * pre : element<XT>(v, i), scale);
        }
    }
    uint2 code = make_uint2(e2m1x8(u), e2m1x8(u + 8));
    if (!finite || !(scale > 0.f)) code = make_uint2(0u, 0u);
    if (FMT == kNvFp4 && !finite) {
        byte = 0x7fu;
        scale = __uint_as_float(0x7fffffffu);
    }
    return code;
}

// A block takes `rpb` (at most 32) output rows, its warps pieces of STEPS x 512
// elements of those that have a source row. PRE: a power of two comes out first.
template <int FMT, typename XT, int STEPS, bool PRE>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const MxQuantArgs a, int rpb, bool vec, bool vec_values) {
    constexpr int kWordLanes = MxFormat<FMT>::kTileK / kLaneElems;  // lanes of one word of 4 scales
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const int r0 = blockIdx.x * rpb;
    int src_l = -1;  // lane l: the source row of output row r0 + l
    if (lane < rpb && r0 + lane < a.rows) src_l = a.row_index ? a.row_index[r0 + lane] : r0 + lane;
    const uint32_t live = __ballot_sync(0xffffffffu, src_l >= 0 && src_l < a.x_rows);
    const int per_row = (a.cols + kStep * STEPS - 1) / (kStep * STEPS);
    const int items = __popc(live) * per_row;
    const int SB = mx_scale_tiles(a.cols, MxFormat<FMT>::kBlock);
    for (int item = threadIdx.x >> 5; item < items; item += kThreads / 32) {
        const int nth = item / per_row;
        // The nth row with a source: the lane that has so many of them before it.
        const int i = __ffs(__ballot_sync(0xffffffffu, (live >> lane & 1u) && __popc(live & ((1u << lane) - 1u)) == nth)) - 1;
        const int r = r0 + i, c0 = (item - nth * per_row) * (kStep * STEPS) + lane * kLaneElems;
        const XT *x = static_cast<const XT *>(a.x) + (int64_t)__shfl_sync(0xffffffffu, src_l, i) * a.ld + c0;
        Raw<XT> v[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            if (c0 + kStep * s < a.cols) v[s] = load16<XT>(x + kStep * s, vec);
            else v[s] = Raw<XT>{};
        }
        uint8_t *codes = a.codes + (int64_t)r * (a.cols / 2) + c0 / 2;
        const int j = c0 / MxFormat<FMT>::kTileK;  // scale tile of this lane's block
        uint8_t *tile = a.scales + (a.plain ? ((int64_t)r * SB + j) * 4
                                            : ((int64_t)(r / 128) * SB + j) * 512 + (r % 32) * 16 + (r % 128 / 32) * 4);
        const int tile_bytes = a.plain ? 4 : 512;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int c = c0 + kStep * s;
            if (c - lane * kLaneElems >= a.cols) break;  // warp-uniform
            uint32_t byte;
            float scale;
            const uint2 code = quantize16<FMT, XT, PRE>(v[s], a.pre, byte, scale);
            constexpr int kBlockLanes = kWordLanes / 4;
            uint32_t word = byte << (8 * (lane / kBlockLanes & 3));
#pragma unroll
            for (int off = kBlockLanes; off < kWordLanes; off <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, off);
            if (lane % kWordLanes == 0 && j + kStep / MxFormat<FMT>::kTileK * s < SB)
                *reinterpret_cast<uint32_t *>(tile + kStep / MxFormat<FMT>::kTileK * s * tile_bytes) = word;
            if (c < a.cols) {
                *reinterpret_cast<uint2 *>(codes + kStep / 2 * s) = code;
                if (a.values) {
                    float o[kLaneElems];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 q = e2m1x2_values((i < 4 ? code.x : code.y) >> (8 * (i % 4)) & 0xffu);
                        o[2 * i] = PRE ? q.x * a.post * scale : q.x * scale;  // in this order: as mx_dequantize_kernel
                        o[2 * i + 1] = PRE ? q.y * a.post * scale : q.y * scale;
                    }
                    store16<XT>(static_cast<XT *>(a.values) + (int64_t)r * a.values_ld + c, vec_values, o);
                }
            }
        }
    }
}

// A value is code 2^e scale, in this order: 2^e times the scale alone may leave fp32's range although the value
// does not, or is 0.
template <int FMT, typename OT>
__global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(const MxDequantArgs a, bool vec) {
    const int per_row = a.cols / 8;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t r = i / per_row;
    if (r >= a.rows) return;
    const int c = static_cast<int>(i - r * per_row) * 8, j = c / MxFormat<FMT>::kBlock;
    const int SB = mx_scale_tiles(a.cols, MxFormat<FMT>::kBlock);
    const uint32_t byte = a.scales[(r / 128 * SB + j / 4) * 512 + (r % 32) * 16 + (r % 128 / 32) * 4 + j % 4];
    const float scale = FMT == kMxFp4 ? e8m0_value(byte) : e4m3_value(byte);
    const uint32_t code = *reinterpret_cast<const uint32_t *>(a.codes + r * (a.cols / 2) + c / 2);
    float o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 q = e2m1x2_values(code >> (8 * k) & 0xffu);
        o[2 * k] = q.x * a.post * scale;
        o[2 * k + 1] = q.y * a.post * scale;
    }
    store8<OT>(static_cast<OT *>(a.out) + r * a.ld + c, vec, o);
}

// Rows of codes and scales to other rows. A warp takes rows i, i + 32, i + 64 and
// i + 96 of 128: their pieces are in flight together, and their words of a scale tile
// are 16 neighbouring bytes. Where a token goes to several experts, quantising it
// once and copying it costs less than quantising each row (8192 tokens x 2048 to 49152 rows, NVFP4: 27 us against 49).
//
// A row's scales in tiles are words of 4 bytes 512 bytes apart, each a 32-byte sector to read: where the codes were
// made for this copy their scales lie row by row (PLAIN; 57280 rows x 2048 NVFP4, with quantising 8192: 26 us
// against 32). Five blocks an SM: 32768 x 7168 to 270272 rows, NVFP4, with quantising 421 us, 432 with the four
// that registers would leave, 448 with six.
template <bool PLAIN>
__global__ void __launch_bounds__(kThreads, 5) mx_gather_kernel(const MxGatherArgs a, int SB) {
    const int lane = threadIdx.x & 31, warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int r0 = warp / 32 * 128 + warp % 32;
    if (r0 >= a.rows) return;
    launch_dependents();
    wait_for_previous();  // what is read below was written while this kernel lived: no read-only loads
    const int pieces = a.cols / 32;
    const int mine = lane < 4 && r0 + 32 * lane < a.rows ? a.row_index[r0 + 32 * lane] : -1;
    const uint4 *from[4];
    const uint8_t *sf[4];
    bool all = true;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int src = __shfl_sync(0xffffffffu, mine, u);
        const bool live = src >= 0 && src < a.src_rows;
        from[u] = live ? reinterpret_cast<const uint4 *>(a.codes + (int64_t)src * (a.cols / 2)) : nullptr;
        sf[u] = a.scales + (PLAIN ? (int64_t)src * SB * 4 : (int64_t)(src / 128) * SB * 512 + (src % 32) * 16 + (src % 128 / 32) * 4);
        all = all && live;
    }
    uint8_t *st = a.out_scales + (int64_t)(r0 / 128) * SB * 512 + (r0 % 32) * 16;
    for (int j = lane; j < SB; j += 32) {
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (from[u]) w[u] = *reinterpret_cast<const uint32_t *>(sf[u] + (int64_t)j * (PLAIN ? 4 : 512));
        uint32_t *to = reinterpret_cast<uint32_t *>(st + (int64_t)j * 512);
        if (all) {
            *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (from[u]) to[u] = w[u];
        }
    }
    uint4 *to = reinterpret_cast<uint4 *>(a.out_codes + (int64_t)r0 * (a.cols / 2));
    for (int i = lane; i < pieces; i += 32) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (from[u]) v[u] = from[u][i];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (from[u]) to[(int64_t)(32 * u) * pieces + i] = v[u];
    }
}

__global__ void __launch_bounds__(kThreads) mx_row_map_kernel(const MxRowMapArgs a) {
    const int r = blockIdx.x * kThreads + threadIdx.x;
    if (r >= a.rows) return;
    const int routed = a.group_start[a.E];
    int token = -1;
    if (r < routed) {
        const int as = a.row_assign[r];
        if (as >= 0) token = as / a.k;
    } else if (a.T_pad > 0 && (r - routed) / a.T_pad < a.S) {
        const int t = (r - routed) % a.T_pad;
        if (t < a.T) token = t;
    }
    a.token[r] = token;
    a.self[r] = token >= 0 ? r : -1;
}

bool vector_rows(const void *p, int64_t ld, int elem, int bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * elem % bytes == 0;
}

template <int FMT, typename XT, int STEPS>
cudaError_t quantize(const MxQuantArgs &a, int num_sms, cudaStream_t s) {
    const int64_t items = (int64_t)a.rows * ((a.cols + kStep * STEPS - 1) / (kStep * STEPS));
    // Rows per block: one piece for each warp, and more (up to 32) where there would be more than 64 blocks for
    // each SM. An index far longer than x has mostly rows that are none: 8 rows a block (one token in 16256 rows x 4096 4 us, 6 with 4;
    // 128 tokens in 17280, some blocks full, 8 us, 10 with 16).
    int rpb = 1;
    while (rpb < 32 && ((int64_t)rpb * items < (int64_t)a.rows * (kThreads / 32) || a.rows / rpb > 64 * num_sms)) rpb *= 2;
    if (a.row_index && (int64_t)a.x_rows * 16 < a.rows) rpb = 8;
    const int blocks = (a.rows + rpb - 1) / rpb;
    const bool vec = vector_rows(a.x, a.ld, sizeof(XT), 32), vv = vector_rows(a.values, a.values_ld, sizeof(XT), 32);
    if (a.pre != 1.f) mx_quantize_kernel<FMT, XT, STEPS, true><<<blocks, kThreads, 0, s>>>(a, rpb, vec, vv);
    else mx_quantize_kernel<FMT, XT, STEPS, false><<<blocks, kThreads, 0, s>>>(a, rpb, vec, vv);
    return cudaGetLastError();
}

template <int FMT, typename OT>
cudaError_t dequantize(const MxDequantArgs &a, cudaStream_t s) {
    const int64_t blocks = ((int64_t)a.rows * (a.cols / 8) + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    mx_dequantize_kernel<FMT, OT><<<(int)blocks, kThreads, 0, s>>>(a, vector_rows(a.out, a.ld, sizeof(OT), 16));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantArgs &a, int format, bool bf16, int num_sms, cudaStream_t s) {
    if (format == kMxFp4)
        return bf16 ? quantize<kMxFp4, __nv_bfloat16, 2>(a, num_sms, s) : quantize<kMxFp4, float, 1>(a, num_sms, s);
    return bf16 ? quantize<kNvFp4, __nv_bfloat16, 2>(a, num_sms, s) : quantize<kNvFp4, float, 1>(a, num_sms, s);
}

cudaError_t launch_mx_gather(const MxGatherArgs &a, int format, cudaStream_t s) {
    const int blocks = (a.rows - 1) / 128 * 4 + 4;  // 32 warps for every 128 rows
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr = early_start_attribute();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, a.plain ? mx_gather_kernel<true> : mx_gather_kernel<false>, a,
                              mx_scale_tiles(a.cols, format == kMxFp4 ? 32 : 16));
}

cudaError_t launch_mx_row_map(const MxRowMapArgs &a, cudaStream_t s) {
    mx_row_map_kernel<<<(a.rows + kThreads - 1) / kThreads, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_mx_dequantize(const MxDequantArgs &a, int format, bool bf16, cudaStream_t s) {
    if (format == kMxFp4) return bf16 ? dequantize<kMxFp4, __nv_bfloat16>(a, s) : dequantize<kMxFp4, float>(a, s);
    return bf16 ? dequantize<kNvFp4, __nv_bfloat16>(a, s) : dequantize<kNvFp4, float>(a, s);
}

}  // namespace moe
