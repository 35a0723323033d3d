// mx_quant.cu - rows to and from microscaled 4-bit floating point.
//
// For every block of 32 (MXFP4) or 16 (NVFP4) elements of u = x 2^-e:
//   MXFP4: scale = 2^(floor(log2 max|u|) - 2), held as E8M0 between 2^-127 and 2^127;
//   NVFP4: scale = max|u| / 6, rounded to nearest even E4M3, at most 448;
//   code = u / scale rounded to nearest even E2M1, at most 6 in magnitude.
// A block with an infinity or a NaN gets the NaN scale and zero codes. Where
// an NVFP4 scale rounds to 0 the codes are 0.
//
// Every rounding is the one of the exact quotient. MXFP4 quotients are exact.
// NVFP4 divides fp32 elements (correctly rounded: a quotient that is not one of
// the rounding borders cannot round onto one, as border times scale has at most
// 7 significant bits). For bf16 elements the quotient times 1 / scale is off by
// less than 2^-20, and is rounded to a multiple of 2^-12: borders (multiples of
// 1/4) come out exactly, and every other quotient is at least 2^-10 away from
// one, since element and border times scale differ by 2^-8 of themselves.
//
// Bound by HBM: 2 (bf16) or 4 bytes are read and 0.5 + 1 / block written per
// element. A thread takes 8 neighbouring elements, a warp 1024 of one row in
// four steps whose loads are in flight together; the block's maximum is a
// shuffle over 4 or 2 lanes, and the lanes of 4 blocks put their scale bytes
// together into the one 32-bit word that the scale tile holds of them.
#include <algorithm>

#include "mx_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 4;                 // steps of 256 elements a warp takes
constexpr int kWarpElems = 256 * kSteps;  // elements of one row per warp

// Two E2M1 codes, `lo` in the low four bits.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// The values of two codes (fp16 holds them exactly), `x` the low one's.
__device__ __forceinline__ float2 e2m1x2_values(uint32_t b) {
    uint32_t h;
    asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(b));
    float lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return make_float2(lo, hi);
}

// E4M3 byte of v >= 0, to nearest even, at most 448.
__device__ __forceinline__ uint32_t e4m3_of(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
    return r & 0xffu;
}

template <typename XT>
__device__ __forceinline__ void load8(const XT *p, bool vec, float (&v)[8]) {
    if constexpr (sizeof(XT) == 2) {
        if (vec) {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p));
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(a[i] << 16);
                v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
            }
            return;
        }
    } else {
        if (vec) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(p[i]);
}

template <typename XT>
__device__ __forceinline__ void store8(XT *p, bool vec, const float (&v)[8]) {
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

template <int FMT, typename XT>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const MxQuantArgs a, bool vec, bool vec_values) {
    constexpr int kLanes = MxFormat<FMT>::kBlock / 8;  // lanes per block
    const int lane = threadIdx.x & 31;
    const int per_row = (a.cols + kWarpElems - 1) / kWarpElems;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int r = static_cast<int>(item / per_row);
    if (r >= a.rows) return;
    const int src = a.row_index ? a.row_index[r] : r;
    if (src < 0 || src >= a.x_rows) return;
    const int c0 = static_cast<int>(item - (int64_t)r * per_row) * kWarpElems + lane * 8;
    const XT *x = static_cast<const XT *>(a.x) + (int64_t)src * a.ld;
    float v[kSteps][8];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        if (c0 + 256 * s < a.cols) {
            load8<XT>(x + c0 + 256 * s, vec, v[s]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[s][i] = 0.f;
        }
    }
    const int SB = mx_scale_tiles(a.cols, MxFormat<FMT>::kBlock);
    uint8_t *srow = a.scales + (int64_t)(r / 128) * SB * 512 + (r % 32) * 16 + (r % 128 / 32) * 4;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int c = c0 + 256 * s;
        if (c - lane * 8 >= a.cols) break;  // warp-uniform
        uint32_t top = 0u;  // max |u| as bits: a NaN is the largest
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[s][i] *= a.pre;
            top = max(top, __float_as_uint(v[s][i]) & 0x7fffffffu);
        }
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        const bool finite = top < 0x7f800000u;
        uint32_t byte;
        float scale;
        if constexpr (FMT == kMxFp4) {
            const int e = static_cast<int>(top >> 23) - 2;
            byte = finite ? static_cast<uint32_t>(e > 0 ? e : 0) : 255u;
            scale = e8m0_value(byte);
            const float inv = __uint_as_float((254u - min(byte, 253u)) << 23);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[s][i] *= inv;
        } else {
            byte = finite ? e4m3_of(__fdiv_rn(__uint_as_float(top), 6.f)) : 0x7fu;
            scale = e4m3_value(byte);
            if constexpr (sizeof(XT) == 2) {
                const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
                constexpr float kSnap = 0x1.8p11f;  // adding it rounds to multiples of 2^-12
#pragma unroll
                for (int i = 0; i < 8; ++i)  // a quotient that becomes 0 keeps its sign
                    v[s][i] = copysignf(__fsub_rn(__fmaf_rn(v[s][i], inv, kSnap), kSnap), v[s][i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[s][i] = scale > 0.f ? __fdiv_rn(v[s][i], scale) : 0.f;
            }
        }
        uint32_t code = 0u;
        if (finite && scale > 0.f) {
#pragma unroll
            for (int i = 0; i < 4; ++i) code |= e2m1x2(v[s][2 * i], v[s][2 * i + 1]) << (8 * i);
        }
        uint32_t word = byte << (8 * (lane / kLanes & 3));
#pragma unroll
        for (int off = kLanes; off < 4 * kLanes; off <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, off);
        const int j = c / MxFormat<FMT>::kTileK;  // scale tile of this lane's block
        if (lane % (4 * kLanes) == 0 && j < SB) *reinterpret_cast<uint32_t *>(srow + (int64_t)j * 512) = word;
        if (c < a.cols) {
            *reinterpret_cast<uint32_t *>(a.codes + (int64_t)r * (a.cols / 2) + c / 2) = code;
            if (a.values) {
                float o[8];
                const float m = scale * a.post;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 q = e2m1x2_values(code >> (8 * i) & 0xffu);
                    o[2 * i] = q.x * m;
                    o[2 * i + 1] = q.y * m;
                }
                store8<XT>(static_cast<XT *>(a.values) + (int64_t)r * a.values_ld + c, vec_values, o);
            }
        }
    }
}

template <int FMT, typename OT>
__global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(const MxDequantArgs a, bool vec) {
    const int per_row = a.cols / 8;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t r = i / per_row;
    if (r >= a.rows) return;
    const int c = static_cast<int>(i - r * per_row) * 8, j = c / MxFormat<FMT>::kBlock;
    const int SB = mx_scale_tiles(a.cols, MxFormat<FMT>::kBlock);
    const uint32_t byte = a.scales[(r / 128 * SB + j / 4) * 512 + (r % 32) * 16 + (r % 128 / 32) * 4 + j % 4];
    const float m = (FMT == kMxFp4 ? e8m0_value(byte) : e4m3_value(byte)) * a.post;
    const uint32_t code = *reinterpret_cast<const uint32_t *>(a.codes + r * (a.cols / 2) + c / 2);
    float o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 q = e2m1x2_values(code >> (8 * k) & 0xffu);
        o[2 * k] = q.x * m;
        o[2 * k + 1] = q.y * m;
    }
    store8<OT>(static_cast<OT *>(a.out) + r * a.ld + c, vec, o);
}

bool vector_rows(const void *p, int64_t ld, int elem) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * elem % 16 == 0;
}

template <int FMT, typename XT>
cudaError_t quantize(const MxQuantArgs &a, cudaStream_t s) {
    const int64_t items = (int64_t)a.rows * ((a.cols + kWarpElems - 1) / kWarpElems);
    const int64_t blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    mx_quantize_kernel<FMT, XT><<<(int)blocks, kThreads, 0, s>>>(a, vector_rows(a.x, a.ld, sizeof(XT)),
                                                                 vector_rows(a.values, a.values_ld, sizeof(XT)));
    return cudaGetLastError();
}

template <int FMT, typename OT>
cudaError_t dequantize(const MxDequantArgs &a, cudaStream_t s) {
    const int64_t blocks = ((int64_t)a.rows * (a.cols / 8) + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    mx_dequantize_kernel<FMT, OT><<<(int)blocks, kThreads, 0, s>>>(a, vector_rows(a.out, a.ld, sizeof(OT)));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantArgs &a, int format, bool bf16, cudaStream_t s) {
    if (format == kMxFp4) return bf16 ? quantize<kMxFp4, __nv_bfloat16>(a, s) : quantize<kMxFp4, float>(a, s);
    return bf16 ? quantize<kNvFp4, __nv_bfloat16>(a, s) : quantize<kNvFp4, float>(a, s);
}

cudaError_t launch_mx_dequantize(const MxDequantArgs &a, int format, bool bf16, cudaStream_t s) {
    if (format == kMxFp4) return bf16 ? dequantize<kMxFp4, __nv_bfloat16>(a, s) : dequantize<kMxFp4, float>(a, s);
    return bf16 ? dequantize<kNvFp4, __nv_bfloat16>(a, s) : dequantize<kNvFp4, float>(a, s);
}

}  // namespace moe
