// mx_common.cuh - the microscaled 4-bit formats: argument blocks, scale layout
// and the tcgen05 wrappers of block-scaled products.
//
// A row of cols elements is stored as cols / 2 bytes of E2M1 codes (two in a
// byte, the even column in the low four bits; magnitudes 0, 0.5, 1, 1.5, 2, 3,
// 4, 6, the sign in bit 3) and one scale byte per block:
//   MXFP4: blocks of 32, E8M0 scales 2^(byte - 127), 255 = NaN;
//   NVFP4: blocks of 16, E4M3 scales, times one power of two for the tensor.
// Scale bytes lie in tiles of 128 rows x 4 blocks, 512 bytes each, which is the
// order tcgen05.cp copies into TMEM: the byte of (row r, block j) is at
//   (r / 128 * SB + j / 4) * 512 + (r % 32) * 16 + (r % 128 / 32) * 4 + j % 4,
// SB = ceil(blocks per row / 4); the bytes of blocks past the row's end are 0.
#pragma once

#include "moe_common.cuh"

namespace moe {

enum { kMxFp4 = 0, kNvFp4 = 1 };

template <int FMT>
struct MxFormat {
    static constexpr int kBlock = FMT == kMxFp4 ? 32 : 16;  // elements per scale
    static constexpr int kTileK = 4 * kBlock;               // elements of K per 512-byte scale tile
};

__host__ __device__ __forceinline__ int mx_scale_tiles(int cols, int block) {
    return (cols + 4 * block - 1) / (4 * block);
}

struct MxQuantArgs {
    const void *x;             // [x_rows][ld] bf16 or fp32
    int64_t ld;
    int x_rows;
    const int32_t *row_index;  // [rows] source row of each output row (others are skipped), or null
    int rows, cols;
    float pre;                 // 2^-scale_exp
    uint8_t *codes;            // [rows][cols / 2]
    uint8_t *scales;           // tiles, or where `plain` rows of 4 SB bytes (for a gather that reads them)
    bool plain = false;
    void *values;              // [rows][values_ld] in x's type, or null
    int64_t values_ld;
    float post;                // 2^scale_exp
};
cudaError_t launch_mx_quantize(const MxQuantArgs &a, int format, bool bf16, int num_sms, cudaStream_t s);

// Gathers quantised rows: output row r is row row_index[r] of the source (others
// are skipped).
struct MxGatherArgs {
    const uint8_t *codes, *scales;  // src_rows x cols; scales in tiles, or where `plain` rows of 4 SB bytes
    bool plain = false;
    int src_rows, rows, cols;
    const int32_t *row_index;       // [rows]
    uint8_t *out_codes, *out_scales;
};
cudaError_t launch_mx_gather(const MxGatherArgs &a, int format, cudaStream_t s);

// Source rows for the rows of a layer's row space: `token` [rows] is the token of
// each kept assignment's row and of each shared expert's row, `self` the row itself;
// -1 for rows that hold nothing.
struct MxRowMapArgs {
    const int32_t *row_assign;   // [routed rows] t k + r, or -1
    const int32_t *group_start;  // [E + S + 1]
    int E, S, k, T, T_pad, rows;
    int32_t *token, *self;
};
cudaError_t launch_mx_row_map(const MxRowMapArgs &a, cudaStream_t s);

struct MxDequantArgs {
    const uint8_t *codes, *scales;
    int rows, cols;
    float post;
    void *out;
    int64_t ld;
};
cudaError_t launch_mx_dequantize(const MxDequantArgs &a, int format, bool bf16, cudaStream_t s);

struct MxGemmArgs {
    const int32_t *group_start, *group_rows;  // [G] or null (one group of all rows)
    int rows, N, K, G;
    int64_t filled;      // about how many of the rows belong to groups
    const float *bias;   // [G][N] or null
    const float *alpha;  // [G] or null
    float post;          // 2^scale_exp of both operands
    int act;             // activation code, -1 none
    void *out;
    int out_f32;
    int64_t out_ld;
    int vec_ok;          // bf16 outputs: out and out_ld allow 16-byte stores
    uint32_t *status;    // or null: the device's word for all such products
};
// Tensor maps of the codes (boxes of 128 bytes x 128 weight rows, 16 or 96 token
// rows) and of the scale tiles (boxes of one stage's tiles of one row block).
struct MxMaps {
    CUtensorMap w, a, a96, sw, sa;
};
// Whether a product runs in the form for short segments (which needs no 96-row map).
bool mx_gemm_narrow(const MxGemmArgs &a);
bool encode_mx_maps(MxMaps *m, bool narrow, int format, const void *a_codes, const void *a_scales, uint64_t rows, const void *w_codes,
                    const void *w_scales, uint64_t groups, int n, int k);
cudaError_t launch_mx_gemm(const MxMaps &m, const MxGemmArgs &a, int format, int num_sms, cudaStream_t s);

// Waits for the stream, reads the current device's word and clears the bits that were set.
cudaError_t mx_take_status(uint32_t *bits, cudaStream_t s);

// Device status bits the product adds to kDevTimeout.
enum : uint32_t { kDevBadGroup = 2u };

// ------------------------------------------------------------------ tcgen05

// Shared-memory descriptors as two words: the low one holds address >> 4 in
// bits [0,14) and the leading byte offset >> 4 in [16,30), so that a step through
// shared memory (below 256 KB) is an addition to it; the high one is constant.
// Operand tiles: K-major, 128B swizzle (see sw128_kmajor_desc).
constexpr uint32_t kOperandDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t operand_desc_lo(uint32_t smem_addr) { return (smem_addr >> 4) | (1u << 16); }
// A 512-byte scale tile (32 rows of 16 bytes, no swizzle, 8-row groups 128
// bytes apart) for tcgen05.cp.32x128b.
constexpr uint32_t kScaleDescHi = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t scale_desc_lo(uint32_t smem_addr) { return (smem_addr >> 4) | ((128u >> 4) << 16); }

// Copies a scale tile into 4 TMEM columns (32 lanes, repeated in the four lane
// quarters). Executes in order with the MMAs this thread issues after it.
template <int CG>
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint32_t desc_lo) {
    if constexpr (CG == 1)
        asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
                     "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr), "r"(desc_lo), "n"(kScaleDescHi)
                     : "memory");
    else
        asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
                     "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr), "r"(desc_lo), "n"(kScaleDescHi)
                     : "memory");
}

// Instruction descriptor of kind::mxf4 / kind::mxf4nvf4 with E2M1 operands,
// fp32 accumulation, K-major, shape M x N x 64: B scale id in [4,6), A format
// in [7,10) and B format in [10,12) (1 = E2M1), N >> 3 in [17,23), scale type
// in bit 23 (1 = UE8M0, 0 = UE4M3), M >> 7 in [27,29), A scale id in [29,31).
// The scale ids are or-ed in (mx_idesc_sf): which bytes of the 4-byte scale
// words the MMA uses.
template <int FMT>
__host__ __device__ constexpr uint32_t mx_idesc(int M, int N) {
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | ((FMT == kMxFp4 ? 1u : 0u) << 23) |
           (static_cast<uint32_t>(M >> 7) << 27);
}
__host__ __device__ constexpr uint32_t mx_idesc_sf(uint32_t id) { return (id << 4) | (id << 29); }

// D[tmem] (+)= (A * scale_a) (B * scale_b)^T over 64 elements of K.
template <int FMT, int CG>
__device__ __forceinline__ void tc_mma_mx(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
#define MOE_MX_MMA(KIND, CGS, VEC)                                                                            \
    asm volatile(                                                                                             \
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"                                                          \
        "setp.ne.b32 p, %6, 0;\n\t"                                                                           \
        "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"                                                    \
        "tcgen05.mma.cta_group::" CGS ".kind::" KIND ".block_scale.scale_vec::" VEC                           \
        " [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),                                                \
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kOperandDescHi)            \
        : "memory")
    if constexpr (FMT == kMxFp4 && CG == 1) MOE_MX_MMA("mxf4", "1", "2X");
    if constexpr (FMT == kMxFp4 && CG == 2) MOE_MX_MMA("mxf4", "2", "2X");
    if constexpr (FMT == kNvFp4 && CG == 1) MOE_MX_MMA("mxf4nvf4", "1", "4X");
    if constexpr (FMT == kNvFp4 && CG == 2) MOE_MX_MMA("mxf4nvf4", "2", "4X");
#undef MOE_MX_MMA
}

// The value of an E4M3 byte (0x7f and 0xff are NaN).
__device__ __forceinline__ float e4m3_value(uint32_t b) {
    const uint32_t e = (b >> 3) & 15u, m = b & 7u;
    if ((b & 0x7fu) == 0x7fu) return __uint_as_float(0x7fffffffu);
    return e ? __uint_as_float(((e + 120u) << 23) | (m << 20)) : static_cast<float>(m) * 0.001953125f;
}

// The value of an E8M0 byte.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    if (b == 255u) return __uint_as_float(0x7fffffffu);
    return b ? __uint_as_float(b << 23) : __uint_as_float(1u << 22);
}

}  // namespace moe
