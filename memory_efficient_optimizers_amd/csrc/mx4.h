// MX4 (microscaling MXFP4) matrices: descriptors, launchers and device helpers.
//
// A matrix [rows][cols] is held as blocks of 32 consecutive values of a row. Block k of
// a row has 16 bytes of codes (value 2i in the low nibble of byte i) and one scale byte
// e, the power of two 2^(e - 127); a code is a sign bit and one of 0, 0.5, 1, 1.5, 2, 3,
// 4, 6. Rows of codes are 16 ceil(cols / 32) bytes, rows of scales ceil(cols / 32);
// the last block of a row is filled with zero codes.
#pragma once
#include "internal.h"

namespace meo {

constexpr int kMxBlock = 32;   // values per scale
constexpr int64_t mx_max_grid(int threads) { return 0xffffffffLL / threads; }  // a launch has fewer than 2^32 threads
constexpr int64_t kMxMaxK = 1 << 23;  // longest contraction of a product (32-bit offsets in a tile)
constexpr int kMxBatch = 32;   // matrices per launch (their descriptors are kernel arguments; one
                               // alone goes by itself: 2.7 us a launch, 4.0 us with all 32)

// One matrix of a quantize or dequantize call.
struct MxMat {
    const void* data;    // values: [rows][ld], or [cols][ld] when transposed
    uint8_t* codes;
    uint8_t* scales;
    int64_t ld;
    int64_t rows, cols;  // of the MX4 matrix: blocks run along cols
    int64_t nb;          // blocks per row
    uint32_t first;      // the matrix's first block in the launch
    uint32_t tiles_y;    // transposed: tiles along rows
    int32_t bf16;        // values are bf16 (else fp32)
    int32_t pairs;       // transposed: adjacent values of even columns allow one access
};

template <int N>
struct MxBatchOf {
    int32_t n;
    MxMat m[N];
};
using MxBatch = MxBatchOf<kMxBatch>;

constexpr int kMxRowThreads = 256;
constexpr int kMxRowIters = 4;
constexpr int64_t kMxRowBlocks = kMxRowThreads / 4 * kMxRowIters;  // MX blocks per thread block (plain)
constexpr int kMxColThreads = 512;                                 // transposed: 8 waves, one MX block each
constexpr int kMxColRows = 128;                                    // rows (columns of the values) per tile
constexpr int kMxColBlocks = kMxColThreads / 64;                   // MX blocks per row and tile

void launch_mx4_quantize(const MxBatch& b, uint32_t grid, bool transposed, hipStream_t s);
void launch_mx4_dequantize(const MxBatch& b, uint32_t grid, bool transposed, hipStream_t s);

// One product C = A B^T of a matmul call.
struct MxProd {
    const uint8_t *ac, *as;  // A [m][k]
    const uint8_t *bc, *bs;  // B [n][k]
    void* c;                 // [m][ldc]
    int64_t ldc;
    int64_t m, n;
    int64_t nb;              // blocks along k
    uint32_t first;          // the product's first block in the launch
    uint32_t tn;             // tiles along n
    int32_t cbf16;
};

template <int N>
struct MxProdBatchOf {
    int32_t n;
    MxProd p[N];
};
using MxProdBatch = MxProdBatchOf<kMxBatch>;

// Tile of a product (rows x columns of C): for at most 128 columns; more; more, and enough
// rows that 128 at a time fill the GPU.
enum MxForm { kMxNarrow = 0, kMxWide, kMxTall, kMxForms };
constexpr int kMxFormRows[kMxForms] = {64, 64, 128};
constexpr int kMxFormCols[kMxForms] = {128, 256, 256};
constexpr int kMxFormThreads[kMxForms] = {256, 512, 512};

void launch_mx4_matmul(const MxProdBatch& b, uint32_t grid, MxForm form, hipStream_t s);

// ----------------------------------------------------------------------------- device

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// C += A B over 64 values of the contraction. Lane l holds one MX block of each operand
// (row l & 31, block l >> 5: 16 bytes of codes) and its scale as byte T of sa and sb. The
// products are exact and the sums fp32.
template <int T>
__device__ __forceinline__ f32x16 mfma_mx4(const u32x4& a, const u32x4& b, const f32x16& c, uint32_t sa, uint32_t sb) {
    const i32x8 x = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w), 0, 0, 0, 0};
    const i32x8 y = {static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w), 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, T, sa, T, sb);
}

// 16-byte accesses at any element's address (the GPU's unaligned access mode): rows of any
// length and views of any offset move as whole ones do.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// 8 values of an fp32 or bf16 array at element i, widened to fp32; the first `valid` of them are
// in range, the rest read 0. And the same stored, bf16 rounded to nearest even.
__device__ __forceinline__ void load_any8(const void* p, int64_t i, int valid, bool bf16, float* f) {
    if (bf16) {
        const uint16_t* q = static_cast<const uint16_t*>(p) + i;
        if (valid == kVec) {
            bf16x8(*gld<u32x4_any>(q), f);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) f[e] = e < valid ? __uint_as_float(static_cast<uint32_t>(*gld<uint16_t>(q + e)) << 16) : 0.0f;
        }
    } else {
        const float* q = static_cast<const float*>(p) + i;
        if (valid == kVec) {
            const f32x4 a = *gld<f32x4_any>(q), b = *gld<f32x4_any>(q + 4);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) f[e] = e < valid ? *gld<float>(q + e) : 0.0f;
        }
    }
}
__device__ __forceinline__ void store_any8(void* p, int64_t i, int valid, bool bf16, const float* f) {
    if (bf16) {
        uint16_t* q = static_cast<uint16_t*>(p) + i;
        if (valid == kVec) {
            *gst<u32x4_any>(q) = pack_bf16x8(f);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (e < valid) *gst<uint16_t>(q + e) = static_cast<uint16_t>(bf16_bits(f[e]));
        }
    } else {
        float* q = static_cast<float*>(p) + i;
        if (valid == kVec) {
            *gst<f32x4_any>(q) = f32x4{f[0], f[1], f[2], f[3]};
            *gst<f32x4_any>(q + 4) = f32x4{f[4], f[5], f[6], f[7]};
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (e < valid) *gst<float>(q + e) = f[e];
        }
    }
}

// 2^(e - 127) as fp32: e = 0 is a subnormal, e = 255 a NaN.
__device__ __forceinline__ float mx4_scale(uint32_t e) {
    return e == 255 ? __uint_as_float(0x7fc00000u) : (e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23));
}

// The largest magnitude's bits (0 for zeros; NaN and infinity compare above every finite
// value) of a block -> its scale byte: floor(log2 amax) - 2, so that amax is 4 to 8 (6 is
// the largest code: larger values saturate), at least 2^-127; 255 for a NaN or infinity.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 255;
    const int e = static_cast<int>(amax_bits >> 23) - 2;
    return e < 0 ? 0u : static_cast<uint32_t>(e);
}

// 8 values times 2^-(e - 127) to the nearest codes (ties to even, saturating), the first
// in the low nibble. The product with the power of two is exact where it matters: below
// 2^-126 it rounds, but such values are far below half of the smallest code.
__device__ __forceinline__ uint32_t mx4_pack8(const float* v, uint32_t e) {
    if (e == 255) return 0;
    const float inv = __uint_as_float((254u - e) << 23);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0] * inv, v[1] * inv, 1.0f, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2] * inv, v[3] * inv, 1.0f, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4] * inv, v[5] * inv, 1.0f, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6] * inv, v[7] * inv, 1.0f, 3);
    return q;
}

// 8 codes times their scale, in fp32 (exact unless the product leaves fp32's range).
__device__ __forceinline__ void mx4_unpack8(uint32_t q, float scale, float* v) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
    v[0] = a.x * scale; v[1] = a.y * scale; v[2] = b.x * scale; v[3] = b.y * scale;
    v[4] = c.x * scale; v[5] = c.y * scale; v[6] = d.x * scale; v[7] = d.y * scale;
}

}  // namespace meo
