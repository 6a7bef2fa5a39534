// MX4 matrices: quantize, dequantize and the product C = A B^T.
//
// Quantize and dequantize stream: 4 or 2 bytes per value on one side, 17/32 on the
// other. Along the rows of the values ("plain") four lanes share an MX block, 8 values
// each, so that a wave's loads and its 4-byte code stores are contiguous; the block's
// maximum goes over the four lanes by two DPP exchanges. Down the columns
// ("transposed") a wave holds one MX block of 128 columns: a lane reads two adjacent
// columns of 32 rows and finds their maxima in registers; the codes of 8 such waves
// (256 values of each column) are exchanged through LDS so that each row of codes is
// written 128 bytes at a time. Both are bound by HBM: along the rows 26 us for 30522 x 1024
// fp32 values (5.4 TB/s) and 44 us back for 11008 x 4096 (4.6); down the columns of 4096 x
// 11008 bf16 values 25 us and 23 us back (4.6 and 4.9).
#include "mx4_tile.h"

namespace meo {

namespace {

template <int N>
__device__ __forceinline__ const MxMat& mx_find(const MxBatchOf<N>& b, uint32_t block) {
    int i = 0;
    while (i + 1 < b.n && block >= b.m[i + 1].first) ++i;
    return b.m[i];
}

__device__ __forceinline__ uint32_t max_quad(uint32_t v) {
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xf, 0xf, true)));
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4E, 0xf, 0xf, true)));
}

}  // namespace

// Blocks of all rows are numbered through: block q is block q % nb of row q / nb.
template <bool BF>
__device__ __forceinline__ void quantize_rows(const MxMat& m, uint32_t tile) {
    const int64_t total = m.rows * m.nb;
    const int64_t b0 = static_cast<int64_t>(tile) * kMxRowBlocks + (threadIdx.x >> 2);
    const int sub = threadIdx.x & 3;
    float v[kMxRowIters][kVec];
#pragma unroll
    for (int k = 0; k < kMxRowIters; ++k) {
        const int64_t q = b0 + k * (kMxRowThreads / 4);
        const bool in = q < total;
        const int64_t row = in ? q / m.nb : 0, col = (in ? q - row * m.nb : 0) * kMxBlock + sub * kVec;
        const int valid = in ? static_cast<int>(min<int64_t>(max<int64_t>(m.cols - col, 0), kVec)) : 0;
        load_any8(m.data, row * m.ld + col, valid, BF, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kMxRowIters; ++k) {
        const int64_t q = b0 + k * (kMxRowThreads / 4);
        uint32_t a = 0;
#pragma unroll
        for (int e = 0; e < kVec; ++e) a = max(a, __float_as_uint(v[k][e]) & 0x7fffffffu);
        const uint32_t s = mx4_scale_byte(max_quad(a));
        const uint32_t c = mx4_pack8(v[k], s);
        if (q < total) {
            *gst<uint32_t>(m.codes + q * 16 + sub * 4) = c;
            if (sub == 0) *gst<uint8_t>(m.scales + q) = static_cast<uint8_t>(s);
        }
    }
}

template <int N>
__global__ __launch_bounds__(kMxRowThreads) void k_mx4_quantize_rows(MxBatchOf<N> b) {
    const MxMat& m = mx_find(b, blockIdx.x);
    if (m.bf16) quantize_rows<true>(m, blockIdx.x - m.first);
    else quantize_rows<false>(m, blockIdx.x - m.first);
}

template <bool BF>
__device__ __forceinline__ void dequantize_rows(const MxMat& m, uint32_t tile) {
    const int64_t total = m.rows * m.nb;
    const int64_t b0 = static_cast<int64_t>(tile) * kMxRowBlocks + (threadIdx.x >> 2);
    const int sub = threadIdx.x & 3;
    uint32_t c[kMxRowIters], s[kMxRowIters];
#pragma unroll
    for (int k = 0; k < kMxRowIters; ++k) {
        const int64_t q = min(b0 + k * (kMxRowThreads / 4), total - 1);
        c[k] = *gld<uint32_t>(m.codes + q * 16 + sub * 4);
        s[k] = *gld<uint8_t>(m.scales + q);
    }
#pragma unroll
    for (int k = 0; k < kMxRowIters; ++k) {
        const int64_t q = b0 + k * (kMxRowThreads / 4);
        if (q >= total) continue;
        const int64_t row = q / m.nb, col = (q - row * m.nb) * kMxBlock + sub * kVec;
        const int valid = static_cast<int>(min<int64_t>(max<int64_t>(m.cols - col, 0), kVec));
        float v[kVec];
        mx4_unpack8(c[k], mx4_scale(s[k]), v);
        store_any8(const_cast<void*>(m.data), row * m.ld + col, valid, BF, v);
    }
}

template <int N>
__global__ __launch_bounds__(kMxRowThreads) void k_mx4_dequantize_rows(MxBatchOf<N> b) {
    const MxMat& m = mx_find(b, blockIdx.x);
    if (m.bf16) dequantize_rows<true>(m, blockIdx.x - m.first);
    else dequantize_rows<false>(m, blockIdx.x - m.first);
}

namespace {

// Two adjacent values of a row of the data: Whole, one aligned access; else the `valid` first
// of them, zero where out of range.
template <bool BF, bool Whole>
__device__ __forceinline__ void load_pair(const MxMat& m, int64_t row, int64_t col, int valid, float& x, float& y) {
    const int64_t i = row * m.ld + col;
    if (BF) {
        const uint16_t* p = static_cast<const uint16_t*>(m.data) + i;
        if constexpr (Whole) {
            const uint32_t w = *gld<uint32_t>(p);
            x = bf16_lo(w);
            y = bf16_hi(w);
        } else {
            x = valid > 0 ? __uint_as_float(static_cast<uint32_t>(*gld<uint16_t>(p)) << 16) : 0.0f;
            y = valid > 1 ? __uint_as_float(static_cast<uint32_t>(*gld<uint16_t>(p + 1)) << 16) : 0.0f;
        }
    } else {
        const float* p = static_cast<const float*>(m.data) + i;
        if constexpr (Whole) {
            const f32x2 w = *gld<f32x2>(p);
            x = w.x;
            y = w.y;
        } else {
            x = valid > 0 ? *gld<float>(p) : 0.0f;
            y = valid > 1 ? *gld<float>(p + 1) : 0.0f;
        }
    }
}

constexpr int kMxColPitch = kMxColBlocks * 16 + 16;  // bytes of codes per LDS row (padded)

}  // namespace

// Tile: kMxColRows rows of the MX4 matrix (columns of the data) x kMxColBlocks blocks.
template <bool BF>
__device__ __forceinline__ void quantize_cols(const MxMat& m, uint32_t tile, uint8_t* lc, uint8_t* ls) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r0 = static_cast<int64_t>(tile % m.tiles_y) * kMxColRows;
    const int64_t k0 = static_cast<int64_t>(tile / m.tiles_y) * kMxColBlocks;
    const int64_t row = r0 + 2 * lane, kb = k0 + wave;
    const int valid = static_cast<int>(min<int64_t>(max<int64_t>(m.rows - row, 0), 2));
    float x[kMxBlock], y[kMxBlock];
    if (m.pairs && r0 + kMxColRows <= m.rows && (k0 + kMxColBlocks) * kMxBlock <= m.cols) {
#pragma unroll
        for (int i = 0; i < kMxBlock; ++i) load_pair<BF, true>(m, kb * kMxBlock + i, row, 2, x[i], y[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kMxBlock; ++i) {
            const int64_t k = kb * kMxBlock + i;
            load_pair<BF, false>(m, k, row, k < m.cols ? valid : 0, x[i], y[i]);
        }
    }
    uint32_t ax = 0, ay = 0;
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) {
        ax = max(ax, __float_as_uint(x[i]) & 0x7fffffffu);
        ay = max(ay, __float_as_uint(y[i]) & 0x7fffffffu);
    }
    const uint32_t sx = mx4_scale_byte(ax), sy = mx4_scale_byte(ay);
    u32x4 cx, cy;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        cx[i] = mx4_pack8(x + 8 * i, sx);
        cy[i] = mx4_pack8(y + 8 * i, sy);
    }
    *reinterpret_cast<u32x4*>(lc + (2 * lane) * kMxColPitch + wave * 16) = cx;
    *reinterpret_cast<u32x4*>(lc + (2 * lane + 1) * kMxColPitch + wave * 16) = cy;
    ls[(2 * lane) * kMxColBlocks + wave] = static_cast<uint8_t>(sx);
    ls[(2 * lane + 1) * kMxColBlocks + wave] = static_cast<uint8_t>(sy);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMxColRows * kMxColBlocks / kMxColThreads; ++i) {
        const int c = threadIdx.x + i * kMxColThreads;
        const int lr = c / kMxColBlocks, lb = c % kMxColBlocks;
        if (r0 + lr < m.rows && k0 + lb < m.nb) {
            const int64_t q = (r0 + lr) * m.nb + k0 + lb;
            *gst<u32x4>(m.codes + q * 16) = *reinterpret_cast<const u32x4*>(lc + lr * kMxColPitch + lb * 16);
            *gst<uint8_t>(m.scales + q) = ls[c];
        }
    }
}

template <int N>
__global__ __launch_bounds__(kMxColThreads) void k_mx4_quantize_cols(MxBatchOf<N> b) {
    __shared__ __attribute__((aligned(16))) uint8_t lc[kMxColRows * kMxColPitch];
    __shared__ uint8_t ls[kMxColRows * kMxColBlocks];
    const MxMat& m = mx_find(b, blockIdx.x);
    if (m.bf16) quantize_cols<true>(m, blockIdx.x - m.first, lc, ls);
    else quantize_cols<false>(m, blockIdx.x - m.first, lc, ls);
}

template <bool BF>
__device__ __forceinline__ void dequantize_cols(const MxMat& m, uint32_t tile, uint8_t* lc, uint8_t* ls) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r0 = static_cast<int64_t>(tile % m.tiles_y) * kMxColRows;
    const int64_t k0 = static_cast<int64_t>(tile / m.tiles_y) * kMxColBlocks;
#pragma unroll
    for (int i = 0; i < kMxColRows * kMxColBlocks / kMxColThreads; ++i) {
        const int c = threadIdx.x + i * kMxColThreads;
        const int lr = c / kMxColBlocks, lb = c % kMxColBlocks;
        if (r0 + lr < m.rows && k0 + lb < m.nb) {
            const int64_t q = (r0 + lr) * m.nb + k0 + lb;
            *reinterpret_cast<u32x4*>(lc + lr * kMxColPitch + lb * 16) = *gld<u32x4>(m.codes + q * 16);
            ls[c] = *gld<uint8_t>(m.scales + q);
        }
    }
    __syncthreads();
    const int64_t row = r0 + 2 * lane, kb = k0 + wave;
    const int valid = static_cast<int>(min<int64_t>(max<int64_t>(m.rows - row, 0), 2));
    if (valid == 0 || kb >= m.nb) return;
    const u32x4 cx = *reinterpret_cast<const u32x4*>(lc + (2 * lane) * kMxColPitch + wave * 16);
    const u32x4 cy = *reinterpret_cast<const u32x4*>(lc + (2 * lane + 1) * kMxColPitch + wave * 16);
    const float sx = mx4_scale(ls[(2 * lane) * kMxColBlocks + wave]);
    const float sy = mx4_scale(ls[(2 * lane + 1) * kMxColBlocks + wave]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x[kVec], y[kVec];
        mx4_unpack8(cx[i], sx, x);
        mx4_unpack8(cy[i], sy, y);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const int64_t k = kb * kMxBlock + 8 * i + e;
            if (k >= m.cols) continue;
            const int64_t at = k * m.ld + row;
            if (BF) {
                uint16_t* p = static_cast<uint16_t*>(const_cast<void*>(m.data)) + at;
                if (m.pairs && valid == 2) {
                    *gst<uint32_t>(p) = bf16_bits(x[e]) | (bf16_bits(y[e]) << 16);
                } else {
                    *gst<uint16_t>(p) = static_cast<uint16_t>(bf16_bits(x[e]));
                    if (valid > 1) *gst<uint16_t>(p + 1) = static_cast<uint16_t>(bf16_bits(y[e]));
                }
            } else {
                float* p = static_cast<float*>(const_cast<void*>(m.data)) + at;
                if (m.pairs && valid == 2) {
                    *gst<f32x2>(p) = f32x2{x[e], y[e]};
                } else {
                    *gst<float>(p) = x[e];
                    if (valid > 1) *gst<float>(p + 1) = y[e];
                }
            }
        }
    }
}

template <int N>
__global__ __launch_bounds__(kMxColThreads) void k_mx4_dequantize_cols(MxBatchOf<N> b) {
    __shared__ __attribute__((aligned(16))) uint8_t lc[kMxColRows * kMxColPitch];
    __shared__ uint8_t ls[kMxColRows * kMxColBlocks];
    const MxMat& m = mx_find(b, blockIdx.x);
    if (m.bf16) dequantize_cols<true>(m, blockIdx.x - m.first, lc, ls);
    else dequantize_cols<false>(m, blockIdx.x - m.first, lc, ls);
}

namespace {

MxBatchOf<1> only(const MxBatch& b) { return MxBatchOf<1>{1, {b.m[0]}}; }
MxProdBatchOf<1> only(const MxProdBatch& b) { return MxProdBatchOf<1>{1, {b.p[0]}}; }

}  // namespace

void launch_mx4_quantize(const MxBatch& b, uint32_t grid, bool transposed, hipStream_t s) {
    if (grid == 0) return;
    const dim3 g(grid), t(transposed ? kMxColThreads : kMxRowThreads);
    if (b.n == 1 && transposed) hipLaunchKernelGGL(k_mx4_quantize_cols<1>, g, t, 0, s, only(b));
    else if (b.n == 1) hipLaunchKernelGGL(k_mx4_quantize_rows<1>, g, t, 0, s, only(b));
    else if (transposed) hipLaunchKernelGGL(k_mx4_quantize_cols<kMxBatch>, g, t, 0, s, b);
    else hipLaunchKernelGGL(k_mx4_quantize_rows<kMxBatch>, g, t, 0, s, b);
}

void launch_mx4_dequantize(const MxBatch& b, uint32_t grid, bool transposed, hipStream_t s) {
    if (grid == 0) return;
    const dim3 g(grid), t(transposed ? kMxColThreads : kMxRowThreads);
    if (b.n == 1 && transposed) hipLaunchKernelGGL(k_mx4_dequantize_cols<1>, g, t, 0, s, only(b));
    else if (b.n == 1) hipLaunchKernelGGL(k_mx4_dequantize_rows<1>, g, t, 0, s, only(b));
    else if (transposed) hipLaunchKernelGGL(k_mx4_dequantize_cols<kMxBatch>, g, t, 0, s, b);
    else hipLaunchKernelGGL(k_mx4_dequantize_rows<kMxBatch>, g, t, 0, s, b);
}

// ----------------------------------------------------------------------------- product

// C = A B^T, stored from the accumulators: 32 consecutive values of two rows per
// instruction. Tiles (MxForm): 128 rows x 256 columns of 8 waves where that fills the GPU,
// 64 x 256 otherwise and 64 x 128 of 4 waves for products of at most 128 columns (32000 x 128 x
// 4096: 25 us, in 256-column tiles 29). 32000 x 256 x 4096 with fp32 outputs takes 33 us, 3.1
// TB/s: its 250 tiles run at once, and all write their part of C's 33 MB at the end.
template <int IB, bool BF>
__device__ __forceinline__ void mx4_store(const MxProd& p, int64_t i0, int64_t j0, int lane, const f32x16 (&acc)[IB][2]) {
    const bool whole = i0 + 32 * IB <= p.m && j0 + 64 <= p.n;
#pragma unroll
    for (int jb = 0; jb < 2; ++jb) {
        const int64_t col = j0 + jb * 32 + (lane & 31);
        if (!whole && col >= p.n) continue;
#pragma unroll
        for (int ib = 0; ib < IB; ++ib)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int64_t row = i0 + ib * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
                if (!whole && row >= p.m) continue;
                if (BF) *gst<uint16_t>(static_cast<uint16_t*>(p.c) + row * p.ldc + col) = static_cast<uint16_t>(bf16_bits(acc[ib][jb][v]));
                else *gst<float>(static_cast<float*>(p.c) + row * p.ldc + col) = acc[ib][jb][v];
            }
    }
}

template <int IB, int WN, int NW, int N>
__global__ __launch_bounds__(NW * 64) void k_mx4_matmul(MxProdBatchOf<N> b) {
    using T = MxTile<IB, WN, NW>;
    __shared__ __attribute__((aligned(16))) uint8_t lds[T::kLds];
    int i = 0;
    while (i + 1 < b.n && blockIdx.x >= b.p[i + 1].first) ++i;
    const MxProd& p = b.p[i];
    const uint32_t tile = blockIdx.x - p.first;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    int64_t i0 = static_cast<int64_t>(uniform(static_cast<int>(tile / p.tn))) * T::kRowsA;
    int64_t j0 = static_cast<int64_t>(uniform(static_cast<int>(tile % p.tn))) * T::kRowsB;
    f32x16 acc[IB][2];
#pragma unroll
    for (int ib = 0; ib < IB; ++ib)
#pragma unroll
        for (int jb = 0; jb < 2; ++jb)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[ib][jb][v] = 0.0f;
    const MxOperand oa{p.ac, p.as, p.m, static_cast<int32_t>(p.nb)}, ob{p.bc, p.bs, p.n, static_cast<int32_t>(p.nb)};
    mx4_accumulate<IB, WN, NW>(oa, ob, i0, j0, lds, acc);
    i0 += (wave / WN) * 32 * IB;
    j0 += (wave % WN) * 64;
    if (p.cbf16) mx4_store<IB, true>(p, i0, j0, lane, acc);
    else mx4_store<IB, false>(p, i0, j0, lane, acc);
}

template <int IB, int WN, int NW>
static void launch_matmul(const MxProdBatch& b, uint32_t grid, hipStream_t s) {
    if (b.n == 1) hipLaunchKernelGGL((k_mx4_matmul<IB, WN, NW, 1>), dim3(grid), dim3(NW * 64), 0, s, only(b));
    else hipLaunchKernelGGL((k_mx4_matmul<IB, WN, NW, kMxBatch>), dim3(grid), dim3(NW * 64), 0, s, b);
}

void launch_mx4_matmul(const MxProdBatch& b, uint32_t grid, MxForm form, hipStream_t s) {
    if (grid == 0) return;
    switch (form) {
        case kMxNarrow: launch_matmul<1, 2, 4>(b, grid, s); break;
        case kMxWide: launch_matmul<1, 4, 8>(b, grid, s); break;
        default: launch_matmul<2, 4, 8>(b, grid, s); break;
    }
}

}  // namespace meo
