// Device helpers shared by the GaLore kernels (bf16 and MX4 projectors): MFMA fragments,
// staging, the epilogue exchange and AdamW on a piece of the low-rank gradient.
#pragma once
#include "galore.h"

#include <type_traits>

namespace meo {

typedef __bf16 bfv8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32(const bfv8& a, const bfv8& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 8 bf16 (raw bits) of row `row` starting at column `col` of a row-major [rows][cols]
// array; out-of-range elements read 0.
__device__ __forceinline__ u32x4 ld_row8(const uint16_t* p, int64_t rows, int64_t cols, int64_t row,
                                         int64_t col, bool vec) {
    if (row >= rows || col >= cols) return u32x4{0u, 0u, 0u, 0u};
    const uint16_t* q = p + row * cols + col;
    if (vec && col + 8 <= cols) return *gld<u32x4>(q);
    const MEO_GLOBAL uint16_t* s = gld<uint16_t>(q);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t lo = col + 2 * e < cols ? s[2 * e] : 0u;
        const uint32_t hi = col + 2 * e + 1 < cols ? s[2 * e + 1] : 0u;
        w[e] = lo | (hi << 16);
    }
    return u32x4{w[0], w[1], w[2], w[3]};
}

__device__ __forceinline__ void st_lds8(uint16_t* p, const u32x4& v) {
    *reinterpret_cast<u32x4*>(p) = v;
}

__device__ __forceinline__ bfv8 ld_frag(const uint16_t* p) {
    return *reinterpret_cast<const bfv8*>(p);
}

// Rows [r0, r0 + NROWS) x contraction columns [k0, k0 + kGaKb) of a row-major
// [rows][cols] bf16 array, zero outside it: loaded into registers first (all of a
// thread's chunks in flight at once, and the next block's while the current one
// is multiplied), then written to LDS (row pitch kGaPitch).
template <int NROWS, int THREADS = kThreads>
struct RowStage {
    static constexpr int kPer = NROWS * (kGaKb / 8) / THREADS;
    u32x4 v[kPer];
    __device__ __forceinline__ void load(const uint16_t* p, int64_t rows, int64_t cols, int64_t r0, int64_t k0,
                                         bool vec) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = threadIdx.x + i * THREADS;
            v[i] = ld_row8(p, rows, cols, r0 + (c >> 3), k0 + (c & 7) * 8, vec);
        }
    }
    __device__ __forceinline__ void store(uint16_t* lds) const {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = threadIdx.x + i * THREADS;
            st_lds8(lds + (c >> 3) * kGaPitch + (c & 7) * 8, v[i]);
        }
    }
};

// The transposed tile A[i][k] = G[k0 + k][i0 + i] (i < kGaTile, k < kGaKb) of the
// row-major gradient G [K][D]: loaded along G's rows, scattered into LDS.
template <int IROWS>
struct TransStage {
    static constexpr int kRowChunks = IROWS / 8;  // 16-byte chunks per row of G
    static constexpr int kPer = kGaKb * kRowChunks / kThreads;
    u32x4 v[kPer];
    __device__ __forceinline__ void load(const uint16_t* g, int64_t K, int64_t D, int64_t i0, int64_t k0, bool vec) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = threadIdx.x + i * kThreads;
            v[i] = ld_row8(g, K, D, k0 + c / kRowChunks, i0 + (c % kRowChunks) * 8, vec);
        }
    }
    __device__ __forceinline__ void store(uint16_t* lds) const {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = threadIdx.x + i * kThreads;
            const int k = c / kRowChunks, ic = (c % kRowChunks) * 8;
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lds[(ic + 2 * e) * kGaPitch + k] = static_cast<uint16_t>(w[e] & 0xffffu);
                lds[(ic + 2 * e + 1) * kGaPitch + k] = static_cast<uint16_t>(w[e] >> 16);
            }
        }
    }
};

// Accumulator element v of a 32x32 block held by `lane`: row and column in the block.
__device__ __forceinline__ int acc_row(int v, int lane) { return 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3); }
__device__ __forceinline__ int acc_col(int lane) { return lane & 31; }

// Epilogue exchange: a wave's 32 x 64 half tile (accumulator blocks (ib, 0) and
// (ib, 1)) goes through LDS so that each lane then holds 8 consecutive columns
// of a row, for 16-byte loads and stores of the row-major outputs. Lane l gets
// rows (l >> 3) + 8 q (q < 4) and columns 8 (l & 7) .. 8 (l & 7) + 7. Only the
// wave itself touches its LDS region, and its LDS accesses run in program order.
constexpr int kEpPitch = 68;  // floats per LDS row of the exchange
constexpr int kEpWave = 32 * kEpPitch;

__device__ __forceinline__ void ep_spill(const f32x16& a0, const f32x16& a1, float* lw, int lane) {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        lw[acc_row(v, lane) * kEpPitch + (lane & 31)] = a0[v];
        lw[acc_row(v, lane) * kEpPitch + 32 + (lane & 31)] = a1[v];
    }
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ void ep_gather(const float* lw, int lane, int q, float* c) {
    const float* p = lw + ((lane >> 3) + 8 * q) * kEpPitch + (lane & 7) * 8;
    const f32x4 x0 = *reinterpret_cast<const f32x4*>(p);
    const f32x4 x1 = *reinterpret_cast<const f32x4*>(p + 4);
    c[0] = x0.x; c[1] = x0.y; c[2] = x0.z; c[3] = x0.w;
    c[4] = x1.x; c[5] = x1.y; c[6] = x1.z; c[7] = x1.w;
    __builtin_amdgcn_wave_barrier();
}

// ------------------------------------------------------------------ projection + AdamW

// Direct staging: rows of 64 bf16 (128 bytes, unpadded) written straight from
// global memory into LDS by global_load_lds (no registers), 8 rows per
// instruction: lane l fills row (l >> 3) of the group at 16-byte slot (l & 7),
// which holds the row's chunk (l & 7) ^ sw_row(row). A fragment read (16 lanes per
// LDS cycle on 64 banks: 16 consecutive rows, one chunk each) then finds rows r and
// r + 8 on different slots as well as the 8 rows of each parity: no bank conflict
// (with sw_row(r) = r & 7 alone rows r and r + 8 collided, which doubled the LDS
// cycles of the projection). Rows past the operand's end read its last row: they
// only reach outputs that are not stored.
constexpr int kDirectPitch = kGaKb;  // bf16 per LDS row
__device__ __forceinline__ int sw_row(int r) { return (r & 7) ^ ((r >> 3) & 1); }
template <int ROWS, int THREADS = kThreads>
__device__ __forceinline__ void stage_direct(const uint16_t* g, int64_t nrows, int64_t cols, int64_t r0, int k0,
                                             uint16_t* dst, int wave, int lane) {
#pragma unroll
    for (int j = wave; j < ROWS / 8; j += THREADS / 64) {
        const int rr = 8 * j + (lane >> 3);
        const int64_t row = min(r0 + rr, nrows - 1);
        const int c = (lane & 7) ^ sw_row(rr);
        const uint16_t* src = g + row * cols + k0 + c * 8;
        __builtin_amdgcn_global_load_lds((const MEO_GLOBAL void*)src,
                                         (__attribute__((address_space(3))) void*)(dst + 8 * j * kDirectPitch),
                                         16, 0, 0);
    }
}

__device__ __forceinline__ bfv8 ld_frag_sw(const uint16_t* base, int row, int kk) {
    return *reinterpret_cast<const bfv8*>(base + row * kDirectPitch + (((kk >> 3) ^ sw_row(row)) << 3));
}


__device__ __forceinline__ void galore_adamw8(const GDesc& d, const GaArgs& a, int64_t row, int col, const float* rv) {
    float m[8], v[8], nh[8], nl[8];
    const int64_t idx = row * d.r + col;
    const bool full = d.rvec && col + 8 <= d.r;
    if (full) {
        const f32x4 m0 = *gld<f32x4>(d.em + idx), m1 = *gld<f32x4>(d.em + idx + 4);
        const f32x4 v0 = *gld<f32x4>(d.ev + idx), v1 = *gld<f32x4>(d.ev + idx + 4);
        m[0] = m0.x; m[1] = m0.y; m[2] = m0.z; m[3] = m0.w; m[4] = m1.x; m[5] = m1.y; m[6] = m1.z; m[7] = m1.w;
        v[0] = v0.x; v[1] = v0.y; v[2] = v0.z; v[3] = v0.w; v[4] = v1.x; v[5] = v1.y; v[6] = v1.z; v[7] = v1.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            m[e] = col + e < d.r ? *gld<float>(d.em + idx + e) : 0.0f;
            v[e] = col + e < d.r ? *gld<float>(d.ev + idx + e) : 0.0f;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        m[e] = fmaf(a.beta1, m[e], a.omb1 * rv[e]);
        v[e] = fmaf(a.beta2, v[e], a.omb2 * (rv[e] * rv[e]));
        const float n = (m[e] * a.inv_bc1) / (sqrtf(v[e] * a.inv_bc2) + a.eps);
        nh[e] = round_bf16(n);
        nl[e] = n - nh[e];
    }
    if (full) {
        *gst<f32x4>(d.em + idx) = f32x4{m[0], m[1], m[2], m[3]};
        *gst<f32x4>(d.em + idx + 4) = f32x4{m[4], m[5], m[6], m[7]};
        *gst<f32x4>(d.ev + idx) = f32x4{v[0], v[1], v[2], v[3]};
        *gst<f32x4>(d.ev + idx + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < d.r) {
                *gst<float>(d.em + idx + e) = m[e];
                *gst<float>(d.ev + idx + e) = v[e];
            }
    }
    if (d.vec && col + 8 <= d.r) {  // the planes are 256-byte aligned; rows of r % 8 == 0
        *gst<u32x4>(d.nh + idx) = pack_bf16x8(nh);
        *gst<u32x4>(d.nl + idx) = pack_bf16x8(nl);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < d.r) {
                *gst<uint16_t>(d.nh + idx + e) = static_cast<uint16_t>(bf16_bits(nh[e]));
                *gst<uint16_t>(d.nl + idx + e) = static_cast<uint16_t>(bf16_bits(nl[e]));
            }
    }
}

// A wave's 32 x 32 exchange block in LDS, unpadded: row r at row r ^ ((r >> 2) & 1), its
// 16-byte chunk c at chunk c ^ ((r >> 1) & 1), so that neither the accumulator spill
// (rows r and r + 4 at once) nor the 8-column gather (rows 4k .. 4k + 3) hits a bank twice.
__device__ __forceinline__ int ur_ex(int r, int col) {
    return ((r ^ ((r >> 2) & 1)) << 5) + ((((col >> 2) ^ ((r >> 1) & 1))) << 2) + (col & 3);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// s_waitcnt with only the vector-memory count (gfx9 encoding: vmcnt in bits 3:0 and
// 15:14, expcnt 6:4 and lgkmcnt 11:8 left at their no-wait maxima).
#define MEO_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (((n) >> 4) << 14) | (7 << 4) | (15 << 8))

}  // namespace meo
