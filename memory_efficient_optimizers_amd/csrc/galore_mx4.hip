// GaLore's projection with an MX4 projector. The step is that of galore.hip,
//
//   m >= n: R = G U,   W <- W (1 - lr wd) - lr scale N U^T
//   m <  n: R = G^T U, W <- W (1 - lr wd) - lr scale U N^T,
//
// with AdamW's direction N of R, but the projector U is held once, as U^T [r][d] in MX4
// (17/32 byte per value instead of two bf16 copies). Both products decode it on the way
// to the matrix cores: a code times its power-of-two scale is exact in bf16, so the bf16
// products are those of the values that the codes stand for. A gradient in MX4 is
// multiplied in its own form on the scaled matrix instructions.
#include "galore_dev.h"
#include "mx4_tile.h"

namespace meo {

namespace {

// AdamW on 8 columns of a row of R (galore_adamw8 with N's planes in rows of rp values): the
// moments up to column r, the planes up to rp, zero past r.
__device__ __forceinline__ void gx_adamw8(const GxDesc& d, const GaArgs& a, int64_t row, int col, const float* rv) {
    float m[8], v[8], nh[8], nl[8];
    const int valid = min(max(d.r - col, 0), 8);
    const int64_t idx = row * d.r + col;
    load_f8(d.em + idx, valid, d.rvec, m);
    load_f8(d.ev + idx, valid, d.rvec, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        m[e] = fmaf(a.beta1, m[e], a.omb1 * rv[e]);
        v[e] = fmaf(a.beta2, v[e], a.omb2 * (rv[e] * rv[e]));
        const float n = e < valid ? (m[e] * a.inv_bc1) / (sqrtf(v[e] * a.inv_bc2) + a.eps) : 0.0f;
        nh[e] = round_bf16(n);
        nl[e] = n - nh[e];
    }
    store_f8(d.em + idx, valid, d.rvec, m);
    store_f8(d.ev + idx, valid, d.rvec, v);
    const int64_t at = row * d.rp + col;  // the planes are 256-byte aligned, rp a multiple of 16
    *gst<u32x4>(d.nh + at) = pack_bf16x8(nh);
    *gst<u32x4>(d.nl + at) = pack_bf16x8(nl);
}

constexpr int kGxEx = 32 * 32;  // floats of a wave's exchange region

// A wave's 32 x 32 exchange block, unpadded (as the back-projection's): conflict-free for
// the accumulator spill and for the gather of 8 columns of a row.
__device__ __forceinline__ int gx_ex(int r, int col) {
    return ((r ^ ((r >> 2) & 1)) << 5) + ((((col >> 2) ^ ((r >> 1) & 1))) << 2) + (col & 3);
}

// AdamW on a wave's 32 x 64 piece of R (accumulator blocks a0, a1) at row i0, column c0,
// through the wave's exchange region lw: lane l ends with rows (l >> 2) + 16 q of a block
// and its columns 8 (l & 3) .. + 7.
__device__ __forceinline__ void gx_epilogue(const GxDesc& d, const GaArgs& a, const f32x16& a0, const f32x16& a1,
                                            int64_t i0, int c0, float* lw, int lane) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const f32x16& acc = b ? a1 : a0;
#pragma unroll
        for (int v = 0; v < 16; ++v) lw[gx_ex(acc_row(v, lane), acc_col(lane))] = acc[v];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int r = (lane >> 2) + 16 * q, c = 8 * (lane & 3);
            const f32x4 x0 = *reinterpret_cast<const f32x4*>(lw + gx_ex(r, c));
            const f32x4 x1 = *reinterpret_cast<const f32x4*>(lw + gx_ex(r, c + 4));
            const float rv[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            const int64_t row = i0 + r;
            const int col = c0 + 32 * b + c;
            if (row < d.D && col < d.rp) gx_adamw8(d, a, row, col, rv);
        }
        __builtin_amdgcn_wave_barrier();  // this block's gathers before the next block's spill
    }
}

template <int IB>
__device__ __forceinline__ void zero_acc(f32x16 (&acc)[IB][2]) {
#pragma unroll
    for (int ib = 0; ib < IB; ++ib)
#pragma unroll
        for (int jb = 0; jb < 2; ++jb)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[ib][jb][v] = 0.0f;
}

}  // namespace

// ------------------------------------------------------------------ bf16 gradient

// Any shape and alignment: the register-staged projection of galore.hip (64 rows of R x all r
// columns per block, wave w columns 64 w .. 64 w + 63), U^T decoded into LDS.
template <bool Left>
__global__ __launch_bounds__(kThreads, 3) void k_gx_project(GxTable t, GaArgs a) {
    constexpr int kRows = kGxFormRows[kGxAny];
    __shared__ __attribute__((aligned(16))) uint16_t arena[(kRows + kGaWide) * kGaPitch];
    static_assert((kRows + kGaWide) * kGaPitch * 2 >= kWaves * kGxEx * 4, "exchange space");
    uint16_t* sa = arena;
    uint16_t* sb = arena + kRows * kGaPitch;
    const int2 it = t.items[blockIdx.x];
    if (it.x < 0) return;
    const GxDesc d = t.desc[it.x];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t i0 = static_cast<int64_t>(it.y) * kRows;
    const bool active = wave * 64 < d.r;
    f32x16 acc[2][2];
    zero_acc(acc);
    typename std::conditional<Left, TransStage<kRows>, RowStage<kRows>>::type pa;
    MxRowStage pb;
    auto fetch = [&](int64_t k0) {
        if constexpr (Left) pa.load(d.g, d.d, d.D, i0, k0, d.vec);
        else pa.load(d.g, d.D, d.d, i0, k0, d.vec);
        pb.load(d, k0);
    };
    fetch(0);
    for (int64_t k0 = 0; k0 < d.d; k0 += kGaKb) {
        pa.store(sa);
        pb.store(sb);
        __syncthreads();
        if (k0 + kGaKb < d.d) fetch(k0 + kGaKb);
        if (active) {
#pragma unroll
            for (int ks = 0; ks < kGaKb; ks += 16) {
                const int kk = ks + 8 * (lane >> 5);
                bfv8 fa[2], fb[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    fa[b] = ld_frag(sa + (b * 32 + (lane & 31)) * kGaPitch + kk);
                    fb[b] = ld_frag(sb + (wave * 64 + b * 32 + (lane & 31)) * kGaPitch + kk);
                }
#pragma unroll
                for (int ib = 0; ib < 2; ++ib)
#pragma unroll
                    for (int jb = 0; jb < 2; ++jb) acc[ib][jb] = mfma32(fa[ib], fb[jb], acc[ib][jb]);
            }
        }
        __syncthreads();
    }
    if (!active) return;
    float* lw = reinterpret_cast<float*>(arena) + wave * kGxEx;
#pragma unroll
    for (int ib = 0; ib < 2; ++ib) gx_epilogue(d, a, acc[ib][0], acc[ib][1], i0 + ib * 32, wave * 64, lw, lane);
}

// d a multiple of 128, 16-byte rows of G and whole words of scales. 8 waves on 64 IB rows of R
// x 256 columns: wave w at rows 32 IB (w / 4), columns 64 (w % 4). One contraction step is
// 128 long: G's tile (256-byte pieces of its rows; left: 128 rows of 128 IB bytes), the codes of
// U^T (64 bytes of each of its 256 rows) and their scales (a word each) go by
// global_load_lds into one of three LDS stages, two steps ahead; the codes are decoded
// as the fragments are read. Lane half h takes values 64 h .. 64 h + 63 of a step: two whole
// MX blocks, so a lane's scale changes once per step.
constexpr int kGdStep = 128;
constexpr int kGdWaves = 8;

template <bool Left, int IB>
__global__ __launch_bounds__(kGdWaves * 64) void k_gx_project_direct(GxTable t, GaArgs a) {
    constexpr int kRows = 64 * IB;
    constexpr int kAg = kRows * kGdStep * 2, kBc = kGaWide * kGdStep / 2;  // bytes of a stage's G and codes
    constexpr int kStage = kAg + kBc + kGaWide * 4;
    constexpr int kA = kAg / 1024 / kGdWaves, kB = kBc / 1024 / kGdWaves, kDma = kA + kB + 1;
    __shared__ __attribute__((aligned(16))) uint8_t stages[3 * kStage];
    static_assert(3 * kStage >= kGdWaves * kGxEx * 4, "exchange space");
    const int2 it = t.items[blockIdx.x];
    if (it.x < 0) return;
    const GxDesc d = t.desc[it.x];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;
    const int64_t i0 = static_cast<int64_t>(it.y) * kRows;
    const int cw = (wave & 3) * 64;   // the wave's first column of R
    const int rw = (wave >> 2) * 32 * IB;
    f32x16 acc[IB][2];
    zero_acc(acc);

    // Transfers. Right: transfer j holds rows 4 j + (l >> 4) of G's tile, 16-byte chunk
    // (l & 15) ^ (row & 15). Left: rows of 128 IB bytes (64 IB columns of G), chunk
    // c ^ lsw(row & 3), so that the transposed reads of four rows (64 bytes each) meet 64 banks.
    auto lsw = [](int e) { return IB == 2 ? e << 2 : (e >> 1) << 2; };
    const uint8_t* const g = reinterpret_cast<const uint8_t*>(d.g);
    constexpr int kChunks = 8 * IB;                 // left: chunks per row
    int64_t ga[kA];
#pragma unroll
    for (int i = 0; i < kA; ++i) {
        const int j = wave + i * kGdWaves;
        if constexpr (Left) {
            const int p = j * 64 + lane, kr = p / kChunks, c = (p % kChunks) ^ lsw(kr & 3);
            const int64_t col = min<int64_t>(i0 + c * 8, d.D - 8);
            ga[i] = (static_cast<int64_t>(kr) * d.D + col) * 2;
        } else {
            const int r = 4 * j + (lane >> 4), c = (lane & 15) ^ (r & 15);
            ga[i] = (min<int64_t>(i0 + r, d.D - 1) * d.d + c * 8) * 2;
        }
    }
    const int64_t gstep = static_cast<int64_t>(kGdStep) * 2 * (Left ? d.D : 1);
    // codes: transfer j holds rows 16 j + (l >> 2) of U^T, block (l & 3) ^ ((row >> 2) & 3)
    uint32_t ub[kB];
#pragma unroll
    for (int i = 0; i < kB; ++i) {
        const int r = 16 * (wave + i * kGdWaves) + (lane >> 2);
        ub[i] = (static_cast<uint32_t>(min(r, d.r - 1)) * d.nb + ((lane & 3) ^ ((r >> 2) & 3))) * 16;
    }
    // scales: transfer j holds rows 64 j + l; waves 4 .. 7 repeat those of 0 .. 3
    const uint32_t us = static_cast<uint32_t>(min(64 * (wave & 3) + lane, d.r - 1)) * d.nb;
    const int steps = d.d / kGdStep;
    auto stage = [&](int k, uint8_t* s) {
        k = min(k, steps - 1);  // past the end: the last step again, for equal counts
        const uint8_t* gk = g + k * gstep;
#pragma unroll
        for (int i = 0; i < kA; ++i) dma16(gk + ga[i], s + (wave + i * kGdWaves) * 1024);
#pragma unroll
        for (int i = 0; i < kB; ++i) dma16(d.uc + (ub[i] + k * 64u), s + kAg + (wave + i * kGdWaves) * 1024);
        dma4(d.us + (us + k * 4u), s + kAg + kBc + (wave & 3) * 256);
    };
    const uint32_t base = lds_addr(stages);
    auto multiply = [&](uint32_t s) {
        // the two blocks of the lane's two columns of R, and their scales
        const int r0 = cw + (lane & 31);
        const uint32_t pb = s + kAg + r0 * 64, sw = (r0 >> 2) & 3;  // rows 32 on share sw
        u32x4 c[4];
        lds_read4(pb + (((2 * h) ^ sw) << 4), pb + (((2 * h + 1) ^ sw) << 4), pb + 2048 + (((2 * h) ^ sw) << 4),
                  pb + 2048 + (((2 * h + 1) ^ sw) << 4), c);
        uint32_t e[4];
        lds_read_words(s + kAg + kBc + r0 * 4, s + kAg + kBc + r0 * 4 + 128, s + kAg + kBc + r0 * 4,
                       s + kAg + kBc + r0 * 4 + 128, e);
        float sc[2][2];  // [column][block]
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
            const uint32_t w = h ? e[jb] >> 16 : e[jb];
            sc[jb][0] = mx4_scale(w & 255u);
            sc[jb][1] = mx4_scale((w >> 8) & 255u);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // two 8-value sub-steps at a time
            bfv8 fa[2][IB];
#pragma unroll
            for (int ib = 0; ib < IB; ++ib) {
                if constexpr (Left) {
                    const int gq = lane >> 4, eq = (lane >> 2) & 3;
                    const int col = rw + ib * 32 + 16 * (gq & 1) + 4 * (lane & 3);
                    const int kr = 64 * h + 16 * q + eq;
                    const uint32_t p = s + kr * (kChunks * 16) + (((col >> 3) ^ lsw(eq)) << 4) + (col & 7) * 2;
                    constexpr uint32_t kFour = 4 * kChunks * 16;
                    u32x2 x0, x1, x2, x3;
                    __asm__ volatile(
                        "ds_read_b64_tr_b16 %0, %4\n\t"
                        "ds_read_b64_tr_b16 %1, %5\n\t"
                        "ds_read_b64_tr_b16 %2, %6\n\t"
                        "ds_read_b64_tr_b16 %3, %7\n\t"
                        "s_waitcnt lgkmcnt(0)"
                        : "=&v"(x0), "=&v"(x1), "=&v"(x2), "=&v"(x3)
                        : "v"(p), "v"(p + kFour), "v"(p + 2 * kFour), "v"(p + 3 * kFour));
                    fa[0][ib] = __builtin_bit_cast(bfv8, u32x4{x0.x, x0.y, x1.x, x1.y});
                    fa[1][ib] = __builtin_bit_cast(bfv8, u32x4{x2.x, x2.y, x3.x, x3.y});
                }
            }
            if constexpr (!Left) {
                const int r = rw + (lane & 31);
                const uint32_t p0 = s + r * 256 + (((8 * h + 2 * q) ^ (r & 15)) << 4);
                const uint32_t p1 = s + r * 256 + (((8 * h + 2 * q + 1) ^ (r & 15)) << 4);
                u32x4 x[4];
                if constexpr (IB == 2) {
                    lds_read4(p0, p0 + 8192, p1, p1 + 8192, x);
                    fa[0][0] = __builtin_bit_cast(bfv8, x[0]);
                    fa[0][1] = __builtin_bit_cast(bfv8, x[1]);
                    fa[1][0] = __builtin_bit_cast(bfv8, x[2]);
                    fa[1][1] = __builtin_bit_cast(bfv8, x[3]);
                } else {
                    lds_read2(p0, p1, x);
                    fa[0][0] = __builtin_bit_cast(bfv8, x[0]);
                    fa[1][0] = __builtin_bit_cast(bfv8, x[1]);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int sub = 2 * q + u;  // 8 values: dword sub & 3 of block sub >> 2
#pragma unroll
                for (int jb = 0; jb < 2; ++jb) {
                    const bfv8 fb = __builtin_bit_cast(bfv8, mx4_to_bf16(c[2 * jb + (sub >> 2)][sub & 3], sc[jb][sub >> 2]));
#pragma unroll
                    for (int ib = 0; ib < IB; ++ib) acc[ib][jb] = mfma32(fa[u][ib], fb, acc[ib][jb]);
                }
            }
        }
    };
    const bool active = cw < d.r;
    stage(0, stages);
    stage(1, stages + kStage);
    int cur = 0;
    for (int k = 0; k < steps; ++k) {
        wait_and_sync<kDma>();
        stage(k + 2, stages + (cur == 0 ? 2 : cur - 1) * kStage);
        if (active) multiply(base + cur * kStage);
        cur = cur == 2 ? 0 : cur + 1;
    }
    wait_and_sync<0>();
    if (!active) return;
    float* lw = reinterpret_cast<float*>(stages) + wave * kGxEx;
#pragma unroll
    for (int ib = 0; ib < IB; ++ib) gx_epilogue(d, a, acc[ib][0], acc[ib][1], i0 + rw + ib * 32, cw, lw, lane);
}

void launch_gx_project(const GxTable& t, int64_t n, const GaArgs& a, bool left, int form, hipStream_t s) {
    if (n <= 0) return;
    const dim3 grid(static_cast<uint32_t>(n)), wide(kGdWaves * 64);
    if (form == kGxAny) {
        if (left) hipLaunchKernelGGL(k_gx_project<true>, grid, dim3(kThreads), 0, s, t, a);
        else hipLaunchKernelGGL(k_gx_project<false>, grid, dim3(kThreads), 0, s, t, a);
    } else if (form == kGxDirect) {
        if (left) hipLaunchKernelGGL((k_gx_project_direct<true, 1>), grid, wide, 0, s, t, a);
        else hipLaunchKernelGGL((k_gx_project_direct<false, 1>), grid, wide, 0, s, t, a);
    } else {
        if (left) hipLaunchKernelGGL((k_gx_project_direct<true, 2>), grid, wide, 0, s, t, a);
        else hipLaunchKernelGGL((k_gx_project_direct<false, 2>), grid, wide, 0, s, t, a);
    }
}

// ------------------------------------------------------------------ MX4 gradient

// The product of mx4_tile.h, one column tile (r <= 256), with AdamW on R.
template <int IB, int WN, int NW, bool Any>
__global__ __launch_bounds__(NW * 64) void k_gx_project_mx4(GxTable t, GaArgs a) {
    using T = MxTile<IB, WN, NW>;
    constexpr int kEx = NW * kGxEx * 4;
    __shared__ __attribute__((aligned(16))) uint8_t stages[Any ? kEx : 3 * T::kStage];
    static_assert(3 * T::kStage >= kEx, "exchange space");
    const int2 it = t.items[blockIdx.x];
    if (it.x < 0) return;
    const GxDesc d = t.desc[it.x];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t i0 = static_cast<int64_t>(it.y) * T::kRowsA;
    const MxOperand oa{reinterpret_cast<const uint8_t*>(d.g), d.gs, d.D, d.nb}, ob{d.uc, d.us, d.r, d.nb};
    float* lw = reinterpret_cast<float*>(stages) + wave * kGxEx;
    for (int c0 = 0; c0 < d.r; c0 += T::kRowsB) {
        f32x16 acc[IB][2];
        zero_acc(acc);
        if constexpr (Any) mx4_accumulate_any(oa, ob, i0, c0, acc);
        else mx4_accumulate<IB, WN, NW>(oa, ob, i0, c0, stages, acc);
        const int64_t row = i0 + (wave / WN) * 32 * IB;
        const int col = c0 + (wave % WN) * 64;
        if (col < d.r)
#pragma unroll
            for (int ib = 0; ib < IB; ++ib) gx_epilogue(d, a, acc[ib][0], acc[ib][1], row + ib * 32, col, lw, lane);
        if (c0 + T::kRowsB < d.r) __syncthreads();  // the exchange regions are read before the stages are filled
    }
}

void launch_gx_project_mx4(const GxTable& t, int64_t n, const GaArgs& a, int form, hipStream_t s) {
    if (n <= 0) return;
    const dim3 grid(static_cast<uint32_t>(n));
    switch (form) {
        case kMxAny: hipLaunchKernelGGL((k_gx_project_mx4<1, 2, 4, true>), grid, dim3(256), 0, s, t, a); break;
        case kMxNarrow: hipLaunchKernelGGL((k_gx_project_mx4<1, 2, 4, false>), grid, dim3(256), 0, s, t, a); break;
        case kMxWide: hipLaunchKernelGGL((k_gx_project_mx4<1, 4, 8, false>), grid, dim3(512), 0, s, t, a); break;
        default: hipLaunchKernelGGL((k_gx_project_mx4<2, 4, 8, false>), grid, dim3(512), 0, s, t, a); break;
    }
}

}  // namespace meo
