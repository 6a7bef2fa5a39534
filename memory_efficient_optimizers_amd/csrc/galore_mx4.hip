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

namespace meo {

// AdamW on a wave's 32 x 64 piece of R (accumulator blocks a0, a1) at row i0, column c0,
// through the wave's exchange region lw.
__device__ __forceinline__ void gx_epilogue(const GxDesc& d, const GaArgs& a, const f32x16& a0, const f32x16& a1,
                                            int64_t i0, int c0, float* lw, int lane) {
    ep_spill(a0, a1, lw, lane);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int64_t row = i0 + (lane >> 3) + 8 * q;
        const int col = c0 + (lane & 7) * 8;
        if (row >= d.D || col >= d.r) continue;
        float rv[8];
        ep_gather(lw, lane, q, rv);
        galore_adamw8(d, a, row, col, rv);
    }
}

// bf16 gradient, any list: the register-staged projection of galore.hip (tile: kGxRows
// rows of R x all r columns, wave w columns 64 w .. 64 w + 63), U^T decoded into LDS.
template <bool Left>
__global__ __launch_bounds__(kThreads, 3) void k_gx_project(GxTable t, GaArgs a) {
    __shared__ __attribute__((aligned(16))) uint16_t arena[(kGxRows + kGaWide) * kGaPitch];
    static_assert((kGxRows + kGaWide) * kGaPitch * 2 >= kWaves * kEpWave * 4, "exchange space");
    uint16_t* sa = arena;
    uint16_t* sb = arena + kGxRows * kGaPitch;
    const int2 it = t.items[blockIdx.x];
    if (it.x < 0) return;
    const GxDesc d = t.desc[it.x];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t i0 = static_cast<int64_t>(it.y) * kGxRows;
    const bool active = wave * 64 < d.r;
    f32x16 acc[2][2];
#pragma unroll
    for (int ib = 0; ib < 2; ++ib)
#pragma unroll
        for (int jb = 0; jb < 2; ++jb)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[ib][jb][v] = 0.0f;
    typename std::conditional<Left, TransStage<kGxRows>, RowStage<kGxRows>>::type pa;
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
    float* lw = reinterpret_cast<float*>(arena) + wave * kEpWave;
#pragma unroll
    for (int ib = 0; ib < 2; ++ib) gx_epilogue(d, a, acc[ib][0], acc[ib][1], i0 + ib * 32, wave * 64, lw, lane);
}

// MX4 gradient, any list: the same tile, every operand fragment read as it lies (a lane
// holds one MX block of a row).
__global__ __launch_bounds__(kThreads) void k_gx_project_mx4(GxTable t, GaArgs a) {
    __shared__ __attribute__((aligned(16))) float ex[kWaves * kEpWave];
    const int2 it = t.items[blockIdx.x];
    if (it.x < 0) return;
    const GxDesc d = t.desc[it.x];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t i0 = static_cast<int64_t>(it.y) * kGxRows;
    if (wave * 64 >= d.r) return;
    f32x16 acc[2][2];
#pragma unroll
    for (int ib = 0; ib < 2; ++ib)
#pragma unroll
        for (int jb = 0; jb < 2; ++jb)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[ib][jb][v] = 0.0f;
    const uint8_t* gc = reinterpret_cast<const uint8_t*>(d.g);
    for (int64_t k = 0; k < d.nb; k += 2) {
        const int64_t kb = k + (lane >> 5);
        u32x4 ca[2], cb[2];
        uint32_t ea[2], eb[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int64_t row = i0 + b * 32 + (lane & 31);
            ca[b] = u32x4{0u, 0u, 0u, 0u};
            ea[b] = 127;
            if (row < d.D && kb < d.nb) {
                ca[b] = *gld<u32x4>(gc + (row * d.nb + kb) * 16);
                ea[b] = *gld<uint8_t>(d.gs + row * d.nb + kb);
            }
            ld_mx_block(d, wave * 64 + b * 32 + (lane & 31), kb, cb[b], eb[b]);
        }
#pragma unroll
        for (int ib = 0; ib < 2; ++ib)
#pragma unroll
            for (int jb = 0; jb < 2; ++jb) acc[ib][jb] = mfma_mx4(ca[ib], cb[jb], acc[ib][jb], ea[ib], eb[jb]);
    }
    float* lw = ex + wave * kEpWave;
#pragma unroll
    for (int ib = 0; ib < 2; ++ib) gx_epilogue(d, a, acc[ib][0], acc[ib][1], i0 + ib * 32, wave * 64, lw, lane);
}

void launch_gx_project(const GxTable& t, int64_t n, const GaArgs& a, bool left, hipStream_t s) {
    if (n <= 0) return;
    const dim3 grid(static_cast<uint32_t>(n)), block(kThreads);
    if (left) hipLaunchKernelGGL(k_gx_project<true>, grid, block, 0, s, t, a);
    else hipLaunchKernelGGL(k_gx_project<false>, grid, block, 0, s, t, a);
}

void launch_gx_project_mx4(const GxTable& t, int64_t n, const GaArgs& a, hipStream_t s) {
    if (n <= 0) return;
    hipLaunchKernelGGL(k_gx_project_mx4, dim3(static_cast<uint32_t>(n)), dim3(kThreads), 0, s, t, a);
}

}  // namespace meo
