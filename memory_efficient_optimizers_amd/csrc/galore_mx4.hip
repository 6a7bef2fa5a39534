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

// AdamW on 8 columns of a row of R: the moments (m, v: as loaded, the `valid` first columns
// in range) are stored back, N goes to its two planes up to column rp, zero past r. (bf16
// parameters need the low plane too: with N rounded to bf16 alone, 3% of the entries of
// a 256 x 200 parameter came out one bf16 step away.)
__device__ __forceinline__ void gx_adamw8(const GxDesc& d, const GaArgs& a, int64_t row, int col, int valid, float* m,
                                          float* v, const float* rv) {
    float nh[8], nl[8];
    const int64_t idx = row * d.r + col;
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

// A wave's piece of R at row i0, column c0: two 32 x 32 blocks, the second 32 columns on or
// (Tall) 32 rows on. Lane l holds, in block b, rows (l >> 2) + 16 q and columns 8 (l & 3) .. + 7.
// The moments of all of them:
template <bool Tall>
struct GxMoments {
    float m[2][2][8], v[2][2][8];
    __device__ __forceinline__ void load(const GxDesc& d, int64_t i0, int c0, int lane) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int64_t row = i0 + (Tall ? 32 * b : 0) + (lane >> 2) + 16 * q;
                const int col = c0 + (Tall ? 0 : 32 * b) + 8 * (lane & 3);
                const int valid = row < d.D ? min(max(d.r - col, 0), 8) : 0;
                load_f8(d.em + row * d.r + col, valid, d.rvec, m[b][q]);
                load_f8(d.ev + row * d.r + col, valid, d.rvec, v[b][q]);
            }
    }
};

// AdamW on that piece (accumulator blocks a0, a1), through the wave's exchange region lw.
template <bool Tall>
__device__ __forceinline__ void gx_epilogue(const GxDesc& d, const GaArgs& a, const f32x16& a0, const f32x16& a1,
                                            GxMoments<Tall>& mv, int64_t i0, int c0, float* lw, int lane) {
    const int c = 8 * (lane & 3);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const f32x16& acc = b ? a1 : a0;
#pragma unroll
        for (int w = 0; w < 16; ++w) lw[gx_ex(acc_row(w, lane), acc_col(lane))] = acc[w];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int r = (lane >> 2) + 16 * q;
            const f32x4 x0 = *reinterpret_cast<const f32x4*>(lw + gx_ex(r, c));
            const f32x4 x1 = *reinterpret_cast<const f32x4*>(lw + gx_ex(r, c + 4));
            const float rv[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            const int64_t row = i0 + (Tall ? 32 * b : 0) + r;
            const int col = c0 + (Tall ? 0 : 32 * b) + c;
            if (row < d.D && col < d.rp)
                gx_adamw8(d, a, row, col, min(max(d.r - col, 0), 8), mv.m[b][q], mv.v[b][q], rv);
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
constexpr int kGxArena = (kGxFormRows[kGxAny] + kGaWide) * kGaPitch;
template <bool Left>
__device__ __forceinline__ void gx_any_tile(const GxDesc& d, int64_t i0, const GaArgs& a, uint16_t* arena) {
    constexpr int kRows = kGxFormRows[kGxAny];
    static_assert(kGxArena * 2 >= kWaves * kGxEx * 4, "exchange space");
    uint16_t* sa = arena;
    uint16_t* sb = arena + kRows * kGaPitch;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
    for (int ib = 0; ib < 2; ++ib) {
        GxMoments<false> mv;
        mv.load(d, i0 + ib * 32, wave * 64, lane);
        gx_epilogue(d, a, acc[ib][0], acc[ib][1], mv, i0 + ib * 32, wave * 64, lw, lane);
    }
}

__global__ __launch_bounds__(kThreads, 3) void k_gx_project(GxTable t, GaArgs a, int nright) {
    __shared__ __attribute__((aligned(16))) uint16_t arena[kGxArena];
    const int2 it = t.items[blockIdx.x];
    const GxDesc d = t.desc[it.x];
    const int64_t i0 = static_cast<int64_t>(it.y) * kGxFormRows[kGxAny];
    if (it.x < nright) gx_any_tile<false>(d, i0, a, arena);
    else gx_any_tile<true>(d, i0, a, arena);
}

// d a multiple of 128, 16-byte rows of G and whole words of scales. 8 waves on 64 rows of R
// x 256 columns, all rows and columns 32 w .. 32 w + 31 each: a wave's decoded codes then serve
// two products, and no two waves decode the same. One contraction step is 128 long. Everything goes by global_load_lds, as in mx4_accumulate: waves 0 .. 3 fetch G's
// tile (256-byte pieces of its rows; left: 128 rows of 128 bytes) into one of five stages,
// four steps ahead, which keeps the 64 KB in flight that HBM takes per CU; waves 4 .. 7 the
// codes of U^T of two steps (a whole 128-byte line of each of its 256 rows) and the
// scales of four (a word per row and step) into one of two buffers each. (All waves
// fetching all, two steps ahead, each step's codes and scales on their own: 84 us for
// the four 4096 x 4096 matrices of a layer.) The codes are decoded as the fragments are read.
// Lane half h takes values 64 h .. 64 h + 63 of a step: two whole MX blocks, so a lane's
// scale changes once per step.
constexpr int kGdRows = kGxFormRows[kGxDirect];
constexpr int kGdStep = 128;
constexpr int kGdWaves = 8;
constexpr int kGdDepth = 5;
constexpr int kGdG = kGdRows * kGdStep * 2;      // bytes of G per stage
constexpr int kGdCodes = kGaWide * kGdStep;      // bytes of codes of two steps
constexpr int kGdScales = kGaWide * 4 * 4;       // bytes of scales of four: [word][row]
constexpr int kGdLds = kGdDepth * kGdG + 2 * kGdCodes + 2 * kGdScales;

template <bool Left>
__device__ __forceinline__ void gx_direct_tile(const GxDesc& d, int64_t i0, const GaArgs& a, uint8_t* lds) {
    constexpr int kA = kGdG / 1024 / 4, kB = kGdCodes / 1024 / 4;  // 1 KB transfers per wave of its kind
    static_assert(kGdWaves == 8 && kGdDepth * kGdG >= kGdWaves * kGxEx * 4, "waves below; exchange space");
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;
    const int cw = wave * 32;  // the wave's first column of R
    const bool fetch_g = wave < 4;
    const int fw = wave & 3;
    f32x16 acc[2];
#pragma unroll
    for (int ib = 0; ib < 2; ++ib)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[ib][v] = 0.0f;

    // G. Right: transfer j holds rows 4 j + (l >> 4) of the tile, 16-byte chunk
    // (l & 15) ^ (row & 15). Left: rows 8 j + (l >> 3) of 128 bytes (64 columns of G), chunk
    // c ^ lsw(row & 3), so that the transposed reads of four rows (64 bytes each) meet 64 banks.
    auto lsw = [](int e) { return (e >> 1) << 2; };
    const uint8_t* const g = reinterpret_cast<const uint8_t*>(d.g);
    int64_t ga[kA];
#pragma unroll
    for (int i = 0; i < kA; ++i) {
        const int j = fw + i * 4;
        if constexpr (Left) {
            const int kr = 8 * j + (lane >> 3), c = (lane & 7) ^ lsw(kr & 3);
            ga[i] = (static_cast<int64_t>(kr) * d.D + min<int64_t>(i0 + c * 8, d.D - 8)) * 2;
        } else {
            const int r = 4 * j + (lane >> 4), c = (lane & 15) ^ (r & 15);
            ga[i] = (min<int64_t>(i0 + r, d.D - 1) * d.d + c * 8) * 2;
        }
    }
    const int64_t gstep = static_cast<int64_t>(kGdStep) * 2 * (Left ? d.D : 1);
    const int steps = d.d / kGdStep;
    auto stage = [&](int k, uint8_t* s) {
        const uint8_t* gk = g + min(k, steps - 1) * gstep;  // past the end: the last again, for equal counts
#pragma unroll
        for (int i = 0; i < kA; ++i) dma16(gk + ga[i], s + (fw + i * 4) * 1024);
    };
    // Codes: transfer j holds rows 8 j + (l >> 3) of U^T, block (l & 7) ^ mx_swz(row).
    uint32_t ub[kB];
    const int cblk = (lane & 7) ^ mx_swz(lane >> 3) ^ (fw & 1);
#pragma unroll
    for (int i = 0; i < kB; ++i)
        ub[i] = static_cast<uint32_t>(min(8 * (fw + i * 4) + (lane >> 3), d.r - 1)) * d.nb;
    uint8_t* const cbuf = lds + kGdDepth * kGdG;
    auto codes = [&](int pair) {
        const uint32_t kc = static_cast<uint32_t>(min(8 * pair + cblk, d.nb - 1));
#pragma unroll
        for (int i = 0; i < kB; ++i) dma16(d.uc + (ub[i] + kc) * 16, cbuf + (pair & 1) * kGdCodes + (fw + i * 4) * 1024);
    };
    // Scales: wave 4 + f fetches the words of rows 64 f + l.
    const uint32_t us = static_cast<uint32_t>(min(64 * fw + lane, d.r - 1)) * d.nb;
    uint8_t* const sbuf = cbuf + 2 * kGdCodes;
    auto scales = [&](int quad) {
#pragma unroll
        for (int w = 0; w < 4; ++w)
            dma4(d.us + (us + static_cast<uint32_t>(min(16 * quad + 4 * w, d.nb - 4))),
                 sbuf + (quad & 1) * kGdScales + w * (kGaWide * 4) + fw * 256);
    };
    const uint32_t base = lds_addr(lds);
    auto multiply = [&](int k, int cur) {
        const uint32_t s = base + cur * kGdG;
        // the two blocks of the lane's column of R, and their scales
        const int r0 = cw + (lane & 31), sw = mx_swz(lane & 31), b0 = 4 * (k & 1) + 2 * h;
        const uint32_t pb = base + kGdDepth * kGdG + ((k >> 1) & 1) * kGdCodes + r0 * 128;
        const uint32_t pe = base + kGdDepth * kGdG + 2 * kGdCodes + ((k >> 2) & 1) * kGdScales + (k & 3) * (kGaWide * 4) + r0 * 4;
        const uint32_t q[2] = {pb + ((b0 ^ sw) << 4), pb + (((b0 + 1) ^ sw) << 4)};
        u32x4 x[2][8], c[2];  // G's fragments of two 32-row halves; codes of two blocks
        uint32_t e;
        if constexpr (Left) {
            const int gq = lane >> 4, eq = (lane >> 2) & 3;
            const int col = 16 * (gq & 1) + 4 * (lane & 3);
            const uint32_t p = s + (64 * h + eq) * 128 + (((col >> 3) ^ lsw(eq)) << 4) + (col & 7) * 2;
            lds_read_codes(q, pe, c, e);
            lds_read_tr(p, x[0]);
            lds_read_tr(p ^ 64, x[1]);  // 32 columns on: the other half of the (aligned) 128-byte row
        } else {
            const int r = lane & 31;
            uint32_t p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = s + r * 256 + (((8 * h + i) ^ (r & 15)) << 4);
            lds_read_row(p, q, pe, x, c, e);
        }
        if (h) e >>= 16;
        const float sc[2] = {mx4_scale(e & 255u), mx4_scale((e >> 8) & 255u)};
#pragma unroll
        for (int u = 0; u < 8; ++u) {  // 8 values: dword u & 3 of block u >> 2
            const bfv8 fb = __builtin_bit_cast(bfv8, mx4_to_bf16(c[u >> 2][u & 3], sc[u >> 2]));
#pragma unroll
            for (int ib = 0; ib < 2; ++ib) acc[ib] = mfma32(__builtin_bit_cast(bfv8, x[ib][u]), fb, acc[ib]);
        }
    };
    // Before step k's barrier a wave that fetches G waits until only steps k + 1 .. k + 3 are
    // outstanding. One that fetches U^T issued the codes of a pair of steps in the even step
    // before it and the scales of four steps two steps before them: before an even step it
    // waits for all, before an odd one for nothing that step k - 1 issued. What a step fills
    // was last read before its barrier.
    // The moments of the wave's piece of R are loaded before everything else.
    const bool active = cw < d.r;
    GxMoments<true> mv;
    if (active) mv.load(d, i0, cw, lane);
    if (fetch_g) {
#pragma unroll
        for (int k = 0; k < kGdDepth - 1; ++k) stage(k, lds + k * kGdG);
    } else {
        scales(0);
        codes(0);
    }
    int cur = 0;
    for (int k = 0; k < steps; ++k) {
        if (fetch_g) wait_and_sync<3 * kA>();
        else if (!(k & 1)) wait_and_sync<0>();
        else if ((k & 3) == 3) wait_and_sync<kB + 4>();
        else wait_and_sync<kB>();
        if (fetch_g) {
            stage(k + kGdDepth - 1, lds + (cur == 0 ? kGdDepth - 1 : cur - 1) * kGdG);
        } else if (!(k & 1)) {
            if ((k & 3) == 2) scales((k >> 2) + 1);
            codes((k >> 1) + 1);
        }
        if (active) multiply(k, cur);
        cur = cur == kGdDepth - 1 ? 0 : cur + 1;
    }
    wait_and_sync<0>();
    if (!active) return;
    float* lw = reinterpret_cast<float*>(lds) + wave * kGxEx;
    gx_epilogue(d, a, acc[0], acc[1], mv, i0, cw, lw, lane);
}

__global__ __launch_bounds__(kGdWaves * 64) void k_gx_project_direct(GxTable t, GaArgs a, int nright) {
    __shared__ __attribute__((aligned(128))) uint8_t lds[kGdLds];
    const int2 it = t.items[blockIdx.x];
    const GxDesc d = t.desc[it.x];
    const int64_t i0 = static_cast<int64_t>(it.y) * kGdRows;
    if (it.x < nright) gx_direct_tile<false>(d, i0, a, lds);
    else gx_direct_tile<true>(d, i0, a, lds);
}

void launch_gx_project(const GxTable& t, int64_t n, int nright, const GaArgs& a, int form, hipStream_t s) {
    if (n <= 0) return;
    const dim3 grid(static_cast<uint32_t>(n)), wide(kGdWaves * 64);
    if (form == kGxAny) hipLaunchKernelGGL(k_gx_project, grid, dim3(kThreads), 0, s, t, a, nright);
    else hipLaunchKernelGGL(k_gx_project_direct, grid, wide, 0, s, t, a, nright);
}

// ------------------------------------------------------------------ MX4 gradient

// The product of mx4_tile.h, one column tile (r <= 256), with AdamW on R.
template <int IB, int WN, int NW, bool Any>
__global__ __launch_bounds__(NW * 64) void k_gx_project_mx4(GxTable t, GaArgs a) {
    using T = MxTile<IB, WN, NW>;
    constexpr int kEx = NW * kGxEx * 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[Any ? kEx : T::kLds];
    static_assert(T::kLds >= kEx, "exchange space");
    const int2 it = t.items[blockIdx.x];
    const GxDesc d = t.desc[it.x];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t i0 = static_cast<int64_t>(it.y) * T::kRowsA;
    const MxOperand oa{reinterpret_cast<const uint8_t*>(d.g), d.gs, d.D, d.nb}, ob{d.uc, d.us, d.r, d.nb};
    float* lw = reinterpret_cast<float*>(lds) + wave * kGxEx;
    for (int c0 = 0; c0 < d.r; c0 += T::kRowsB) {
        f32x16 acc[IB][2];
        zero_acc(acc);
        if constexpr (Any) mx4_accumulate_any(oa, ob, i0, c0, acc);
        else mx4_accumulate<IB, WN, NW>(oa, ob, i0, c0, lds, acc);
        const int64_t row = i0 + (wave / WN) * 32 * IB;
        const int col = c0 + (wave % WN) * 64;
        if (col < d.r)
#pragma unroll
            for (int ib = 0; ib < IB; ++ib) {
                GxMoments<false> mv;
                mv.load(d, row + ib * 32, col, lane);
                gx_epilogue(d, a, acc[ib][0], acc[ib][1], mv, row + ib * 32, col, lw, lane);
            }
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
