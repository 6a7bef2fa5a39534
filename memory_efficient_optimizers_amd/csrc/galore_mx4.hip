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
#include "galore_mx4.h"
#include "mx4_tile.h"

namespace meo {

namespace {

// 8 codes times their scale as bf16 (exact: a code has two significant bits).
__device__ __forceinline__ u32x4 mx4_to_bf16(uint32_t q, float scale) {
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3))};
}

// One block of the MX4 projector: row `row` of U^T, block kb; zero outside it.
__device__ __forceinline__ void ld_mx_block(const GxDesc& d, int64_t row, int64_t kb, u32x4& c, uint32_t& e) {
    c = u32x4{0u, 0u, 0u, 0u};
    e = 127;
    if (row >= d.r || kb >= d.nb) return;
    c = *gld<u32x4>(d.uc + (row * d.nb + kb) * 16);
    e = *gld<uint8_t>(d.us + row * d.nb + kb);
}

// AdamW on 8 columns of a row of R: the moments (m, v: as loaded, the `valid` first columns
// in range) are stored back, N goes to its two planes up to column rp, zero past r. (bf16
// parameters need the low plane too: with N rounded to bf16 alone, 3% of the entries of
// a 256 x 200 parameter came out one bf16 step away.)
__device__ __forceinline__ void gx_adamw8(const GxDesc& d, const GaArgs& a, int64_t row, int col, int valid, float* m,
                                          float* v, const float* rv) {
    float n[8], nh[8], nl[8];
    const int64_t idx = row * d.r + col;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        m[e] = fmaf(a.beta1, m[e], a.omb1 * rv[e]);
        v[e] = fmaf(a.beta2, v[e], a.omb2 * (rv[e] * rv[e]));
    }
    // N is kept to 2^-17 (its planes), so the instructions' own root and reciprocal, off by one unit
    // of 2^-23 each, do: 19 instead of 23 us for a 4096 x 4096 MX4 gradient at rank 128. They take
    // subnormal numbers for zero, which beside a usual eps is out of sight; with a smaller one
    // the full root and quotient are taken.
    if (a.eps >= 0x1p-40f) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            n[e] = (m[e] * a.inv_bc1) * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(v[e] * a.inv_bc2) + a.eps);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = (m[e] * a.inv_bc1) / (sqrtf(v[e] * a.inv_bc2) + a.eps);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (e >= valid) n[e] = 0.0f;
        nh[e] = round_bf16(n[e]);
        nl[e] = n[e] - nh[e];
    }
    store_any8(d.em, idx, valid, false, m);
    store_any8(d.ev, idx, valid, false, v);
    const int64_t at = row * d.rp + col;  // the planes are 256-byte aligned, rp a multiple of 32
    *gst<u32x4>(d.nh + at) = pack_bf16x8(nh);
    *gst<u32x4>(d.nl + at) = pack_bf16x8(nl);
}

constexpr int kGxEx = 32 * 32;  // floats of a wave's exchange region

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
                load_any8(d.em, row * d.r + col, valid, false, m[b][q]);
                load_any8(d.ev, row * d.r + col, valid, false, v[b][q]);
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
        for (int w = 0; w < 16; ++w) lw[ur_ex(acc_row(w, lane), acc_col(lane))] = acc[w];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int r = (lane >> 2) + 16 * q;
            const f32x4 x0 = *reinterpret_cast<const f32x4*>(lw + ur_ex(r, c));
            const f32x4 x1 = *reinterpret_cast<const f32x4*>(lw + ur_ex(r, c + 4));
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

// 8 waves on 64 rows of R x 256 columns, all rows and columns 32 w .. 32 w + 31 each: a wave's
// decoded codes then serve two products, and no two waves decode the same. One contraction
// step is 128 long. Waves 0 .. 3 fetch G's tile (256-byte pieces of its rows; left: 128 rows
// of 128 bytes) into one of five LDS stages, waves 4 .. 7 the codes of U^T of two steps (a
// whole 128-byte line of each of its 256 rows) and the scales of four (a word per row and
// step) into one of two buffers each; the codes are decoded as the fragments are read.
// kGxDirect (d a multiple of 128, 16-byte rows of G, whole words of scales): everything by
// global_load_lds, as in mx4_accumulate, G four steps ahead, which keeps the 64 KB in flight
// that HBM takes per CU. kGxAny: G through registers two steps ahead, with 16-byte loads
// at any address and zeros past its end; the scales through registers too; codes as there
// (they are always aligned). (All waves fetching all, each step's codes and scales on
// their own: 8 us more for the four 4096 x 4096 matrices of a layer.)
// Those take 73 us at rank 256, of which their bytes need 45 at the rate of a copy: about 11 go
// into the start and the first stages, 16 into the epilogue's moments and N at the end of
// the tiles, which all run at once.
// Lane half h takes values 64 h .. 64 h + 63 of a step: two whole MX blocks, so a lane's
// scale changes once per step.
constexpr int kGdRows = kGxFormRows[kGxDirect];
constexpr int kGdStep = kGxStep;
constexpr int kGdWaves = 8;
constexpr int kGdDepth = 5;
constexpr int kGdG = kGdRows * kGdStep * 2;      // bytes of G per stage
constexpr int kGdCodes = kGaWide * kGdStep;      // bytes of codes of two steps
constexpr int kGdScales = kGaWide * 4 * 4;       // bytes of scales of four: [word][row]
constexpr int kGdLds = kGdDepth * kGdG + 2 * kGdCodes + 2 * kGdScales;

// Values `from` on of 8 bf16 values, the `valid` first of them, zeros behind.
__device__ __forceinline__ u32x4 row_part(const u32x4& v, int from, int valid) {
    uint64_t lo = static_cast<uint64_t>(v.y) << 32 | v.x, hi = static_cast<uint64_t>(v.w) << 32 | v.z;
    if (from >= 4) {
        lo = hi;
        hi = 0;
        from -= 4;
    }
    if (from > 0) {
        lo = lo >> (16 * from) | hi << (64 - 16 * from);
        hi >>= 16 * from;
    }
    lo = valid >= 4 ? lo : valid <= 0 ? 0 : lo & (~0ull >> (64 - 16 * valid));
    hi = valid >= 8 ? hi : valid <= 4 ? 0 : hi & (~0ull >> (128 - 16 * valid));
    return u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
}

// The contraction's parts (GxDesc::ks) from `part` on, kitem of them. kWhole: it has one. kFold: all
// of them are here, and their sums are added up as k_gx_join does. kStore: each one's sum is stored
// for k_gx_join. (A form each: moments and sums of parts are in registers at once in kFold's alone.
// In kStore an item's sums are not added up first: Any then spills.)
enum GxParts { kWhole, kFold, kStore };
template <bool Left, bool Any, GxParts Parts>
__device__ __forceinline__ void gx_tile(const GxDesc& d, int64_t i0, int part, const GaArgs& a, uint8_t* lds) {
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
    f32x16 sum[2] = {acc[0], acc[1]};  // kFold

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
    const int steps = (d.d + kGdStep - 1) / kGdStep;
    const int k0 = part * d.kper, k1 = min(k0 + d.kitem * d.kper, steps);  // k0 a multiple of 4
    auto stage = [&](int k, uint8_t* s) {
        const uint8_t* gk = g + min(k, steps - 1) * gstep;  // past the end: the last again, for equal counts
#pragma unroll
        for (int i = 0; i < kA; ++i) dma16(gk + ga[i], s + (fw + i * 4) * 1024);
    };
    // The same tile through registers: the thread's four chunks of a step, and their places. Every
    // load is 16 bytes inside the tensor, without a branch (with the rest of a row read value
    // by value behind one, each load waited for the others: 59 instead of 31 us for 2048 x 5461 at rank 16): chunk
    // places past the last are moved back to it. What a step's last tile then holds wrongly
    // (values of a later row, or moved back) is put right when it is stored.
    const int64_t last = static_cast<int64_t>(d.m) * d.n - 8;
    auto place = [&](int k, int i, int64_t& at, int& valid) {
        const int j = fw + i * 4;
        if constexpr (Left) {  // (columns past D reach rows of R that are not stored)
            const int64_t kr = static_cast<int64_t>(k) * kGdStep + 8 * j + (lane >> 3);
            at = min<int64_t>(kr, d.d - 1) * d.D + min<int64_t>(i0 + (lane & 7) * 8, d.D - 1);
            valid = kr < d.d ? 8 : 0;
        } else {
            const int kc = k * kGdStep + (lane & 15) * 8;
            at = min<int64_t>(i0 + 4 * j + (lane >> 4), d.D - 1) * d.d + min(kc, d.d - 1);
            valid = min(max(d.d - kc, 0), 8);
        }
    };
    auto load_g = [&](int k, u32x4 (&v)[kA]) {
#pragma unroll
        for (int i = 0; i < kA; ++i) {
            int64_t at;
            int valid;
            place(k, i, at, valid);
            if (last >= 0) {
                v[i] = *gld<u32x4_any>(d.g + min(at, last));
            } else {  // fewer than 8 values in all
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = at + e < last + 8 ? *gld<uint16_t>(d.g + at + e) : 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] = w[2 * e] | w[2 * e + 1] << 16;
            }
        }
    };
    auto store_g = [&](int k, u32x4 (&v)[kA], uint8_t* s) {
        const bool edge = (k + 1) * kGdStep > d.d || (Left && i0 + kGdRows > d.D);
#pragma unroll
        for (int i = 0; i < kA; ++i) {
            if (edge) {
                int64_t at;
                int valid;
                place(k, i, at, valid);
                v[i] = row_part(v[i], last >= 0 ? static_cast<int>(max<int64_t>(at - last, 0)) : 0, valid);
            }
            const int j = fw + i * 4;
            const int r = Left ? 8 * j + (lane >> 3) : 4 * j + (lane >> 4);
            const int at = Left ? r * 128 + (((lane & 7) ^ lsw(r & 3)) << 4) : r * 256 + (((lane & 15) ^ (r & 15)) << 4);
            *reinterpret_cast<u32x4*>(s + at) = v[i];
        }
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
    uint32_t sw4[4];  // Any: of the quad that is stored next
    auto scales = [&](int quad) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int kb = 16 * quad + 4 * w;
            if constexpr (Any) sw4[w] = mx_scales_load(d.us + us, kb, d.nb);
            else dma4(d.us + (us + static_cast<uint32_t>(min(kb, d.nb - 4))),
                      sbuf + (quad & 1) * kGdScales + w * (kGaWide * 4) + fw * 256);
        }
    };
    auto store_scales = [&](int quad) {
#pragma unroll
        for (int w = 0; w < 4; ++w)
            *reinterpret_cast<uint32_t*>(sbuf + (quad & 1) * kGdScales + w * (kGaWide * 4) + fw * 256 + lane * 4) =
                mx_scales_take(sw4[w], 16 * quad + 4 * w, d.nb);
    };
    const uint32_t base = lds_addr(lds);
    u32x4 x[2][8], c[2];  // a step's fragments: G's of two 32-row halves; codes of two blocks
    float sc[2];          // and their scales
    auto read = [&](int k, int cur) {
        const uint32_t s = base + cur * kGdG;
        // the two blocks of the lane's column of R, and their scales
        const int r0 = cw + (lane & 31), sw = mx_swz(lane & 31), b0 = 4 * (k & 1) + 2 * h;
        const uint32_t pb = base + kGdDepth * kGdG + ((k >> 1) & 1) * kGdCodes + r0 * 128;
        const uint32_t pe = base + kGdDepth * kGdG + 2 * kGdCodes + ((k >> 2) & 1) * kGdScales + (k & 3) * (kGaWide * 4) + r0 * 4;
        const uint32_t q[2] = {pb + ((b0 ^ sw) << 4), pb + (((b0 + 1) ^ sw) << 4)};
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
        sc[0] = mx4_scale(e & 255u);
        sc[1] = mx4_scale((e >> 8) & 255u);
        if constexpr (Any) {  // past the end G is zero; codes and scales are whatever is there
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (4 * k + 2 * h + t >= d.nb) sc[t] = 1.0f;
        }
    };
    auto multiply = [&]() {
#pragma unroll
        for (int u = 0; u < 8; ++u) {  // 8 values: dword u & 3 of block u >> 2
            const bfv8 fb = __builtin_bit_cast(bfv8, mx4_to_bf16(c[u >> 2][u & 3], sc[u >> 2]));
#pragma unroll
            for (int ib = 0; ib < 2; ++ib) acc[ib] = mfma32(__builtin_bit_cast(bfv8, x[ib][u]), fb, acc[ib]);
        }
    };
    // Before step k's barrier a wave that fetches G waits until only steps k + 1 .. k + 3 are
    // outstanding (Any: has stored step k). One that fetches U^T issued the codes of a pair of
    // steps in the even step before it and the scales of four steps two steps before them:
    // before an even step it waits for all, before an odd one for nothing that step k - 1
    // issued. What a step fills was last read before its barrier.
    // The moments of the wave's piece of R are loaded before everything else (Any with kFold: after
    // the products, for want of registers).
    const bool active = cw < d.r;
    constexpr bool kEarly = Parts == kWhole || (!Any && Parts == kFold);
    GxMoments<true> mv;
    if (kEarly && active) mv.load(d, i0, cw, lane);
    auto next_u = [&](int k) {  // waves 4 .. 7, even steps
        if constexpr (Any) {  // loaded two steps before they are stored
            if (k & 2) store_scales((k >> 2) + 1);
            else if (d.nb >= 4) scales((k >> 2) + 1);
        } else {
            if (k & 2) scales((k >> 2) + 1);
        }
        codes((k >> 1) + 1);
    };
    if (!fetch_g) {
        scales(k0 >> 2);
        if constexpr (Any) store_scales(k0 >> 2);
        codes(k0 >> 1);
    }
    // kGxDirect: the waves that fetch U^T multiply a step's fragments behind the next barrier, before
    // they read that step's: their products run beside the LDS reads of the others (each SIMD
    // has one of either kind): 74 us for the four 4096 x 4096 matrices, 78 without. (Any:
    // 97 and 90 us for 1951 x 3810 and 3750 x 4266, so there every wave multiplies at once.)
    int cur = 0;
    auto store_part = [&]() {
        int ln = lane;
        __asm__ volatile("" : "+v"(ln));  // addresses are computed here: before the loop they cost 1 us
        float* const p = d.part + (part * static_cast<int64_t>(d.D) + i0) * d.rp + cw;
        const int rows = static_cast<int>(min<int64_t>(d.D - i0, kGdRows));
#pragma unroll
        for (int ib = 0; ib < 2; ++ib)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int r = ib * 32 + acc_row(v, ln);
                if (r < rows) *gst<float>(p + r * d.rp + acc_col(ln)) = acc[ib][v];
            }
        ++part;
    };
    int part_end = k0 + d.kper;
    auto end_part = [&](int done) {  // the steps before `done` are in acc; the last part's end is below
        if (Parts == kWhole || done != part_end || done == k1) return;
        part_end += d.kper;
        if (Parts == kStore) store_part();
#pragma unroll
        for (int ib = 0; ib < 2; ++ib)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                if (Parts == kFold) sum[ib][v] += acc[ib][v];
                acc[ib][v] = 0.0f;
            }
    };
    auto first_half = [&](int k) {  // waves 0 .. 3
        if (active) {
            read(k, cur);
            multiply();
            end_part(k + 1);
        }
        cur = cur == kGdDepth - 1 ? 0 : cur + 1;
    };
    auto second_half = [&](int k) {  // waves 4 .. 7
        if (active) {
            if (!Any && k > k0) multiply();
            if (!Any) end_part(k);
#pragma unroll
            for (int ib = 0; ib < 2; ++ib) __asm__ volatile("" : "+v"(acc[ib]));  // before the reads
            read(k, cur);
            if (Any) {
                multiply();
                end_part(k + 1);
            }
        }
        cur = cur == kGdDepth - 1 ? 0 : cur + 1;
    };
    if constexpr (Any) {
        u32x4 ve[kA], vo[kA];  // even and odd steps
        if (fetch_g) {
            load_g(k0, ve);
            load_g(k0 + 1, vo);
            store_g(k0, ve, lds);
            load_g(k0 + 2, ve);
        }
        // (two loops, as in mx4_accumulate)
        if (fetch_g) {
            auto step = [&](int k, u32x4 (&v)[kA]) {
                wait_lds_and_sync(false);
                store_g(k + 1, v, lds + (cur == kGdDepth - 1 ? 0 : cur + 1) * kGdG);
                load_g(k + 3, v);
                first_half(k);
            };
            for (int k = k0; k < k1; k += 2) {
                step(k, vo);
                if (k + 1 < k1) step(k + 1, ve);
            }
        } else {
            for (int k = k0; k < k1; ++k) {
                wait_lds_and_sync(!(k & 1));
                if (!(k & 1)) next_u(k);
                second_half(k);
            }
        }
    } else {
        if (fetch_g) {
#pragma unroll
            for (int k = 0; k < kGdDepth - 1; ++k) stage(k0 + k, lds + k * kGdG);
        }
        if (fetch_g) {
            for (int k = k0; k < k1; ++k) {
                wait_and_sync<3 * kA>();
                stage(k + kGdDepth - 1, lds + (cur == 0 ? kGdDepth - 1 : cur - 1) * kGdG);
                first_half(k);
            }
        } else {
            for (int k = k0; k < k1; ++k) {
                if (!(k & 1)) wait_and_sync<0>();
                else if ((k & 3) == 3) wait_and_sync<kB + 4>();
                else wait_and_sync<kB>();
                if (!(k & 1)) next_u(k);
                second_half(k);
            }
        }
    }
    if (!Any && !fetch_g && active) multiply();
    wait_and_sync<0>();
    if (!active) return;
    if constexpr (Parts == kFold) {
#pragma unroll
        for (int ib = 0; ib < 2; ++ib)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[ib][v] = sum[ib][v] + acc[ib][v];
    } else if constexpr (Parts == kStore) {
        store_part();
        return;
    }
    if (!kEarly) mv.load(d, i0, cw, lane);
    float* lw = reinterpret_cast<float*>(lds) + wave * kGxEx;
    gx_epilogue(d, a, acc[0], acc[1], mv, i0, cw, lw, lane);
}

template <bool Any>
__global__ __launch_bounds__(kGdWaves * 64) void k_gx_project(GxTable t, GaArgs a, int nright) {
    __shared__ __attribute__((aligned(128))) uint8_t lds[kGdLds];
    const int2 it = t.items[blockIdx.x];
    const GxDesc d = t.desc[it.x];
    const int64_t i0 = static_cast<int64_t>(it.y / d.kitems) * kGdRows;
    const int part = it.y % d.kitems * d.kitem;
    auto tile = [&](auto parts) {
        constexpr GxParts kParts = decltype(parts)::value;
        if (it.x < nright) gx_tile<false, Any, kParts>(d, i0, part, a, lds);
        else gx_tile<true, Any, kParts>(d, i0, part, a, lds);
    };
    if (d.ks == 1) tile(std::integral_constant<GxParts, kWhole>{});
    else if (d.kitems == 1) tile(std::integral_constant<GxParts, kFold>{});
    else tile(std::integral_constant<GxParts, kStore>{});
}

void launch_gx_project(const GxTable& t, int64_t n, int nright, const GaArgs& a, int form, hipStream_t s) {
    if (n <= 0) return;
    const dim3 grid(static_cast<uint32_t>(n)), block(kGdWaves * 64);
    if (form == kGxAny) hipLaunchKernelGGL(k_gx_project<true>, grid, block, 0, s, t, a, nright);
    else hipLaunchKernelGGL(k_gx_project<false>, grid, block, 0, s, t, a, nright);
}

// R of a split contraction: its parts' sums added up in order, then AdamW; a thread has 8 columns of a row.
__global__ __launch_bounds__(kGxJoinChunks) void k_gx_join(GxTable t, GaArgs a) {
    const int2 it = t.items[blockIdx.x];
    const GxDesc d = t.desc[it.x];
    const int chunks = d.rp / 8;
    const int64_t c = static_cast<int64_t>(it.y) * kGxJoinChunks + threadIdx.x;
    const int64_t row = c / chunks;
    if (row >= d.D) return;
    const int col = 8 * static_cast<int>(c - row * chunks);
    const int valid = min(max(d.r - col, 0), 8);
    float m[8], v[8], r[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    load_any8(d.em, row * d.r + col, valid, false, m);
    load_any8(d.ev, row * d.r + col, valid, false, v);
    for (int s = 0; s < d.ks; ++s) {
        float x[8];
        load_any8(d.part, (s * static_cast<int64_t>(d.D) + row) * d.rp + col, 8, false, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] += x[e];
    }
    gx_adamw8(d, a, row, col, valid, m, v, r);
}

void launch_gx_join(const GxTable& t, int64_t n, const GaArgs& a, hipStream_t s) {
    if (n <= 0) return;
    hipLaunchKernelGGL(k_gx_join, dim3(static_cast<uint32_t>(n)), dim3(kGxJoinChunks), 0, s, t, a);
}

// ------------------------------------------------------------------ MX4 gradient

// The product of mx4_tile.h, whose column tile holds all of R's columns (MxForm), with AdamW on R:
// 61 us for 11008 x 4096 and 4096 x 11008 at rank 256 (128-row tiles; 77 with 64), whose bytes
// take 33 at the rate of a copy: 172 tiles on 256 CUs, each first multiplying, then streaming
// its moments. (Their first half loaded before the product: 63 us.)
template <int IB, int WN, int NW>
__global__ __launch_bounds__(NW * 64) void k_gx_project_mx4(GxTable t, GaArgs a) {
    using T = MxTile<IB, WN, NW>;
    constexpr int kEx = NW * kGxEx * 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[T::kLds];
    static_assert(T::kLds >= kEx, "exchange space");
    const int2 it = t.items[blockIdx.x];
    const GxDesc d = t.desc[it.x];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t i0 = static_cast<int64_t>(it.y) * T::kRowsA;
    const MxOperand oa{reinterpret_cast<const uint8_t*>(d.g), d.gs, d.D, d.nb}, ob{d.uc, d.us, d.r, d.nb};
    float* lw = reinterpret_cast<float*>(lds) + wave * kGxEx;
    f32x16 acc[IB][2];
    zero_acc(acc);
    mx4_accumulate<IB, WN, NW>(oa, ob, i0, 0, lds, acc);
    const int64_t row = i0 + (wave / WN) * 32 * IB;
    const int col = (wave % WN) * 64;
    if (col >= d.r) return;
#pragma unroll
    for (int ib = 0; ib < IB; ++ib) {
        GxMoments<false> mv;
        mv.load(d, row + ib * 32, col, lane);
        gx_epilogue(d, a, acc[ib][0], acc[ib][1], mv, row + ib * 32, col, lw, lane);
    }
}

void launch_gx_project_mx4(const GxTable& t, int64_t n, const GaArgs& a, int form, hipStream_t s) {
    if (n <= 0) return;
    const dim3 grid(static_cast<uint32_t>(n));
    switch (form) {
        case kMxNarrow: hipLaunchKernelGGL((k_gx_project_mx4<1, 2, 4>), grid, dim3(256), 0, s, t, a); break;
        case kMxWide: hipLaunchKernelGGL((k_gx_project_mx4<1, 4, 8>), grid, dim3(512), 0, s, t, a); break;
        default: hipLaunchKernelGGL((k_gx_project_mx4<2, 4, 8>), grid, dim3(512), 0, s, t, a); break;
    }
}

// ------------------------------------------------------------------ back-projection + update

// W <- decay W - coef N U^T (left: U N^T) with U decoded into registers. An item is a band of
// 256 rows of U and up to tpi tiles of 64 rows of N. 8 waves: wave w holds the fragments of U
// rows 32 w .. + 31 for the whole rank (64 VGPRs) and multiplies them by each tile of N.
// N's two planes are staged by global_load_lds into one of two buffers (64 KB each: rows of
// 256, chunk c of row r at c ^ (r & 15)), the next tile's while the current one is
// multiplied; the parameter part of a tile is loaded a whole tile ahead. (64 rows of U per wave and
// 32 of N read half as much LDS, but their 128 VGPRs of U leave no registers to read
// fragments ahead: 144 instead of 130 us for the MLP matrices of a layer, bf16.)
// At rank 256 four 4096 x 4096 fp32 matrices take 120 us (a copy of their bytes 114) and 11008 x
// 4096 and 4096 x 11008 in bf16 125 (75; by the counters LDS serves accesses in 31% of the CUs'
// cycles and the matrix units work in 39%, one after the other within a wave: reads of W, fragment
// reads, products and stores of a tile overlap only in part).
constexpr int kGbN = kGaTile;                                 // rows of N per tile
constexpr int kGbDma = 2 * kGbN * (kGaWide / 8) / 512;        // 16-byte transfers per lane per tile: 8

__device__ __forceinline__ void gb_stage(const GxDesc& d, int64_t n0, uint16_t* buf, int wave, int lane) {
    // instruction j: rows 2 jr, 2 jr + 1 of plane j / 32 (jr = j % 32), 32 chunks each
    __asm__ volatile("" : "+v"(lane));
#pragma unroll
    for (int i = 0; i < kGbDma; ++i) {
        const int j = wave + 8 * i;
        const int plane = j >> 5, jr = j & 31;
        const int row = 2 * jr + (lane >> 5);
        const int cc = min((lane & 31) ^ (row & 15), d.rp / 8 - 1);  // global chunk held at position lane & 31
        const int64_t grow = min(n0 + row, static_cast<int64_t>(d.D) - 1);
        const uint16_t* src = (plane ? d.nl : d.nh) + grow * d.rp + cc * 8;
        __builtin_amdgcn_global_load_lds((const MEO_GLOBAL void*)src,
                                         (__attribute__((address_space(3))) void*)(buf + j * 512), 16, 0, 0);
    }
}

template <bool Left, bool XB>
__device__ __forceinline__ void gb_item(const GxDesc& d, int item, const GaArgs& a, uint16_t* nb0, uint16_t* nb1, float* exb) {
    static_assert(kGbDma == 8, "wait counts below");
    constexpr int kP = XB ? 4 : 8;  // 16-byte parameter loads (and stores) per lane per tile
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int nc = d.btj;  // chunks of tpi tiles per band
    const int band = item / nc, chunk = item % nc;
    const int64_t u0 = static_cast<int64_t>(band) * kGaWide;
    const int64_t nt0 = static_cast<int64_t>(chunk) * d.tpi;
    const int ntiles = static_cast<int>(min<int64_t>(d.tpi, (d.D + kGbN - 1) / kGbN - nt0));
    const int nks = d.rp / 16;  // 16-wide contraction sub-steps, an even number
    using PT = typename std::conditional<XB, uint16_t, float>::type;
    PT* const x = static_cast<PT*>(d.x);
    // The wave's 32 rows of U are one block of each row of U^T: decoded into LDS as [r][32]
    // (the stages are free yet) and read back transposed.
    bfv8 uf[16];
    {
        uint16_t* lu = (wave < 4 ? nb0 : nb1) + (wave & 3) * 8192;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = lane + 64 * j;
            u32x4 c;
            uint32_t e;
            ld_mx_block(d, r, u0 / kMxBlock + wave, c, e);
            const float sc = mx4_scale(e);
#pragma unroll
            for (int i = 0; i < 4; ++i) st_lds8(lu + r * 32 + i * 8, mx4_to_bf16(c[i], sc));
        }
        __syncthreads();
        const int g = lane >> 4, e = (lane >> 2) & 3, q = lane & 3;
#pragma unroll
        for (int ks = 0; ks < 16; ++ks) {
            const uint16_t* p = lu + (16 * ks + 8 * (g >> 1) + e) * 32 + 16 * (g & 1) + 4 * q;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p + 4 * 32));
            const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            uf[ks] = __builtin_bit_cast(bfv8, v);
        }
    }
    MEO_WAIT_VM(0);
#pragma unroll
    for (int ks = 0; ks < 16; ++ks) __asm__ volatile("" : "+v"(uf[ks]));
    __syncthreads();  // every wave has its fragments: the stages may be filled
    // W cells of the wave: two 32 x 32 blocks (nb: the tile's 32-row halves of N); in block nb,
    // lane holds rows (lane >> 2) + 16 q (q < 2), columns 8 (lane & 3) .. + 7.
    auto cell = [&](int64_t n0, int nb, int q, int64_t& row, int64_t& col) {
        int ln = lane;
        __asm__ volatile("" : "+v"(ln));
        const int r = (ln >> 2) + 16 * q, c = 8 * (ln & 3);
        if (Left) {  // rows from U, columns from N
            row = u0 + wave * 32 + r;
            col = n0 + nb * 32 + c;
        } else {     // rows from N, columns from U
            row = n0 + nb * 32 + r;
            col = u0 + wave * 32 + c;
        }
    };
    u32x4 w0[2][2][2], w1[2][2][2];  // even and odd tiles: [nb][q][16-byte half]
    // exactly kP loads, rows and columns clamped into the tensor
    auto load_w = [&](int64_t n0, u32x4 (&wp)[2][2][2]) {
        if (d.n < 8) return;
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                int64_t row, col;
                cell(n0, nb, q, row, col);
                row = min(row, static_cast<int64_t>(d.m) - 1);
                col = min(col, static_cast<int64_t>(d.n) - 8);
                const PT* p = x + row * d.n + col;
                wp[nb][q][0] = *gld<u32x4_any>(p);
                if (!XB) wp[nb][q][1] = *gld<u32x4_any>(p + 4);
            }
    };
    f32x16 acc[2];
    auto multiply = [&](const uint16_t* buf) {
        // Fragment reads in asm blocks that wait for their own reads (the compiler cannot tell
        // which stage an LDS read hits). Two sub-steps per block; the low plane sits 32 KB
        // after the high one, rows 32 on 16 KB (the same swizzle).
        static_assert(kGbN * 256 * 2 == 32768, "offsets in the reads below");
        const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(buf)) + (lane & 31) * 512;
        const int sw = lane & 15;
#pragma unroll
        for (int ks = 0; ks < 16; ks += 2) {
            if (ks >= nks) break;
            int swv = sw;
            __asm__ volatile("" : "+v"(swv));  // computed here, not hoisted and spilled
            const uint32_t a0 = base + static_cast<uint32_t>(((2 * ks + (lane >> 5)) ^ swv) << 4);
            const uint32_t a1 = base + static_cast<uint32_t>(((2 * ks + 2 + (lane >> 5)) ^ swv) << 4);
            u32x4 h0, l0, h1, l1, h2, l2, h3, l3;
            __asm__ volatile(
                "ds_read_b128 %0, %8\n\t"
                "ds_read_b128 %1, %8 offset:32768\n\t"
                "ds_read_b128 %2, %8 offset:16384\n\t"
                "ds_read_b128 %3, %8 offset:49152\n\t"
                "ds_read_b128 %4, %9\n\t"
                "ds_read_b128 %5, %9 offset:32768\n\t"
                "ds_read_b128 %6, %9 offset:16384\n\t"
                "ds_read_b128 %7, %9 offset:49152\n\t"
                "s_waitcnt lgkmcnt(0)"
                : "=&v"(h0), "=&v"(l0), "=&v"(h1), "=&v"(l1), "=&v"(h2), "=&v"(l2), "=&v"(h3), "=&v"(l3)
                : "v"(a0), "v"(a1));
            // [sub-step][plane][half of N]
            const u32x4 f[2][2][2] = {{{h0, h1}, {l0, l1}}, {{h2, h3}, {l2, l3}}};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int pl = 0; pl < 2; ++pl)
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb) {
                        const bfv8 fn = __builtin_bit_cast(bfv8, f[i][pl][nb]);
                        acc[nb] = Left ? mfma32(uf[ks + i], fn, acc[nb]) : mfma32(fn, uf[ks + i], acc[nb]);
                    }
        }
    };
    // W <- decay W - coef C for a tile, through the wave's exchange region (one 32 x 32 block
    // at a time, so that each lane ends with 8 consecutive columns of a row). exact: every
    // cell inside the tensor, exactly kP 16-byte stores; otherwise a full wait after them.
    auto update = [&](int64_t n0, auto ec, const u32x4 (&wp)[2][2][2]) {
        constexpr bool exact = decltype(ec)::value;
        int ln = lane;
        __asm__ volatile("" : "+v"(ln));
        float* lw = exb + wave * kGxEx;
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
            for (int v = 0; v < 16; ++v) lw[ur_ex(acc_row(v, ln), acc_col(ln))] = acc[nb][v];
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float cq[8], w[8];
                {
                    const int r = (ln >> 2) + 16 * q, c = 8 * (ln & 3);
                    const f32x4 c0 = *reinterpret_cast<const f32x4*>(lw + ur_ex(r, c));
                    const f32x4 c1 = *reinterpret_cast<const f32x4*>(lw + ur_ex(r, c + 4));
                    cq[0] = c0.x; cq[1] = c0.y; cq[2] = c0.z; cq[3] = c0.w;
                    cq[4] = c1.x; cq[5] = c1.y; cq[6] = c1.z; cq[7] = c1.w;
                }
                int64_t row, col;
                cell(n0, nb, q, row, col);
                if constexpr (exact) {
                    PT* xp = x + row * d.n + col;
                    if (XB) {
                        bf16x8(wp[nb][q][0], w);
                    } else {
                        const u32x4 x0 = wp[nb][q][0], x1 = wp[nb][q][1];
                        w[0] = __uint_as_float(x0.x); w[1] = __uint_as_float(x0.y);
                        w[2] = __uint_as_float(x0.z); w[3] = __uint_as_float(x0.w);
                        w[4] = __uint_as_float(x1.x); w[5] = __uint_as_float(x1.y);
                        w[6] = __uint_as_float(x1.z); w[7] = __uint_as_float(x1.w);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = a.decay * w[e] - a.coef * cq[e];
                    if (XB) {
                        *gst<u32x4_any>(xp) = pack_bf16x8(w);
                    } else {
                        *gst<f32x4_any>(xp) = f32x4{w[0], w[1], w[2], w[3]};
                        *gst<f32x4_any>(xp + 4) = f32x4{w[4], w[5], w[6], w[7]};
                    }
                } else {
                    if (row >= d.m || col >= d.n) continue;
                    const int64_t at = row * d.n + col;
                    const int valid = static_cast<int>(min<int64_t>(d.n - col, 8));
                    load_any8(x, at, valid, XB, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = a.decay * w[e] - a.coef * cq[e];
                    store_any8(x, at, valid, XB, w);
                }
            }
            __builtin_amdgcn_wave_barrier();  // this block's gathers before the next block's spill
        }
        if constexpr (!exact) MEO_WAIT_VM(0);
    };
    auto zero = [&]() {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[b][v] = 0.0f;
    };
    // Exact counts need every tile of the item whole.
    const bool exact = d.n >= 8 && (nt0 + ntiles) * kGbN <= d.D && u0 + kGaWide <= d.d;
    // Tile i uses buffer i & 1. One barrier a tile: behind it stage i has landed for every wave and
    // every wave has multiplied tile i - 1, so the stage for tile i + 1 goes out (past the last
    // tile that one again, so counts stay fixed). Waves 0 .. 3 then multiply tile i and update
    // it; waves 4 .. 7 (the others of each SIMD) first update tile i - 1 and then multiply, so
    // that one's products run beside the other's update (all in one order: 131 us for the
    // MLP matrices of a layer, bf16). A tile's parameters are loaded a tile before their use.
    const int last = ntiles - 1;
    auto row0 = [&](int i) { return (nt0 + min(i, last)) * kGbN; };
    auto sync_and_stage = [&](int i, uint16_t* next) {
        __asm__ volatile("s_barrier" ::: "memory");
        gb_stage(d, row0(i + 1), next, wave, lane);
    };
    // The compiler's own wait for loaded parameters, put where the order of what is in flight is
    // plain to it.
    auto landed = [&](u32x4 (&w)[2][2][2]) {
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                __asm__ volatile("" : "+v"(w[nb][q][0]));
                if (!XB) __asm__ volatile("" : "+v"(w[nb][q][1]));
            }
    };
    gb_stage(d, row0(0), nb0, wave, lane);
    load_w(row0(0), w0);
    MEO_WAIT_VM(0);
    auto run = [&](auto ec) {
        constexpr bool kExact = decltype(ec)::value;
        if (wave < 4) {
            // before the barrier only the update's kP stores may be in flight
            auto tile = [&](int i, uint16_t* cur, uint16_t* next, u32x4 (&wc)[2][2][2], u32x4 (&wn)[2][2][2]) {
                sync_and_stage(i, next);
                load_w(row0(i + 1), wn);
                zero();
                multiply(cur);
                update(row0(i), ec, wc);
                if constexpr (kExact) MEO_WAIT_VM(kP);
                else MEO_WAIT_VM(0);
                landed(wn);
            };
            tile(0, nb0, nb1, w0, w1);
            for (int i = 1; i < ntiles; i += 2) {
                tile(i, nb1, nb0, w1, w0);
                if (i + 1 >= ntiles) break;
                tile(i + 1, nb0, nb1, w0, w1);
            }
        } else {
            // before the barrier the update's stores and the loads after them may be in flight
            auto tile = [&](int i, uint16_t* cur, uint16_t* next, u32x4 (&wc)[2][2][2], u32x4 (&wn)[2][2][2], auto first) {
                sync_and_stage(i, next);
                if constexpr (!decltype(first)::value) update(row0(i - 1), ec, wn);
                load_w(row0(i + 1), wn);
                zero();
                multiply(cur);
                if constexpr (!kExact) MEO_WAIT_VM(0);
                else if constexpr (decltype(first)::value) MEO_WAIT_VM(kP);
                else MEO_WAIT_VM(2 * kP);
                landed(wc);
            };
            tile(0, nb0, nb1, w0, w1, std::true_type{});
            for (int i = 1; i < ntiles; i += 2) {
                tile(i, nb1, nb0, w1, w0, std::false_type{});
                if (i + 1 >= ntiles) break;
                tile(i + 1, nb0, nb1, w0, w1, std::false_type{});
            }
            if (last & 1) update(row0(last), ec, w1);
            else update(row0(last), ec, w0);
        }
    };
    if (exact) run(std::true_type{});
    else run(std::false_type{});
    MEO_WAIT_VM(0);
}

template <bool XB>
__global__ __launch_bounds__(512, 1) void k_gx_back(GxTable t, GaArgs a, int nright) {
    __shared__ __attribute__((aligned(16))) uint16_t nb0[2 * kGbN * 256];
    __shared__ __attribute__((aligned(16))) uint16_t nb1[2 * kGbN * 256];
    __shared__ __attribute__((aligned(16))) float exb[8 * kGxEx];
    const int2 it = t.items[blockIdx.x];
    if (it.x < 0) return;  // an empty item of the XCD-dealt list
    const GxDesc d = t.desc[it.x];
    if (it.x < nright) gb_item<false, XB>(d, it.y, a, nb0, nb1, exb);
    else gb_item<true, XB>(d, it.y, a, nb0, nb1, exb);
}

void launch_gx_back(const GxTable& t, int64_t n, int nright, const GaArgs& a, bool xbf16, hipStream_t s) {
    if (n <= 0) return;
    const dim3 grid(static_cast<uint32_t>(n));
    if (xbf16) hipLaunchKernelGGL(k_gx_back<true>, grid, dim3(512), 0, s, t, a, nright);
    else hipLaunchKernelGGL(k_gx_back<false>, grid, dim3(512), 0, s, t, a, nright);
}

}  // namespace meo
