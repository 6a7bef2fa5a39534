// The product of two MX4 operands over a tile, shared by the matmul and by GaLore's
// projection of an MX4 gradient.
#pragma once
#include "mx4.h"

#include <type_traits>

namespace meo {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct MxOperand {
    const uint8_t* codes;   // [rows][16 nb]
    const uint8_t* scales;  // [rows][nb]
    int64_t rows;
    int32_t nb;
};

// Waits until at most N vector-memory operations are outstanding and every LDS access has
// finished, then for the block's other waves.
template <int N>
__device__ __forceinline__ void wait_and_sync() {
    __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16 bytes per lane straight from global memory into LDS, lane l at dst + 16 l (4: 4 bytes).
__device__ __forceinline__ void dma16(const uint8_t* src, void* dst) {
    __builtin_amdgcn_global_load_lds((const MEO_GLOBAL void*)src, (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}
__device__ __forceinline__ void dma4(const uint8_t* src, void* dst) {
    __builtin_amdgcn_global_load_lds((const MEO_GLOBAL void*)src, (__attribute__((address_space(3))) void*)dst, 4, 0, 0);
}

// The LDS reads of a step's fragments are one asm block with their wait: before a plain read
// the compiler, which cannot tell what a transfer in flight writes, would wait for every
// transfer. The stages read have landed (the wait and barrier before), and one wait for
// all reads exposes the LDS latency once per step.

// An MX4 step: four 16-byte chunks (p[t]) of A's row and of the rows 32 on (IB = 2), the
// same of B's two rows (q[t]), the scale words at ea (and 32 rows on), eb and 32 rows on.
template <int IB>
__device__ __forceinline__ void lds_read_mx(const uint32_t* p, const uint32_t* q, uint32_t ea, uint32_t eb, u32x4 (&ca)[2][4],
                                            u32x4 (&cb)[2][4], uint32_t* e) {
    u32x4 a0, a1, a2, a3, a4, a5, a6, a7, b0, b1, b2, b3, b4, b5, b6, b7;
    uint32_t e0, e1, e2, e3;
    if constexpr (IB == 2) {
        __asm__ volatile(
            "ds_read_b32 %16, %28\n\t"
            "ds_read_b32 %17, %28 offset:128\n\t"
            "ds_read_b32 %18, %29\n\t"
            "ds_read_b32 %19, %29 offset:128\n\t"
            "ds_read_b128 %0, %20\n\t"
            "ds_read_b128 %8, %24\n\t"
            "ds_read_b128 %12, %24 offset:4096\n\t"
            "ds_read_b128 %4, %20 offset:4096\n\t"
            "ds_read_b128 %1, %21\n\t"
            "ds_read_b128 %9, %25\n\t"
            "ds_read_b128 %13, %25 offset:4096\n\t"
            "ds_read_b128 %5, %21 offset:4096\n\t"
            "ds_read_b128 %2, %22\n\t"
            "ds_read_b128 %10, %26\n\t"
            "ds_read_b128 %14, %26 offset:4096\n\t"
            "ds_read_b128 %6, %22 offset:4096\n\t"
            "ds_read_b128 %3, %23\n\t"
            "ds_read_b128 %11, %27\n\t"
            "ds_read_b128 %15, %27 offset:4096\n\t"
            "ds_read_b128 %7, %23 offset:4096\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(a0), "=&v"(a1), "=&v"(a2), "=&v"(a3), "=&v"(a4), "=&v"(a5), "=&v"(a6), "=&v"(a7), "=&v"(b0), "=&v"(b1),
              "=&v"(b2), "=&v"(b3), "=&v"(b4), "=&v"(b5), "=&v"(b6), "=&v"(b7), "=&v"(e0), "=&v"(e1), "=&v"(e2), "=&v"(e3)
            : "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]), "v"(q[0]), "v"(q[1]), "v"(q[2]), "v"(q[3]), "v"(ea), "v"(eb));
        ca[1][0] = a4; ca[1][1] = a5; ca[1][2] = a6; ca[1][3] = a7;
    } else {
        __asm__ volatile(
            "ds_read_b32 %12, %23\n\t"
            "ds_read_b32 %13, %24\n\t"
            "ds_read_b32 %14, %24 offset:128\n\t"
            "ds_read_b128 %0, %15\n\t"
            "ds_read_b128 %4, %19\n\t"
            "ds_read_b128 %8, %19 offset:4096\n\t"
            "ds_read_b128 %1, %16\n\t"
            "ds_read_b128 %5, %20\n\t"
            "ds_read_b128 %9, %20 offset:4096\n\t"
            "ds_read_b128 %2, %17\n\t"
            "ds_read_b128 %6, %21\n\t"
            "ds_read_b128 %10, %21 offset:4096\n\t"
            "ds_read_b128 %3, %18\n\t"
            "ds_read_b128 %7, %22\n\t"
            "ds_read_b128 %11, %22 offset:4096\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(a0), "=&v"(a1), "=&v"(a2), "=&v"(a3), "=&v"(b0), "=&v"(b1), "=&v"(b2), "=&v"(b3), "=&v"(b4), "=&v"(b5),
              "=&v"(b6), "=&v"(b7), "=&v"(e0), "=&v"(e2), "=&v"(e3)
            : "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]), "v"(q[0]), "v"(q[1]), "v"(q[2]), "v"(q[3]), "v"(ea), "v"(eb));
        e1 = 0;
    }
    ca[0][0] = a0; ca[0][1] = a1; ca[0][2] = a2; ca[0][3] = a3;
    cb[0][0] = b0; cb[0][1] = b1; cb[0][2] = b2; cb[0][3] = b3;
    cb[1][0] = b4; cb[1][1] = b5; cb[1][2] = b6; cb[1][3] = b7;
    e[0] = e0; e[1] = e1; e[2] = e2; e[3] = e3;
}

// A bf16 step: eight 16-byte chunks (p[i]) of G's row and of the row 32 on, two chunks (q[t])
// of a row of codes and their scale word (pe).
__device__ __forceinline__ void lds_read_row(const uint32_t* p, const uint32_t* q, uint32_t pe, u32x4 (&g)[2][8], u32x4* c,
                                             uint32_t& e) {
    u32x4 g0, g1, g2, g3, g4, g5, g6, g7, h0, h1, h2, h3, h4, h5, h6, h7, c0, c1;
    uint32_t e0;
    __asm__ volatile(
        "ds_read_b32 %18, %29\n\t"
        "ds_read_b128 %16, %27\n\t"
        "ds_read_b128 %0, %19\n\t"
        "ds_read_b128 %8, %19 offset:8192\n\t"
        "ds_read_b128 %1, %20\n\t"
        "ds_read_b128 %9, %20 offset:8192\n\t"
        "ds_read_b128 %2, %21\n\t"
        "ds_read_b128 %10, %21 offset:8192\n\t"
        "ds_read_b128 %3, %22\n\t"
        "ds_read_b128 %11, %22 offset:8192\n\t"
        "ds_read_b128 %17, %28\n\t"
        "ds_read_b128 %4, %23\n\t"
        "ds_read_b128 %12, %23 offset:8192\n\t"
        "ds_read_b128 %5, %24\n\t"
        "ds_read_b128 %13, %24 offset:8192\n\t"
        "ds_read_b128 %6, %25\n\t"
        "ds_read_b128 %14, %25 offset:8192\n\t"
        "ds_read_b128 %7, %26\n\t"
        "ds_read_b128 %15, %26 offset:8192\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(g0), "=&v"(g1), "=&v"(g2), "=&v"(g3), "=&v"(g4), "=&v"(g5), "=&v"(g6), "=&v"(g7), "=&v"(h0), "=&v"(h1),
          "=&v"(h2), "=&v"(h3), "=&v"(h4), "=&v"(h5), "=&v"(h6), "=&v"(h7), "=&v"(c0), "=&v"(c1), "=&v"(e0)
        : "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]), "v"(p[4]), "v"(p[5]), "v"(p[6]), "v"(p[7]), "v"(q[0]), "v"(q[1]), "v"(pe));
    g[0][0] = g0; g[0][1] = g1; g[0][2] = g2; g[0][3] = g3; g[0][4] = g4; g[0][5] = g5; g[0][6] = g6; g[0][7] = g7;
    g[1][0] = h0; g[1][1] = h1; g[1][2] = h2; g[1][3] = h3; g[1][4] = h4; g[1][5] = h5; g[1][6] = h6; g[1][7] = h7;
    c[0] = c0; c[1] = c1;
    e = e0;
}

// Two chunks of codes and their scale word; and the eight fragments of 32 rows of G^T from
// its tile as it lies: sixteen transposed 8-byte reads of 16-bit values, 4 rows of 128
// bytes apart each.
__device__ __forceinline__ void lds_read_codes(const uint32_t* q, uint32_t pe, u32x4* c, uint32_t& e) {
    u32x4 c0, c1;
    uint32_t e0;
    __asm__ volatile(
        "ds_read_b32 %2, %5\n\t"
        "ds_read_b128 %0, %3\n\t"
        "ds_read_b128 %1, %4\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(c0), "=&v"(c1), "=&v"(e0)
        : "v"(q[0]), "v"(q[1]), "v"(pe));
    c[0] = c0; c[1] = c1;
    e = e0;
}
__device__ __forceinline__ void lds_read_tr(uint32_t p, u32x4* g) {
    u32x2 x0, x1, x2, x3, x4, x5, x6, x7, x8, x9, xa, xb, xc, xd, xe, xf;
    __asm__ volatile(
        "ds_read_b64_tr_b16 %0, %16\n\t"
        "ds_read_b64_tr_b16 %1, %16 offset:512\n\t"
        "ds_read_b64_tr_b16 %2, %16 offset:1024\n\t"
        "ds_read_b64_tr_b16 %3, %16 offset:1536\n\t"
        "ds_read_b64_tr_b16 %4, %16 offset:2048\n\t"
        "ds_read_b64_tr_b16 %5, %16 offset:2560\n\t"
        "ds_read_b64_tr_b16 %6, %16 offset:0xc00\n\t"
        "ds_read_b64_tr_b16 %7, %16 offset:3584\n\t"
        "ds_read_b64_tr_b16 %8, %16 offset:4096\n\t"
        "ds_read_b64_tr_b16 %9, %16 offset:4608\n\t"
        "ds_read_b64_tr_b16 %10, %16 offset:5120\n\t"
        "ds_read_b64_tr_b16 %11, %16 offset:5632\n\t"
        "ds_read_b64_tr_b16 %12, %16 offset:6144\n\t"
        "ds_read_b64_tr_b16 %13, %16 offset:6656\n\t"
        "ds_read_b64_tr_b16 %14, %16 offset:7168\n\t"
        "ds_read_b64_tr_b16 %15, %16 offset:7680\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x0), "=&v"(x1), "=&v"(x2), "=&v"(x3), "=&v"(x4), "=&v"(x5), "=&v"(x6), "=&v"(x7), "=&v"(x8), "=&v"(x9),
          "=&v"(xa), "=&v"(xb), "=&v"(xc), "=&v"(xd), "=&v"(xe), "=&v"(xf)
        : "v"(p));
    g[0] = u32x4{x0.x, x0.y, x1.x, x1.y}; g[1] = u32x4{x2.x, x2.y, x3.x, x3.y};
    g[2] = u32x4{x4.x, x4.y, x5.x, x5.y}; g[3] = u32x4{x6.x, x6.y, x7.x, x7.y};
    g[4] = u32x4{x8.x, x8.y, x9.x, x9.y}; g[5] = u32x4{xa.x, xa.y, xb.x, xb.y};
    g[6] = u32x4{xc.x, xc.y, xd.x, xd.y}; g[7] = u32x4{xe.x, xe.y, xf.x, xf.y};
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));  // the low half of a generic LDS address
}

// The same where only the wave's own accesses to LDS, and (all) everything it issued, have to be
// over.
__device__ __forceinline__ void wait_lds_and_sync(bool all) {
    if (all) __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

typedef uint32_t u32_any __attribute__((aligned(1)));

// The scale bytes of blocks kb .. kb + 3 (kb a multiple of 4) of a row of nb blocks: a load
// inside the row and, once it has landed, its part of them, 0 past the row's end.
__device__ __forceinline__ uint32_t mx_scales_load(const uint8_t* row, int kb, int nb) {
    if (nb >= 4) return *gld<u32_any>(row + min(kb, nb - 4));
    uint32_t w = 0;
    for (int t = 0; t < nb; ++t) w |= static_cast<uint32_t>(*gld<uint8_t>(row + t)) << (8 * t);
    return w;
}
__device__ __forceinline__ uint32_t mx_scales_take(uint32_t w, int kb, int nb) {
    const int past = nb >= 4 ? max(kb - (nb - 4), 0) : kb;
    return past >= 4 ? 0u : w >> (8 * past);
}

// A pointer that is the same in every lane, in scalar registers.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v)));
    const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v >> 32)));
    return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(hi) << 32 | lo);
}

// Position of 16-byte chunk c of row r in a stage of 128-byte rows: 16 consecutive rows
// read at one chunk (a fragment read's LDS cycle) then touch every bank once.
__device__ __forceinline__ int mx_swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

constexpr int kMxStep = 8;  // MX blocks (256 values) per contraction step

// The tile of a block: NW waves, WN along B's rows (64 each) and NW / WN along A's (32 IB
// each). acc: the wave's 32 IB x 64 part of C. LDS: five stages of A (the codes of kMxStep
// blocks of every row), two of B, two buffers of both operands' scales of two steps (4
// words, [word][row]).
template <int IB, int WN, int NW>
struct MxTile {
    static constexpr int kRowsA = 32 * IB * NW / WN;
    static constexpr int kRowsB = 64 * WN;
    static constexpr int kRows = kRowsA + kRowsB;
    static constexpr int kDepth = 5;
    static constexpr int kStageA = kRowsA * 128, kStageB = kRowsB * 128;
    static constexpr int kScales = 4 * kRows * 4;
    static constexpr int kLds = kDepth * kStageA + 2 * kStageB + 2 * kScales;
};

// acc += A B^T over the whole contraction. Codes (16-byte aligned) go by global_load_lds into
// LDS, so that nothing in the loop waits for their loads. A wave's transfers land in order, so
// one that fetched both operands could keep A, which comes from HBM, no further ahead than
// B, which every block reads from L2 and whose stages are the larger: half of the waves fetch
// A, four steps ahead (64 KB in flight per CU in the 128-row tile), the others B, one step
// ahead, and the scales of two steps at a time (8 bytes per row and step: fetched singly
// they cost the L2 as many requests as the codes). Rows of scales have
// any length and alignment, so these go through registers, loaded in the pair's even step
// and stored in its odd one, by waves that wait for their transfers at each barrier anyway
// (whole words by global_load_lds are no faster, and fragments of other rows read from global
// memory took 181 instead of 33 us for 32000 x 256 x 4096). Products put off behind the next barrier,
// beside the others' LDS reads, gave nothing here: 34 us.
// Lane half h takes blocks 4 h .. 4 h + 3 of a step: its codes are 64 contiguous bytes and
// its scales one word (the order of the contraction is free as long as both operands agree).
// Rows past an operand's end repeat its last one (they reach outputs that are not stored);
// past the contraction's end lanes multiply zero codes under scales of 1.
// Offsets within the tile's rows of an operand are 32 bits (kMxMaxK).
template <int IB, int WN, int NW>
__device__ __forceinline__ void mx4_accumulate(const MxOperand& a, const MxOperand& b, int64_t i0, int64_t j0,
                                               uint8_t* lds, f32x16 (&acc)[IB][2]) {
    using T = MxTile<IB, WN, NW>;
    constexpr int kHalf = NW / 2;  // waves of each kind
    constexpr int kA = T::kRowsA / 8 / kHalf, kB = T::kRowsB / 8 / kHalf;  // 1 KB transfers per wave: 8 rows each
    constexpr int kGroups = T::kRows / 64;  // of 64 rows, for the scales
    static_assert(kA * 8 * kHalf == T::kRowsA && kB * 8 * kHalf == T::kRowsB && T::kRowsA % 64 == 0, "whole transfers");
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;
    const bool fetch_a = wave < kHalf;
    const int fw = fetch_a ? wave : wave - kHalf;  // its number among its kind
    const int nb = a.nb;
    if (nb == 0) return;
    const uint32_t ra = uniform(static_cast<int>(min<int64_t>(a.rows - i0, T::kRowsA))) - 1;  // last valid row
    const uint32_t rb = uniform(static_cast<int>(min<int64_t>(b.rows - j0, T::kRowsB))) - 1;
    uint8_t* const ldsb = lds + T::kDepth * T::kStageA;
    uint8_t* const ldss = ldsb + 2 * T::kStageB;
    // The wave's i-th transfer of codes is transfer fw + i kHalf of its operand: 8 rows of 8
    // chunks. op: row offsets in blocks.
    constexpr int kMost = kA > kB ? kA : kB;
    const uint8_t* const cp = uniform(fetch_a ? a.codes + i0 * nb * 16 : b.codes + j0 * nb * 16);
    uint32_t op[kMost];
    static_assert(kHalf % 2 == 0, "the swizzle of a transfer's rows follows its wave");
    const int cblk = (lane & 7) ^ mx_swz(lane >> 3) ^ (fw & 1);  // mx_swz of the row
#pragma unroll
    for (int i = 0; i < kMost; ++i)
        op[i] = min<uint32_t>(8 * (fw + i * kHalf) + (lane >> 3), fetch_a ? ra : rb) * static_cast<uint32_t>(nb);
    auto codes = [&](int k, uint8_t* s, auto count) {
        const uint32_t kc = static_cast<uint32_t>(min(k * kMxStep + cblk, nb - 1));
#pragma unroll
        for (int i = 0; i < decltype(count)::value; ++i) dma16(cp + (op[i] + kc) * 16, s + (fw + i * kHalf) * 1024);
    };
    using CA = std::integral_constant<int, kA>;
    using CB = std::integral_constant<int, kB>;
    // Scales: group g is rows 64 g .. 64 g + 63 of [A; B], a word of four blocks per row and w.
    constexpr int kG = (kGroups + kHalf - 1) / kHalf;
    uint32_t sw4[kG][4];
    auto load_scales = [&](int pair) {
#pragma unroll
        for (int i = 0; i < kG; ++i) {
            const int g = fw + i * kHalf;
            if (g >= kGroups) break;
            const bool ga = g < T::kRowsA / 64;
            const uint8_t* p = (ga ? a.scales + i0 * nb : b.scales + j0 * nb) +
                               (ga ? min<uint32_t>(64 * g + lane, ra) : min<uint32_t>(64 * g - T::kRowsA + lane, rb)) *
                                   static_cast<uint32_t>(nb);
#pragma unroll
            for (int w = 0; w < 4; ++w) sw4[i][w] = mx_scales_load(p, 16 * pair + 4 * w, nb);
        }
    };
    auto store_scales = [&](int pair) {
#pragma unroll
        for (int i = 0; i < kG; ++i) {
            const int g = fw + i * kHalf;
            if (g >= kGroups) break;
            uint8_t* s = ldss + (pair & 1) * T::kScales + g * 256 + lane * 4;
#pragma unroll
            for (int w = 0; w < 4; ++w) *reinterpret_cast<uint32_t*>(s + w * T::kRows * 4) = mx_scales_take(sw4[i][w], 16 * pair + 4 * w, nb);
        }
    };
    const int wr = (wave / WN) * 32 * IB + (lane & 31), wc = (wave % WN) * 64 + (lane & 31);  // the lane's rows
    const int sw = mx_swz(lane & 31);  // rows 32 apart share it
    const uint32_t base = lds_addr(lds);
    auto multiply = [&](int k, int cur) {
        const uint32_t pa = base + cur * T::kStageA + wr * 128;
        const uint32_t pb = base + T::kDepth * T::kStageA + (k & 1) * T::kStageB + wc * 128;
        const uint32_t q = base + T::kDepth * T::kStageA + 2 * T::kStageB + ((k >> 1) & 1) * T::kScales +
                           (2 * (k & 1) + h) * (T::kRows * 4);
        const uint32_t qa = q + wr * 4, qb = q + (T::kRowsA + wc) * 4;
        uint32_t p[4], r[4], e[4];  // e: scales, A's one or two rows, B's two
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            p[t] = pa + (((4 * h + t) ^ sw) << 4);
            r[t] = pb + (((4 * h + t) ^ sw) << 4);
        }
        u32x4 ca[2][4], cb[2][4];
        lds_read_mx<IB>(p, r, qa, qb, ca, cb, e);
        if ((k + 1) * kMxStep > nb) {
            const int valid = nb - k * kMxStep - 4 * h;  // of the lane's blocks
#pragma unroll
            for (int jb = 0; jb < 2; ++jb)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t >= valid) cb[jb][t] = u32x4{0u, 0u, 0u, 0u};
            const uint32_t past = valid >= 4 ? 0u : valid <= 0 ? ~0u : ~0u << (8 * valid);
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = (e[i] & ~past) | (0x7f7f7f7fu & past);
        }
#pragma unroll
        for (int ib = 0; ib < IB; ++ib) {
#pragma unroll
            for (int jb = 0; jb < 2; ++jb) {
                acc[ib][jb] = mfma_mx4<0>(ca[ib][0], cb[jb][0], acc[ib][jb], e[ib], e[2 + jb]);
                acc[ib][jb] = mfma_mx4<1>(ca[ib][1], cb[jb][1], acc[ib][jb], e[ib], e[2 + jb]);
                acc[ib][jb] = mfma_mx4<2>(ca[ib][2], cb[jb][2], acc[ib][jb], e[ib], e[2 + jb]);
                acc[ib][jb] = mfma_mx4<3>(ca[ib][3], cb[jb][3], acc[ib][jb], e[ib], e[2 + jb]);
            }
        }
    };
    // Before step k's barrier a wave that fetches A waits until only steps k + 1 .. k + 3 are
    // outstanding, one that fetches B for all it issued. The stages that step k fills, A's of
    // step k + 4 and B's of k + 1, were last read in step k - 1, the scales' buffer in the
    // pair before. Past the end the last blocks are fetched
    // again, for equal counts.
    const int steps = (nb + kMxStep - 1) / kMxStep;
    if (fetch_a) {
#pragma unroll
        for (int k = 0; k < T::kDepth - 1; ++k) codes(k, lds + k * T::kStageA, CA{});
    } else {
        load_scales(0);
        store_scales(0);
        codes(0, ldsb, CB{});
    }
    // (Two loops: in one, the compiler lets the waves that fetch A wait for the others' registers.)
    int cur = 0;
    if (fetch_a) {
        for (int k = 0; k < steps; ++k) {
            wait_and_sync<3 * kA>();
            codes(k + T::kDepth - 1, lds + (cur == 0 ? T::kDepth - 1 : cur - 1) * T::kStageA, CA{});
            multiply(k, cur);
            cur = cur == T::kDepth - 1 ? 0 : cur + 1;
        }
    } else {
        for (int k = 0; k < steps; ++k) {
            wait_and_sync<0>();
            if (k & 1) store_scales((k + 1) >> 1);
            else if (nb >= 4) load_scales((k >> 1) + 1);
            codes(k + 1, ldsb + ((k + 1) & 1) * T::kStageB, CB{});
            multiply(k, cur);
            cur = cur == T::kDepth - 1 ? 0 : cur + 1;
        }
    }
    wait_and_sync<0>();  // transfers past the end have landed before the stages are reused
}

}  // namespace meo
