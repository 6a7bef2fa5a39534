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

// Four 16-byte LDS reads that have landed when it returns. In one asm block with their wait:
// before a plain read the compiler, which cannot tell what a transfer in flight writes, would
// wait for every transfer. The stage read has landed (the wait and barrier before).
__device__ __forceinline__ void lds_read4(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, u32x4* v) {
    u32x4 v0, v1, v2, v3;
    __asm__ volatile(
        "ds_read_b128 %0, %4\n\t"
        "ds_read_b128 %1, %5\n\t"
        "ds_read_b128 %2, %6\n\t"
        "ds_read_b128 %3, %7\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v0), "=&v"(v1), "=&v"(v2), "=&v"(v3)
        : "v"(a0), "v"(a1), "v"(a2), "v"(a3));
    v[0] = v0; v[1] = v1; v[2] = v2; v[3] = v3;
}

__device__ __forceinline__ void lds_read2(uint32_t a0, uint32_t a1, u32x4* v) {
    u32x4 v0, v1;
    __asm__ volatile(
        "ds_read_b128 %0, %2\n\t"
        "ds_read_b128 %1, %3\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v0), "=&v"(v1)
        : "v"(a0), "v"(a1));
    v[0] = v0; v[1] = v1;
}

__device__ __forceinline__ void lds_read_words(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t* w) {
    uint32_t w0, w1, w2, w3;
    __asm__ volatile(
        "ds_read_b32 %0, %4\n\t"
        "ds_read_b32 %1, %5\n\t"
        "ds_read_b32 %2, %6\n\t"
        "ds_read_b32 %3, %7\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(w0), "=&v"(w1), "=&v"(w2), "=&v"(w3)
        : "v"(a0), "v"(a1), "v"(a2), "v"(a3));
    w[0] = w0; w[1] = w1; w[2] = w2; w[3] = w3;
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));  // the low half of a generic LDS address
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
// each). acc: the wave's 32 IB x 64 part of C.
template <int IB, int WN, int NW>
struct MxTile {
    static constexpr int kRowsA = 32 * IB * NW / WN;
    static constexpr int kRowsB = 64 * WN;
    // one LDS stage: the codes of kMxStep blocks of every row of A, then of B, then the scales
    static constexpr int kScales = (kRowsA + kRowsB) * 128;
    static constexpr int kStage = kScales + (kRowsA + kRowsB) * 8;
};

// acc += A B^T over the whole contraction; nb a multiple of 4 and the scales 4-byte aligned.
// Codes and scales of both operands go by global_load_lds into one of three LDS stages, two
// steps ahead, so that nothing in the loop waits for a register load. Lane half h takes
// blocks 4 h .. 4 h + 3 of a step: its codes are 64 contiguous bytes and its scales one
// word (the order of the contraction is free as long as both operands agree).
// Rows past an operand's end repeat its last one (they reach outputs that are not stored);
// in a last step of 4 blocks, lane half 1 multiplies zero codes under scales of 1.
// Offsets within the tile's rows of an operand are 32 bits (kMxMaxK).
template <int IB, int WN, int NW>
__device__ __forceinline__ void mx4_accumulate(const MxOperand& a, const MxOperand& b, int64_t i0, int64_t j0,
                                               uint8_t* stages, f32x16 (&acc)[IB][2]) {
    using T = MxTile<IB, WN, NW>;
    constexpr int kA = T::kRowsA / 8 / NW, kB = T::kRowsB / 8 / NW;  // 1 KB transfers per wave: 8 rows each
    constexpr int kS = (T::kRowsA / 32 + NW - 1) / NW, kT = (T::kRowsB / 32 + NW - 1) / NW;  // 32 rows' scales each
    constexpr int kDma = kA + kB + kS + kT;
    static_assert(kA * 8 * NW == T::kRowsA && kB * 8 * NW == T::kRowsB, "whole transfers");
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;
    const int nb = a.nb;
    const uint8_t* const ac = uniform(a.codes + i0 * nb * 16);
    const uint8_t* const bc = uniform(b.codes + j0 * nb * 16);
    const uint8_t* const as = uniform(a.scales + i0 * nb);
    const uint8_t* const bs = uniform(b.scales + j0 * nb);
    const uint32_t ra = uniform(static_cast<int>(min<int64_t>(a.rows - i0, T::kRowsA))) - 1;  // last valid row
    const uint32_t rb = uniform(static_cast<int>(min<int64_t>(b.rows - j0, T::kRowsB))) - 1;
    // Row offsets (in blocks) of the wave's transfers; wave w's i-th is transfer w + i NW.
    uint32_t oa[kA], ob[kB], sa[kS], sb[kT];
    auto row_of = [&](int i) { return static_cast<uint32_t>(8 * (wave + i * NW) + (lane >> 3)); };
    const int chunk = (lane & 7) ^ mx_swz(lane >> 3);  // rows 8 j + (l >> 3): odd j flips one bit
    const int odd = wave & 1;                          // NW is even: the parity of j is the wave's
    const int cblk = chunk ^ odd;
#pragma unroll
    for (int i = 0; i < kA; ++i) oa[i] = min(row_of(i), ra) * static_cast<uint32_t>(nb);
#pragma unroll
    for (int i = 0; i < kB; ++i) ob[i] = min(row_of(i), rb) * static_cast<uint32_t>(nb);
    // scales: transfer j holds rows 32 j + (l >> 1), word l & 1; past the last transfer a wave
    // repeats one, so that every wave has the same number in flight
#pragma unroll
    for (int i = 0; i < kS; ++i)
        sa[i] = min<uint32_t>(32 * ((wave + i * NW) % (T::kRowsA / 32)) + (lane >> 1), ra) * static_cast<uint32_t>(nb);
#pragma unroll
    for (int i = 0; i < kT; ++i)
        sb[i] = min<uint32_t>(32 * ((wave + i * NW) % (T::kRowsB / 32)) + (lane >> 1), rb) * static_cast<uint32_t>(nb);
    auto stage = [&](int k0, uint8_t* s) {
        const uint32_t kc = static_cast<uint32_t>(min(k0 + cblk, nb - 1));
        const uint32_t ks = static_cast<uint32_t>(min(k0 + 4 * (lane & 1), nb - 4));
#pragma unroll
        for (int i = 0; i < kA; ++i) dma16(ac + (oa[i] + kc) * 16, s + (wave + i * NW) * 1024);
#pragma unroll
        for (int i = 0; i < kB; ++i) dma16(bc + (ob[i] + kc) * 16, s + T::kRowsA * 128 + (wave + i * NW) * 1024);
#pragma unroll
        for (int i = 0; i < kS; ++i) dma4(as + (sa[i] + ks), s + T::kScales + ((wave + i * NW) % (T::kRowsA / 32)) * 256);
#pragma unroll
        for (int i = 0; i < kT; ++i)
            dma4(bs + (sb[i] + ks), s + T::kScales + T::kRowsA * 8 + ((wave + i * NW) % (T::kRowsB / 32)) * 256);
    };
    const int wr = (wave / WN) * 32 * IB + (lane & 31), wc = (wave % WN) * 64 + (lane & 31);  // the lane's rows
    const int sw = mx_swz(lane & 31);  // rows 32 apart share it
    const uint32_t base = lds_addr(stages);
    auto multiply = [&](int k0, uint32_t s) {
        const uint32_t pa = s + wr * 128, pb = s + (T::kRowsA + wc) * 128;
        const uint32_t qa = s + T::kScales + wr * 8 + 4 * h, qb = s + T::kScales + (T::kRowsA + wc) * 8 + 4 * h;
        auto at = [&](int t) { return static_cast<uint32_t>(((4 * h + t) ^ sw) << 4); };
        uint32_t e[4];  // scales: A's one or two rows, B's two
        lds_read_words(qa, qa + (IB - 1) * 256, qb, qb + 256, e);
        u32x4 cb[2][4];
        lds_read4(pb + at(0), pb + at(1), pb + at(2), pb + at(3), cb[0]);
        lds_read4(pb + 4096 + at(0), pb + 4096 + at(1), pb + 4096 + at(2), pb + 4096 + at(3), cb[1]);
        if (k0 + kMxStep > nb) {
#pragma unroll
            for (int jb = 0; jb < 2; ++jb)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (h) cb[jb][t] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (h) e[i] = 0x7f7f7f7fu;
        }
#pragma unroll
        for (int ib = 0; ib < IB; ++ib) {
            u32x4 ca[4];
            lds_read4(pa + ib * 4096 + at(0), pa + ib * 4096 + at(1), pa + ib * 4096 + at(2), pa + ib * 4096 + at(3), ca);
#pragma unroll
            for (int jb = 0; jb < 2; ++jb) {
                acc[ib][jb] = mfma_mx4<0>(ca[0], cb[jb][0], acc[ib][jb], e[ib], e[2 + jb]);
                acc[ib][jb] = mfma_mx4<1>(ca[1], cb[jb][1], acc[ib][jb], e[ib], e[2 + jb]);
                acc[ib][jb] = mfma_mx4<2>(ca[2], cb[jb][2], acc[ib][jb], e[ib], e[2 + jb]);
                acc[ib][jb] = mfma_mx4<3>(ca[3], cb[jb][3], acc[ib][jb], e[ib], e[2 + jb]);
            }
        }
    };
    // Step k: its stage has landed once only the next stage's transfers are outstanding; the
    // stage that the new transfers fill was read in step k - 1, before the barrier.
    const int steps = (nb + kMxStep - 1) / kMxStep;
    stage(0, stages);
    stage(kMxStep, stages + T::kStage);
    int cur = 0;
    for (int k = 0; k < steps; ++k) {
        wait_and_sync<kDma>();
        const int next = cur == 0 ? 2 : cur - 1;
        stage((k + 2) * kMxStep, stages + next * T::kStage);
        multiply(k * kMxStep, base + cur * T::kStage);
        cur = cur == 2 ? 0 : cur + 1;
    }
    wait_and_sync<0>();  // transfers past the end have landed before the stages are reused
}

// The same product for any nb and alignment, every fragment read as it lies: 4 waves, 2 along
// each side, 32 x 64 each. A lane's block past the contraction's end is zero codes.
__device__ __forceinline__ void mx4_accumulate_any(const MxOperand& a, const MxOperand& b, int64_t i0, int64_t j0,
                                                   f32x16 (&acc)[1][2]) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;
    const int nb = a.nb;
    const int64_t ra = min<int64_t>(i0 + (wave >> 1) * 32 + (lane & 31), a.rows - 1) * nb;
    int64_t rb[2];
#pragma unroll
    for (int jb = 0; jb < 2; ++jb) rb[jb] = min<int64_t>(j0 + (wave & 1) * 64 + jb * 32 + (lane & 31), b.rows - 1) * nb;
    for (int k = 0; k < nb; k += 4) {
        u32x4 ca[2], cb[2][2];
        uint32_t ea[2], eb[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int kb = k + 2 * t + h;
            const bool in = kb < nb;
            ca[t] = u32x4{0u, 0u, 0u, 0u};
            ea[t] = 127;
            if (in) {
                ca[t] = *gld<u32x4>(a.codes + (ra + kb) * 16);
                ea[t] = *gld<uint8_t>(a.scales + ra + kb);
            }
#pragma unroll
            for (int jb = 0; jb < 2; ++jb) {
                cb[t][jb] = u32x4{0u, 0u, 0u, 0u};
                eb[t][jb] = 127;
                if (in) {
                    cb[t][jb] = *gld<u32x4>(b.codes + (rb[jb] + kb) * 16);
                    eb[t][jb] = *gld<uint8_t>(b.scales + rb[jb] + kb);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int jb = 0; jb < 2; ++jb) acc[0][jb] = mfma_mx4<0>(ca[t], cb[t][jb], acc[0][jb], ea[t], eb[t][jb]);
    }
}

}  // namespace meo
