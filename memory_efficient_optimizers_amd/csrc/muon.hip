// Orthogonalization of matrices by Newton-Schulz steps, and the Muon step around it.
//
// With X0 = U / max(|U|, eps) (Frobenius norm; the shorter side as rows, m <= n), each step is
//     A = X X^T,   X <- a X + (b A + c A^2) X.
// The products run on fp16 matrix cores with fp32 sums. What is rounded to fp16 (relative 2^-11,
// bf16 would be 2^-8 at the same rate) and why that is enough:
//   * X as an operand. The linear term, which alone carries the small singular values, takes X
//     as the sum of two fp16 parts (hi + lo, 22 bits): with hi alone 300 x 300 of rank 8 plus 1%
//     noise came out 2.3e-2 off, so 2.6e-4. B takes hi only; the diagonal of B takes lo as well
//     as far as the row's norm is that of a finished matrix (B_ii min(1, d_i^2)). Where singular
//     values are all near 1 that is most of what B lo is (gaussian 256 x 256: 9.6e-4 off, without
//     it 1.3e-3); where few are, it would add a noise of full rank (100 x 100, rank 1 plus 1e-4
//     noise: 4e-3 with B_ii lo whole, 5e-4 so).
//   * A and B = b A + c A^2 off their diagonals. The diagonals, which near the end are most of
//     A, are held in fp32 (d, and q = a + B_ii) and enter by row: (A^2)_ij = (O^2)_ij +
//     O_ij (d_i + d_j) off the diagonal, with O the rest of A. That halves the error of
//     well-conditioned matrices (gaussian 256 x 256: 1.7e-3 to 9.6e-4). d is that of both parts of
//     X: the product has the hi parts', and whoever stores X adds up what the lo parts make of it
//     (mu_fix). In rows with few entries of any size hi's roundings do not average out (identity of
//     343 rows: 8.4e-3 off without, 1.9e-3 so).
// What is left is two roundings of every off-diagonal product a step, 1e-3 of the result where they
// average out, more where they do not (meo.h has the figures).
// Values are held times powers of two, so that they are normal fp16 numbers far down: X times 2^12
// (muon.h), O and B times 2^8.
// Matrices with few rows are worked on in muon_small.hip.
#include "muon_device.h"

namespace meo {

namespace {

struct MuNone {};

// ----------------------------------------------------------------------------- the caller's tensors

// The momentum's update and the sum of squares of the direction, in fp64 (the squares of any
// fp32 value neither vanish nor overflow). One block per part of a matrix; parts are joined by
// every block of the next pass, in order. Bound by memory: 12.6 M values, all fp32, in 27 us (151 MB at
// 5.6 TB/s).
template <int N>
__global__ __launch_bounds__(kMuThreads) void k_mu_momentum(MuListOf<MuTensor, N> l, MuStepArgs a) {
    __shared__ double sums[kMuThreads / 64];
    const int k = mu_find(l, blockIdx.x);
    const MuTensor& t = l.d[k];
    const uint32_t item = mu_item(l, k, blockIdx.x);
    const int b = static_cast<int>(item / t.parts), part = static_cast<int>(item % t.parts);
    const int64_t size = static_cast<int64_t>(t.rows) * t.cols, base = b * size;
    const int64_t i0 = part * t.tiles_per_part * kMuPart, i1 = min(size, i0 + t.tiles_per_part * kMuPart);
    if (part == 0 && mu_few(min(t.rows, t.cols), max(t.rows, t.cols)) == 0) {  // for k_mu_scatter's sums
        int32_t* const e = reinterpret_cast<int32_t*>(t.ws + b * t.stride + MuPlace(t.mp, t.np, 1).low(0, t.mp));
        for (int i = threadIdx.x; i < t.mp; i += kMuThreads) *gst<int32_t>(e + i) = 0;
    }
    double sum = 0.0;
    for (int64_t i = i0 + threadIdx.x * kVec; i - threadIdx.x * kVec < i1; i += kMuThreads * kVec) {
        const int valid = clamp_valid(i1 - i);
        float u[kVec];
        mu_take8(t, a, b, base, i, valid, u);
#pragma unroll
        for (int e = 0; e < kVec; ++e) sum += static_cast<double>(u[e]) * static_cast<double>(u[e]);
    }
    const double s = block_sum_d(sum, sums);
    if (threadIdx.x == 0) *gst<double>(t.norm + item) = s;
}

// The factor of matrix b, from the sums of its parts.
__device__ __forceinline__ double mu_factor(const MuTensor& t, int b, double eps, double* sums) {
    const double* p = t.norm + static_cast<int64_t>(b) * t.parts;
    double s = 0.0;
    for (int i = threadIdx.x; i < t.parts; i += kMuThreads) s += *gld<double>(p + i);
    s = block_sum_d(s, sums);
    if (threadIdx.x == 0) sums[kMuThreads / 64] = mu_factor_of(s, eps);
    __syncthreads();
    return sums[kMuThreads / 64];
}

// The directions, scaled, into the workspace: a square tile of the padded matrix per block,
// zeros outside the matrix. A tall matrix is transposed on the way, through LDS. Bound by memory: 12.6 M
// values in 27.5 us (gradient and momentum again, two parts out: 151 MB at 5.5 TB/s); the direction is formed
// twice, since keeping it between the passes would move more. The low parts' sums for A's diagonal are
// 1 to 1.5 us of it.
template <int N>
__global__ __launch_bounds__(kMuThreads) void k_mu_scatter(MuListOf<MuTensor, N> l, MuStepArgs a) {
    __shared__ double sums[kMuThreads / 64 + 1];
    __shared__ float tile[kMuTile][kMuTile + 1];
    const int k = mu_find(l, blockIdx.x);
    const MuTensor& t = l.d[k];
    const uint32_t item = mu_item(l, k, blockIdx.x);
    const uint32_t tn = t.np / kMuTile, per = tn * (t.mp / kMuTile);
    const int b = static_cast<int>(item / per);
    const int r0 = static_cast<int>(item % per / tn) * kMuTile, c0 = static_cast<int>(item % per % tn) * kMuTile;
    const double f = mu_factor(t, b, a.eps, sums);
    const MuPlace at(t.mp, t.np, 1);
    uint8_t* const w = t.ws + b * t.stride;
    // the piece of row r that a thread stores: in two parts, and what the low ones add to the diagonal
    auto store = [&](int r, const float* v) {
        const int q = threadIdx.x & 7;
        uint32_t h[kVec], o[kVec];
        float low = 0.0f;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            mu_split(v[e], h[e], o[e]);
            const float hi = mu_half(u32x2{h[e], 0u}, 0);
            low = fmaf(v[e] - hi, hi, low);
        }
        const int64_t i = mu_at(r0 + r, c0 + q * kVec, t.np) * 2;
        *gst<u32x4>(w + at.hi(0) + i) = u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
        *gst<u32x4>(w + at.lo + i) = u32x4{o[0] | o[1] << 16, o[2] | o[3] << 16, o[4] | o[5] << 16, o[6] | o[7] << 16};
        uint32_t sum = mu_fix(low);
#pragma unroll
        for (int k = 1; k < 8; k *= 2) sum += __shfl_xor(sum, k);
        if (q == 0 && sum != 0) mu_fixed_add(reinterpret_cast<int32_t*>(w + at.low(0, t.mp)) + r0 + r, sum);
    };
    const int64_t size = static_cast<int64_t>(t.rows) * t.cols;
    const int s0 = t.tall ? c0 : r0, z0 = t.tall ? r0 : c0;  // the source's first row and column
    const int q = threadIdx.x & 7;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int r = (threadIdx.x >> 3) + 32 * p, row = s0 + r, col = z0 + q * kVec;
        const int valid = row < t.rows ? clamp_valid(static_cast<int64_t>(t.cols) - col) : 0;
        float u[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) u[e] = 0.0f;
        if (valid > 0) {
            const int64_t i = static_cast<int64_t>(row) * t.cols + col;
            float g[kVec], m[kVec];
            // (a row's piece, so that row and column need no division)
            load_any8(t.g, (static_cast<int64_t>(b) * t.rows + row) * t.ldg + col, valid, t.gbf16, g);
            if (t.m) {
                mu_load_m(t, b * size + i, valid, m);
                mu_direction(a, g, m, u);
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) u[e] = g[e];
            }
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) u[e] = e < valid ? static_cast<float>(u[e] * f) : 0.0f;
        if (!t.tall) {
            store(r, u);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) tile[r][q * kVec + e] = u[e];
        }
    }
    if (!t.tall) return;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int r = (threadIdx.x >> 3) + 32 * p;
        float v[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = tile[q * kVec + e][r];
        store(r, v);
    }
}

// ----------------------------------------------------------------------------- products

// A T x T tile of a product of NW waves, WM along P's rows and NW / WM along Q's: 32 MB x 32 NB
// values each. LDS: a ring of kDepth stages of 32 values of the contraction of both operands.
// What bounds the products is the way from L2 to LDS (256 x 256): with two stages of 64 values (64 KB in
// flight per CU) a step took 1.16 us without any multiplication, and 0.85 us is what its
// multiplications take; with five of 32 there are 128 KB in flight.
template <int T, int WM, int NW>
struct MuTileOf {
    static constexpr int kT = T, kWM = WM, kWN = NW / WM, kNW = NW;
    static constexpr int MB = T / 32 / WM, NB = T / 32 / (NW / WM);
    static constexpr int kDepth = T == 192 ? 6 : 5;
    static constexpr int kOperand = T * 64;  // bytes of one operand's stage
    static constexpr int kStage = 2 * kOperand;
    static constexpr int kLds = kDepth * kStage;
    static constexpr int kBlocks = T >= 192 ? 1 : T == 128 ? 2 : 4;  // per CU
};
template <int F> struct MuTiles;
template <> struct MuTiles<kMuSmall> : MuTileOf<64, 2, 4> {};
template <> struct MuTiles<kMuMedium> : MuTileOf<128, 2, 4> {};
template <> struct MuTiles<kMuThreeQuarters> : MuTileOf<192, 2, 4> {};
template <> struct MuTiles<kMuLarge> : MuTileOf<256, 2, 4> {};

// 16 bytes per lane from base + offset into LDS, lane l at dst + 16 l. In asm, because before
// every LDS read the compiler would wait for all of its own transfers (it cannot tell what they
// write); it writes no vector registers, and mu_arrive waits for it. (m0 is the compiler's own, which it warns
// of; told so, it keeps no value there over a transfer.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void mu_fetch16(const uint8_t* base, uint32_t offset, uint32_t dst) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst), "v"(offset), "s"(base) : "m0");
}
#pragma clang diagnostic pop
// At most N of the wave's transfers are outstanding; then the same for the block.
template <int N>
__device__ __forceinline__ void mu_arrive() {
    __asm__ volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

// acc += the tile's product over `steps` steps of 32 values, from step k0 on: P's rows i0 .. (TR:
// its columns, the contraction runs down its rows), Q's rows j0 .., matrices of cols_p and cols_q
// columns. Blocks past the operands' end (rows_p and rows_q: columns_p, TR) repeat the last ones;
// they reach values that are not stored.
// A step's operands go straight into their stage, kDepth - 1 steps ahead. The fragments of 16
// values of the contraction are read while the ones before are multiplied; the barrier of a step
// comes before its last multiplication, when the next stage has landed: so one wave per SIMD (a
// large tile) keeps its matrix core busy. The barrier does not wait for the wave's own LDS reads: the
// stage that is overwritten behind it is the one of the step before (256 x 256 tiles of 4096 x 4096
// without transfers: X' 115 us with that wait, 98 without). Past the end the last step is fetched
// again, for equal counts of transfers.
template <class M, bool TR>
__device__ __forceinline__ void mu_accumulate(const uint16_t* P, int cols_p, int rows_p, const uint16_t* Q, int cols_q, int rows_q,
                                              int i0, int j0, int k0, int steps, uint8_t* lds, f32x16 (&acc)[M::MB][M::NB]) {
    constexpr int T = M::kT, NW = M::kNW, kCount = T / 16 / NW, kAll = 2 * kCount;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;
    const uint32_t base = uniform(static_cast<int>(lds_addr(lds)));
    steps = uniform(steps);  // (the transfers' addresses and counts stay in scalar registers)
    cols_p = uniform(cols_p);
    // Transfers: 1 KB each, 16 rows of a block, kCount of either operand per wave. In LDS a row's
    // chunk c (16 bytes) lies at position c ^ (row >> 2 & 3): 16 rows read at one chunk then touch
    // every bank once. TR: as they come; a transposed read's 8 rows of 64 bytes do so too.
    uint32_t op[kCount], oq[kCount];
    const uint32_t chunk = ((lane & 3) ^ ((lane >> 4) & 3)) * 16;
    const uint8_t* cp = uniform(reinterpret_cast<const uint8_t*>(P) +
                                (TR ? static_cast<int64_t>(k0 >> 1) * cols_p * 128 + (k0 & 1) * 2048 + static_cast<int64_t>(i0) * 128
                                    : static_cast<int64_t>(i0) * cols_p * 2 + static_cast<int64_t>(k0) * 4096));
    const uint8_t* cq = uniform(reinterpret_cast<const uint8_t*>(Q) + static_cast<int64_t>(j0) * cols_q * 2 + static_cast<int64_t>(k0) * 4096);
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
        const int t = wave + i * NW;  // 16 rows t of the tile; TR: half t & 1 of a block's 32 rows
        oq[i] = static_cast<uint32_t>(min(t >> 2, (rows_q - j0) / 64 - 1)) * static_cast<uint32_t>(cols_q) * 128u +
                (16 * (t & 3) + (lane >> 2)) * 64u + chunk;
        op[i] = TR ? static_cast<uint32_t>(min(t >> 1, (rows_p - i0) / 32 - 1)) * 4096u + (t & 1) * 1024u + lane * 16u
                   : static_cast<uint32_t>(min(t >> 2, (rows_p - i0) / 64 - 1)) * static_cast<uint32_t>(cols_p) * 128u +
                         (16 * (t & 3) + (lane >> 2)) * 64u + chunk;
    }
    // from one step of P to the next: TR: the other half of a row of blocks, or the next row
    const int64_t step_p = TR ? static_cast<int64_t>(cols_p) * 128 - 2048 : 4096;
    // The i-th transfer of an operand's next step.
    int next_p = 1, next_q = 1;
    auto fetch_p = [&](uint32_t stage, int i) {
        mu_fetch16(cp, op[i], base + stage + (wave + i * NW) * 1024);
        if (i == kCount - 1) {
            cp += next_p >= steps ? 0 : TR && (next_p + k0) % 2 != 0 ? 2048 : step_p;
            ++next_p;
        }
    };
    auto fetch_q = [&](uint32_t stage, int i) {
        mu_fetch16(cq, oq[i], base + stage + M::kOperand + (wave + i * NW) * 1024);
        if (i == kCount - 1) cq += next_q++ < steps ? 4096 : 0;
    };
    // fragments: the lane's addresses in the first stage
    const int wm = wave / M::kWN, wn = wave % M::kWN;
    uint32_t pa[2], qa[2];
    const int sw = (lane >> 2) & 3;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        qa[s] = base + M::kOperand + (wn * 32 * M::NB + (lane & 31)) * 64 + (((2 * s + h) ^ sw) << 4);
        pa[s] = base + (wm * 32 * M::MB + (lane & 31)) * 64 + (((2 * s + h) ^ sw) << 4);
    }
    // TR: 16 lanes read 4 rows of 16 columns; columns 16 on in the next 16 lanes, rows 8 on in the other half
    const uint32_t pt = base + wm * M::MB * 2048 + (8 * h + ((lane >> 2) & 3)) * 64 + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
    struct Frags {
        u32x4 p[M::MB], q[M::NB];
    };
    auto read_q = [&](Frags& f, uint32_t stage, int s, int j) { f.q[j] = mu_lds(qa[s] + stage + j * 2048); };
    auto read_p = [&](Frags& f, uint32_t stage, int s, int i) {
        if constexpr (TR) {
            const uint32_t a0 = pt + stage + i * 2048 + s * 1024;
            const u32x2 a = mu_lds_tr(a0), b = mu_lds_tr(a0 + 256);
            f.p[i] = u32x4{a.x, a.y, b.x, b.y};
        } else {
            f.p[i] = mu_lds(pa[s] + stage + i * 2048);
        }
    };
    // Half a step: the products of `now`, a row of them at a time, between them the reads of
    // `next` (all of Q's fragments first, which its first row needs) and, after each row, a
    // transfer: in a burst after the barrier they held up the products behind them (a wave
    // issues in order; 256 x 256 tiles, 64 values: 1.20 us in bursts).
    auto half = [&](const Frags& now, Frags& next, uint32_t stage, int s, auto fetch) {
        constexpr int kReads = M::NB + M::MB;
#pragma unroll
        for (int i = 0; i < M::MB; ++i) {
#pragma unroll
            for (int e = i * kReads / M::MB; e < (i + 1) * kReads / M::MB; ++e)
                if (e < M::NB) read_q(next, stage, s, e);
                else read_p(next, stage, s, e - M::NB);
#pragma unroll
            for (int j = 0; j < M::NB; ++j) acc[i][j] = mfma_f16(now.p[i], now.q[j], acc[i][j]);
#pragma unroll
            for (int j = 0; j < M::NB; ++j) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
                __builtin_amdgcn_sched_group_barrier(0x100, TR ? 2 : 1, 0);  // LDS reads
            }
            __builtin_amdgcn_sched_barrier(0);
            fetch(i);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    static_assert(kCount == M::MB, "a transfer of either operand per row of products");
    if constexpr (M::MB == 1 && M::NB == 1) {
        // A tile of 64 has two products a step and wave, too few to hide the reads of half a step: a step's
        // fragments are read a whole step ahead (six tiles of 2112 values 11.0 to 10.3 us, 272 of 4096 25.4
        // to 23.3, many short ones 1 to 3% less).
        Frags a[2], b[2];
        auto fetch = [&](uint32_t stage) {
            fetch_p(stage, 0);
            fetch_q(stage, 0);
        };
        auto read = [&](Frags (&to)[2], uint32_t stage) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                read_q(to[s], stage, s, 0);
                read_p(to[s], stage, s, 0);
            }
        };
        uint32_t stage = 0, free = (M::kDepth - 1) * M::kStage;  // the next step's, and the one left last
        auto after = [](uint32_t s) { return s == (M::kDepth - 1) * M::kStage ? 0u : s + M::kStage; };
        auto step = [&](const Frags (&now)[2], Frags (&next)[2]) {
            mu_arrive<(M::kDepth - 3) * kAll>();
            stage = after(stage);
            read(next, stage);  // (past the last step: of no use, in bounds)
            __builtin_amdgcn_sched_barrier(0);
            fetch(free);
            free = after(free);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < 2; ++s) acc[0][0] = mfma_f16(now[s].p[0], now[s].q[0], acc[0][0]);
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int k = 0; k < M::kDepth - 1; ++k) fetch(k * M::kStage);
        mu_arrive<(M::kDepth - 2) * kAll>();
        read(a, 0);
        for (int k = 0; k < steps; k += 2) {  // (an even number)
            step(a, b);
            step(b, a);
        }
        wait_and_sync<0>();
        return;
    }
    Frags f, g;
#pragma unroll
    for (int k = 0; k < M::kDepth - 1; ++k) {
#pragma unroll
        for (int i = 0; i < kCount; ++i) fetch_p(k * M::kStage, i);
        if (k == M::kDepth - 2) break;
#pragma unroll
        for (int i = 0; i < kCount; ++i) fetch_q(k * M::kStage, i);
    }
    mu_arrive<(M::kDepth - 3) * kAll + kCount>();
#pragma unroll
    for (int j = 0; j < M::NB; ++j) read_q(f, 0, 0, j);
#pragma unroll
    for (int i = 0; i < M::MB; ++i) read_p(f, 0, 0, i);
    // `last`: the stage of the step fetched last; after a step's barrier it is the one that the step
    // before has left (its fragments were multiplied before the barrier, so nobody reads it).
    uint32_t stage = 0, last = (M::kDepth - 2) * M::kStage;
    auto after = [](uint32_t s) { return s == (M::kDepth - 1) * M::kStage ? 0u : s + M::kStage; };
    for (int k = 0; k < steps; ++k) {
        half(f, g, stage, 1, [&](int i) { fetch_q(last, i); });
        mu_arrive<(M::kDepth - 3) * kAll>();
        last = after(last);
        stage = after(stage);
        // (past the last step: read of no use, in bounds)
        half(g, f, stage, 0, [&](int i) { fetch_p(last, i); });
    }
    wait_and_sync<0>();  // transfers past the end have landed before the stages are reused
}

// Blocks go round-robin to the 8 XCDs: consecutive tiles of a tensor on one XCD. (Of the whole list,
// some XCDs had all tiles of the tensors with a long contraction.)
__device__ __forceinline__ uint32_t mu_swizzle(uint32_t id, uint32_t n) {
    constexpr uint32_t kX = 8;
    const uint32_t x = id % kX, q = n / kX, r = n % kX;
    return x * q + min(x, r) + id / kX;
}

constexpr int kMuGroup = 4;  // tile rows that consecutive tiles share columns of

// Tile t of the upper triangle (i <= j) of n x n tiles, kMuGroup rows at a time, by columns.
__device__ __forceinline__ void mu_triangle(uint32_t t, int n, int& i, int& j) {
    int r = 0;
    while (true) {
        const int rows = min(kMuGroup, n - r);
        const uint32_t count = rows * (rows + 1) / 2 + rows * (n - r - rows);
        if (t < count) {
            j = r;
            while (true) {
                const uint32_t c = min(rows, j - r + 1);
                if (t < c) break;
                t -= c;
                ++j;
            }
            i = r + t;
            return;
        }
        t -= count;
        r += kMuGroup;
    }
}

template <class M>
__device__ __forceinline__ void mu_zero(f32x16 (&acc)[M::MB][M::NB]) {
#pragma unroll
    for (int i = 0; i < M::MB; ++i)
#pragma unroll
        for (int j = 0; j < M::NB; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
}

// What follows the contraction works on the wave's part of the tile in rounds of 32 columns j, in
// the wave's own share of LDS, without barriers: fp16 values [32 j][kI i], where an accumulator
// finds its four rows i of a column as 8 bytes, a row of memory goes by 16 bytes per lane
// and, turned round, a transposed read has 8 columns of a row i. (One wave per SIMD issues an
// instruction in 4 cycles, so this is kept to a few per value: with fp32 values through LDS
// and a comparison each, it took 20 us of a 4096 x 4096 product's 104.)
template <class M>
struct MuRound {
    static constexpr int kI = 32 * M::MB;
    static constexpr int kP = M::MB == 3 ? 128 : kI;  // values from column to column in LDS: a power of two
    static constexpr int kIters = kI / 16;  // 1 KB accesses to memory per round: 16 columns of a block each
    static constexpr int kBytes = 32 * kP * 2;
    typedef __attribute__((address_space(3))) u32x2 L2;
    typedef __attribute__((address_space(3))) u32x4 L4;
    typedef __attribute__((address_space(3))) f32x4 F4;
    uint32_t base;  // of the wave's share
    int lane, ib, jb, j, h;  // first row and column of the wave's part; the lane's accumulator column and half

    __device__ MuRound(uint8_t* lds, int i0, int j0, int share) {
        const int wave = uniform(threadIdx.x >> 6);
        lane = threadIdx.x & 63;
        base = uniform(static_cast<int>(lds_addr(lds))) + wave * share;
        ib = i0 + wave / M::kWN * kI;
        jb = j0 + wave % M::kWN * 32 * M::NB;
        j = lane & 31;
        h = lane >> 5;
    }
    // Bytes of chunk c (4 values) of column j: columns that an access touches at one chunk lie on
    // different banks; columns 16 apart in the two halves of 16 bytes.
    __device__ static uint32_t at(int j, int c) {
        constexpr int kPer = 128 / kP;  // columns per 256 bytes
        return j * (kP * 2) + ((c ^ 2 * (j / kPer & (kP / 8 - 1)) ^ (j >> 4 & 1)) << 3);
    }
    __device__ u32x2 get(int array, int ii, int v) const {
        return *(const L2*)static_cast<uintptr_t>(base + array * kBytes + at(j, 8 * ii + 2 * v + h));
    }
    __device__ void put(int array, int ii, int v, u32x2 w) const {
        *(L2*)static_cast<uintptr_t>(base + array * kBytes + at(j, 8 * ii + 2 * v + h)) = w;
    }
    // The lane's 16 bytes of access e: column row(e) (a row of memory), rows col(e) .. + 7.
    __device__ int row(int e) const { return 16 * (e & 1) + (lane >> 2); }
    __device__ int col(int e) const { return 32 * (e >> 1) + (lane & 3) * 8; }
    __device__ uint32_t line(int array, int e) const {  // (their halves are swapped from column 16 on)
        return base + array * kBytes + (at(row(e), col(e) / 4) & ~8u);
    }
    __device__ u32x4 get_line(int array, int e) const {
        const u32x4 w = *(const L4*)static_cast<uintptr_t>(line(array, e));
        return e & 1 ? u32x4{w.z, w.w, w.x, w.y} : w;
    }
    __device__ void put_line(int array, int e, u32x4 w) const {
        *(L4*)static_cast<uintptr_t>(line(array, e)) = e & 1 ? u32x4{w.z, w.w, w.x, w.y} : w;
    }
    // Where they are in a matrix of `cols` columns in the workspace, of the round from column j0 on:
    // a kilobyte, and whether the matrix has it.
    __device__ uint16_t* place(uint16_t* s, int cols, int j0, int e) const {
        const int64_t at = mu_rows(j0 + 16 * (e & 1), cols) + static_cast<int64_t>(ib + 32 * (e >> 1)) * 64;
        return const_cast<uint16_t*>(reinterpret_cast<const uint16_t*>(uniform(reinterpret_cast<const uint8_t*>(s + at)))) + lane * 8;
    }
    __device__ bool has(int rows, int cols, int j0, int e) const { return j0 < rows && ib + 32 * (e >> 1) < cols; }
    // 8 columns, from turned_col() on, of row turned_row(t), t < kI / 16.
    __device__ int turned_row(int t) const { return 16 * t + (lane & 15); }
    __device__ int turned_col() const { return lane >> 4 << 3; }
    __device__ u32x4 get_turned(int t) const {
        const int r = (lane >> 4) * 8 + (lane >> 2 & 3), c = 4 * t + (lane & 3);
        const u32x2 a = mu_lds_tr(base + at(r, c)), b = mu_lds_tr(base + at(r + 4, c));
        return u32x4{a.x, a.y, b.x, b.y};
    }
    // fp32 values in chunks of 4, [32 j][kP i], at an offset of the share.
    __device__ uint32_t at32(int j, int c) const { return j * (kP * 4) + ((c ^ (j & (kP / 4 - 1))) << 4); }
    __device__ void put32(uint32_t offset, int ii, int v, f32x4 w) const {
        *(F4*)static_cast<uintptr_t>(base + offset + at32(j, 8 * ii + 2 * v + h)) = w;
    }
    __device__ f32x4 get32(uint32_t offset, int j, int c) const {
        return *(const F4*)static_cast<uintptr_t>(base + offset + at32(j, c));
    }
    __device__ float get32_value(uint32_t offset, int j, int i) const {
        return *(const __attribute__((address_space(3))) float*)static_cast<uintptr_t>(base + offset + at32(j, i >> 2) + (i & 3) * 4);
    }
};

// A finished round of a symmetric product of mp rows: columns j0 .. and, turned round, rows j0 ...
template <class M>
__device__ __forceinline__ void mu_store_sym(const MuRound<M>& r, uint16_t* s, int mp, int j0) {
    using R = MuRound<M>;
#pragma unroll
    for (int e = 0; e < R::kIters; ++e)
        if (r.has(mp, mp, j0, e)) *gst<u32x4>(r.place(s, mp, j0, e)) = r.get_line(0, e);
#pragma unroll
    for (int t = 0; t < R::kI / 16; ++t) {
        const int i = r.ib + 16 * t;
        if (i >= mp || j0 >= mp) continue;
        const int64_t at = mu_rows(i, mp) + static_cast<int64_t>(j0) * 64;  // 16 rows of a block: a kilobyte
        uint8_t* const p = const_cast<uint8_t*>(uniform(reinterpret_cast<const uint8_t*>(s + at)));
        *gst<u32x4>(p + (r.lane & 15) * 64 + (r.lane >> 4) * 16) = r.get_turned(t);
    }
}

// A = X X^T: tiles of the upper triangle, stored both ways round (sums over k in the same
// order, so A is symmetric to the bit), 2^8 times; the diagonal in fp32. A contraction in parts
// (small tiles only) leaves each part's fp32 sums for k_mu_join. Median times: 4096 x 4096 76 to 80 us
// (192-tiles, 253 of them; 65% of the matrix units' cycles, the library's product with twice the work
// 102 us), 4096 x 11008 182 us; 256 x 512 5.9 us, ten tiles' latency. The low parts' sums are 1 to 1.5 us of
// a large tile.
template <int F, int N>
__global__ __launch_bounds__(kMuTileThreads, MuTiles<F>::kBlocks) void k_mu_gram(MuListOf<MuMatrix, N> l, int src) {
    using M = MuTiles<F>;
    __shared__ __attribute__((aligned(16))) uint8_t lds[M::kLds];
    const int k = mu_find(l, blockIdx.x);
    const MuMatrix& m = l.d[k];
    const int nt = (m.mp + M::kT - 1) / M::kT;
    const uint32_t per = nt * (nt + 1) / 2;
    uint32_t t = mu_swizzle(mu_item(l, k, blockIdx.x), per * m.parts * m.batch);
    const uint32_t b = t / (per * m.parts);
    t -= b * (per * m.parts);
    const int part = static_cast<int>(t / per);
    int ti, tj;
    mu_triangle(t % per, nt, ti, tj);
    ti = uniform(ti);
    tj = uniform(tj);
    const MuPlace at(m.mp, m.np, m.parts);
    uint8_t* const w = m.ws + b * m.stride;
    const uint16_t* x = reinterpret_cast<const uint16_t*>(w + at.hi(src));
    const int k0 = part * m.steps * 2, steps = min(m.steps, m.np / 64 - part * m.steps);
    const MuRound<M> r(lds, ti * M::kT, tj * M::kT, MuRound<M>::kBytes);
    // What the low parts add to the diagonal, of the lane's columns (read here, by all tiles: the product
    // hides it; behind a branch for tiles on the diagonal the compiler waited for it there).
    int32_t low[M::NB];
#pragma unroll
    for (int jj = 0; jj < M::NB; ++jj)
        low[jj] = *gld<int32_t>(reinterpret_cast<const int32_t*>(w + at.low(src, m.mp)) + min(r.jb + 32 * jj + r.j, m.mp - 1));
    f32x16 acc[M::MB][M::NB];
    mu_zero<M>(acc);
    mu_accumulate<M, false>(x, m.np, m.mp, x, m.np, m.mp, ti * M::kT, tj * M::kT, k0, 2 * steps, lds, acc);
    if (r.ib == r.jb && part == 0) {  // k_mu_apply adds up the next ones
        int32_t* const next = reinterpret_cast<int32_t*>(w + at.low(src ^ 1, m.mp));
        for (int j = r.lane; j < 32 * M::NB; j += 64)
            if (r.jb + j < m.mp) *gst<int32_t>(next + r.jb + j) = 0;
    }
    if (F == kMuSmall && m.parts > 1) {
        float* const o = reinterpret_cast<float*>(w + at.part) + static_cast<int64_t>(part) * m.mp * m.mp;
#pragma unroll
        for (int jj = 0; jj < M::NB; ++jj)
#pragma unroll
            for (int ii = 0; ii < M::MB; ++ii)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int i = r.ib + 32 * ii + 8 * v + 4 * r.h, j = r.jb + 32 * jj + r.j;
                    const f32x16& a = acc[ii][jj];
                    f32x4 c = {a[4 * v], a[4 * v + 1], a[4 * v + 2], a[4 * v + 3]};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (i + e == j && part == 0) c[e] += mu_unfix(low[jj]);
                    if (i < m.mp && j < m.mp) *gst<f32x4>(o + static_cast<int64_t>(j) * m.mp + i) = c;
                }
        return;
    }
    uint16_t* const o = reinterpret_cast<uint16_t*>(w + at.a);
    float* const d = reinterpret_cast<float*>(w + at.d);
    constexpr float un = kMuGramUnlift, scale = kMuLift * un;  // powers of two: exact
#pragma unroll
    for (int jj = 0; jj < M::NB; ++jj) {
        const int j0 = r.jb + 32 * jj;
        __builtin_amdgcn_sched_barrier(0);  // (one round's accumulators in registers at a time)
#pragma unroll
        for (int ii = 0; ii < M::MB; ++ii) {
            const f32x16& c = acc[ii][jj];
#pragma unroll
            for (int v = 0; v < 4; ++v)
                r.put(0, ii, v, mu_pack4(c[4 * v] * scale, c[4 * v + 1] * scale, c[4 * v + 2] * scale, c[4 * v + 3] * scale));
            if (r.ib + 32 * ii == j0) {  // the diagonal: the lane whose row is its column
#pragma unroll
                for (int v = 0; v < 4; ++v)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (8 * v + 4 * r.h + e == r.j) {
                            if (j0 + r.j < m.mp) stf(d + j0 + r.j, (c[4 * v + e] + mu_unfix(low[jj])) * un);
                            r.put(0, ii, v, mu_pack4(e == 0 ? 0.0f : c[4 * v] * scale, e == 1 ? 0.0f : c[4 * v + 1] * scale,
                                                     e == 2 ? 0.0f : c[4 * v + 2] * scale, e == 3 ? 0.0f : c[4 * v + 3] * scale));
                        }
            }
        }
        mu_store_sym(r, o, m.mp, j0);
    }
}

// The sums of A's parts, in order: 4 rows of a column j per thread (of the upper triangle). 5 to 6 us, a
// launch and the way to memory.
template <int N>
__global__ __launch_bounds__(kMuThreads) void k_mu_join(MuListOf<MuMatrix, N> l) {
    const int k = mu_find(l, blockIdx.x);
    const MuMatrix& m = l.d[k];
    const uint32_t per = static_cast<uint32_t>(m.mp / 4) * m.mp / kMuThreads;  // blocks per matrix (mp is a multiple of 64)
    const uint32_t item = mu_item(l, k, blockIdx.x), b = item / per;
    const int64_t q = static_cast<int64_t>(item % per) * kMuThreads + threadIdx.x;
    const int j = static_cast<int>(q / (m.mp / 4)), i = static_cast<int>(q % (m.mp / 4)) * 4;
    if (i > j) return;
    const MuPlace at(m.mp, m.np, m.parts);
    uint8_t* const w = m.ws + b * m.stride;
    const float* p = reinterpret_cast<const float*>(w + at.part) + static_cast<int64_t>(j) * m.mp + i;
    f32x4 s = *gld<f32x4>(p);
    for (int e = 1; e < m.parts; ++e) s += *gld<f32x4>(p + static_cast<int64_t>(e) * m.mp * m.mp);
    constexpr float un = kMuGramUnlift;
    float v[4] = {s.x * un, s.y * un, s.z * un, s.w * un};
    float* const d = reinterpret_cast<float*>(w + at.d);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (i + e == j) stf(d + j, v[e]);
        v[e] *= kMuLift;
    }
    uint16_t* const o = reinterpret_cast<uint16_t*>(w + at.a);
    // (rows past the diagonal belong to the other half: their values were not summed there)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (i + e > j) break;
        const uint16_t c = i + e == j ? 0 : __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[e]));
        *gst<uint16_t>(o + mu_at(j, i + e, m.mp)) = c;
        *gst<uint16_t>(o + mu_at(i + e, j, m.mp)) = c;
    }
}

// B = b A + c A^2 from A's off-diagonal part O and its diagonal d, 2^8 times off the diagonal,
// q = a + B_ii on it. As k_mu_gram, with O's tile read in the end: 4096 x 4096 in 78 to 83 us (medians).
template <int F, int N>
__global__ __launch_bounds__(kMuTileThreads, MuTiles<F>::kBlocks) void k_mu_poly(MuListOf<MuMatrix, N> l, MuPoly p) {
    using M = MuTiles<F>;
    __shared__ __attribute__((aligned(16))) uint8_t lds[M::kLds];
    const int k = mu_find(l, blockIdx.x);
    const MuMatrix& m = l.d[k];
    const int nt = (m.mp + M::kT - 1) / M::kT;
    const uint32_t per = nt * (nt + 1) / 2;
    const uint32_t t = mu_swizzle(mu_item(l, k, blockIdx.x), per * m.batch), b = t / per;
    int ti, tj;
    mu_triangle(t % per, nt, ti, tj);
    ti = uniform(ti);
    tj = uniform(tj);
    const MuPlace at(m.mp, m.np, m.parts);
    uint8_t* const w = m.ws + b * m.stride;
    const uint16_t* o = reinterpret_cast<const uint16_t*>(w + at.a);
    uint16_t* const out = reinterpret_cast<uint16_t*>(w + at.b);
    const float* const d = reinterpret_cast<const float*>(w + at.d);
    float* const q = reinterpret_cast<float*>(w + at.q);
    using R = MuRound<M>;
    const R r(lds, ti * M::kT, tj * M::kT, R::kBytes + R::kI * 4);
    auto load = [&](int j0, u32x4* f) {  // O's round
#pragma unroll
        for (int e = 0; e < R::kIters; ++e)
            if (r.has(m.mp, m.mp, j0, e)) f[e] = *gld<u32x4>(r.place(const_cast<uint16_t*>(o), m.mp, j0, e));
    };
    u32x4 next[R::kIters];
    if (M::kT < 256) load(r.jb, next);  // (the first round's before the product, which hides it; large: no registers)
    f32x16 acc[M::MB][M::NB];
    mu_zero<M>(acc);
    mu_accumulate<M, false>(o, m.mp, m.mp, o, m.mp, m.mp, ti * M::kT, tj * M::kT, 0, m.mp / 32, lds, acc);
    if (M::kT == 256) load(r.jb, next);
    // d_i of the wave's rows, in LDS
    const uint32_t di = r.base + R::kBytes;
    for (int i = r.lane; i < R::kI; i += 64)
        *(__attribute__((address_space(3))) float*)static_cast<uintptr_t>(di + i * 4) = ldf(d + min(r.ib + i, m.mp - 1));
    const float cs = p.c * kMuUnlift;
#pragma unroll
    for (int jj = 0; jj < M::NB; ++jj) {
        const int j0 = r.jb + 32 * jj;
        __builtin_amdgcn_sched_barrier(0);  // (one round's accumulators in registers at a time)
#pragma unroll
        for (int e = 0; e < R::kIters; ++e) r.put_line(0, e, next[e]);
        if (jj + 1 < M::NB) load(j0 + 32, next);
        const float dj = ldf(d + min(j0 + r.j, m.mp - 1));
#pragma unroll
        for (int ii = 0; ii < M::MB; ++ii) {
            const f32x16& c = acc[ii][jj];
            const bool diagonal = r.ib + 32 * ii == j0;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                // b A + c (O^2 + O (d_i + d_j)) = O (b + c (d_i + d_j)) + c O^2, the same bits for (j, i): a
                // tile on the diagonal forms and stores both
                const u32x2 x = r.get(0, ii, v);
                const f32x4 dd = *(const typename R::F4*)static_cast<uintptr_t>(di + (32 * ii + 8 * v + 4 * r.h) * 4);
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = fmaf(mu_half(x, e), fmaf(p.c, dd[e] + dj, p.b), c[4 * v + e] * cs);
                if (diagonal) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (8 * v + 4 * r.h + e == r.j) {
                            const float sq = c[4 * v + e] * (kMuUnlift * kMuUnlift);
                            if (j0 + r.j < m.mp) stf(q + j0 + r.j, p.a + fmaf(p.b, dj, p.c * fmaf(dj, dj, sq)));
                            y[e] = 0.0f;
                        }
                }
                r.put(0, ii, v, mu_pack4(y[0], y[1], y[2], y[3]));
            }
        }
        mu_store_sym(r, out, m.mp, j0);
    }
}

// X' = q hi + t lo + B hi (t = a + B_ii min(1, d_i^2)): X^T's tile (rows: X's columns) times B (symmetric: its rows), so that a
// lane's four values are consecutive in a row of X'. Into the other buffer, and the low part in place;
// the last step's into the caller's tensors. Medians: 4096 x 4096 in 141 to 145 us with 256-tiles (58% of
// the matrix units' cycles; the two parts in and out are 134 MB, 28 us of it, which the one round of tiles
// does not overlap), 4096 x 11008 in 383 us; 24 x 256 x 688 in 14 us, memory. What the low parts add to the
// next A's diagonal is 2 us of a 4096 x 4096 step.

// 8 values of the result in a row, from element i on, the first `valid` of them: the
// parameter's update or the rounded values.
__device__ __forceinline__ void mu_finish8(const MuTensor& t, bool update, float decay, int64_t i, int valid, float* v) {
    if (update) {
        float x[8];
        load_any8(t.x, i, valid, t.xbf16, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = x[e] * decay - t.coef * v[e];
    }
    store_any8(t.x, i, valid, t.xbf16, v);
}

template <int F, int N, class Last>
__global__ __launch_bounds__(kMuTileThreads, MuTiles<F>::kBlocks) void k_mu_apply(MuListOf<MuMatrix, N> l, int src, float linear, Last z) {
    using M = MuTiles<F>;
    constexpr bool kLast = !std::is_same<Last, MuNone>::value;
    __shared__ __attribute__((aligned(16))) uint8_t lds[M::kLds];
    const int k = mu_find(l, blockIdx.x);
    const MuMatrix& m = l.d[k];
    const uint32_t tm = (m.mp + M::kT - 1) / M::kT, tn = (m.np + M::kT - 1) / M::kT, per = tm * tn;
    uint32_t t = mu_swizzle(mu_item(l, k, blockIdx.x), per * m.batch);
    const uint32_t b = t / per;
    t -= b * per;
    // kMuGroup rows of X' at a time, by columns
    const uint32_t g = t / (kMuGroup * tn), rows = min<uint32_t>(kMuGroup, tm - g * kMuGroup);
    t -= g * kMuGroup * tn;
    const int ti = uniform(static_cast<int>(t / rows)), tj = uniform(static_cast<int>(g * kMuGroup + t % rows));
    const MuPlace at(m.mp, m.np, m.parts);
    uint8_t* const w = m.ws + b * m.stride;
    const uint16_t* const x = reinterpret_cast<const uint16_t*>(w + at.hi(src));
    uint16_t* const lo = reinterpret_cast<uint16_t*>(w + at.lo);
    const float* const q = reinterpret_cast<const float*>(w + at.q);
    uint16_t* const hi = reinterpret_cast<uint16_t*>(w + at.hi(src ^ 1));
    using R = MuRound<M>;
    constexpr uint32_t kPlanes = 2 * R::kBytes;  // X's two parts, then (last) the result
    const R r(lds, ti * M::kT, tj * M::kT, kLast ? 2 * kPlanes : kPlanes);
    static_assert(M::kNW * 2 * kPlanes <= M::kLds, "the waves' shares fit the stages");
    auto load = [&](int j0, u32x4* f) {
#pragma unroll
        for (int e = 0; e < R::kIters; ++e) {
            if (!r.has(m.mp, m.np, j0, e)) continue;
            f[2 * e] = *gld<u32x4>(r.place(const_cast<uint16_t*>(x), m.np, j0, e));
            f[2 * e + 1] = *gld<u32x4>(r.place(lo, m.np, j0, e));
        }
    };
    u32x4 next[2 * R::kIters];
    if (M::kT < 256) load(r.jb, next);  // (the first round's before the product, which hides it; large: no registers)
    f32x16 acc[M::MB][M::NB];
    mu_zero<M>(acc);
    mu_accumulate<M, true>(x, m.np, m.np, reinterpret_cast<const uint16_t*>(w + at.b), m.mp, m.mp, ti * M::kT, tj * M::kT, 0,
                           m.mp / 32, lds, acc);
    if (M::kT == 256) load(r.jb, next);
    constexpr float un = kMuXUnlift * kMuUnlift;
    const float* const d = reinterpret_cast<const float*>(w + at.d);
#pragma unroll
    for (int jj = 0; jj < M::NB; ++jj) {
        const int j0 = r.jb + 32 * jj;
        __builtin_amdgcn_sched_barrier(0);  // (one round's accumulators in registers at a time)
#pragma unroll
        for (int e = 0; e < R::kIters; ++e) {
            r.put_line(0, e, next[2 * e]);
            r.put_line(1, e, next[2 * e + 1]);
        }
        if (jj + 1 < M::NB) load(j0 + 32, next);
        const float dj = ldf(d + min(j0 + r.j, m.mp - 1)), qj = ldf(q + min(j0 + r.j, m.mp - 1)) * kMuLift;
        const float al = linear * kMuLift, tl = fmaf(qj - al, fminf(dj * dj, 1.0f), al);
        uint32_t sum = 0;  // what the low parts add to row j's norm
#pragma unroll
        for (int ii = 0; ii < M::MB; ++ii) {
            const f32x16& c = acc[ii][jj];
            float low = 0.0f;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const u32x2 xh = r.get(0, ii, v), xl = r.get(1, ii, v);
                float y[4];  // 2^8 X'
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = fmaf(tl, mu_half(xl, e), fmaf(qj, mu_half(xh, e), c[4 * v + e]));
                if constexpr (kLast) {
                    r.put32(kPlanes, ii, v, f32x4{y[0] * un, y[1] * un, y[2] * un, y[3] * un});
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] *= kMuUnlift;
                    const u32x2 n = mu_pack4(y[0], y[1], y[2], y[3]);
                    r.put(0, ii, v, n);
                    float o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[e] = y[e] - mu_half(n, e);
                        low = fmaf(o[e], mu_half(n, e), low);
                    }
                    r.put(1, ii, v, mu_pack4(o[0], o[1], o[2], o[3]));
                }
            }
            if (!kLast && r.ib + 32 * ii < m.np) sum += mu_fix(low);
        }
        if constexpr (!kLast) {
            sum = mu_halves(sum);
            if (r.h == 0 && j0 < m.mp && r.ib < m.np)
                mu_fixed_add(reinterpret_cast<int32_t*>(w + at.low(src ^ 1, m.mp)) + j0 + r.j, sum);
#pragma unroll
            for (int e = 0; e < R::kIters; ++e) {
                if (!r.has(m.mp, m.np, j0, e)) continue;
                *gst<u32x4>(r.place(hi, m.np, j0, e)) = r.get_line(0, e);
                *gst<u32x4>(r.place(lo, m.np, j0, e)) = r.get_line(1, e);
            }
        } else {
            const MuTensor& t = z.t.d[k];
            const int64_t first = b * (static_cast<int64_t>(t.rows) * t.ldx);
            if (t.tall) {  // row j of X' is column j of the caller's matrix: 8 of them of its row i
#pragma unroll 2
                for (int e = 0; e < R::kI / 16; ++e) {
                    const int i = r.ib + 16 * e + (r.lane >> 2), j = j0 + (r.lane & 3) * 8;
                    const int valid = i < t.rows ? clamp_valid(static_cast<int64_t>(t.cols) - j) : 0;
                    float v[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) v[u] = r.get32_value(kPlanes, (r.lane & 3) * 8 + u, 16 * e + (r.lane >> 2));
                    if (valid > 0) mu_finish8(t, z.update, z.decay, first + i * t.ldx + j, valid, v);
                }
            } else {
#pragma unroll 2
                for (int e = r.lane; e < 32 * R::kI / 8; e += 64) {  // 8 values of a row j each
                    const int row = e / (R::kI / 8), col = e % (R::kI / 8) * 8, i = r.ib + col, j = j0 + row;
                    const int valid = j < t.rows ? clamp_valid(static_cast<int64_t>(t.cols) - i) : 0;
                    const f32x4 a = r.get32(kPlanes, row, col / 4), c = r.get32(kPlanes, row, col / 4 + 1);
                    float v[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
                    if (valid > 0) mu_finish8(t, z.update, z.decay, first + j * t.ldx + i, valid, v);
                }
            }
        }
    }
}

}  // namespace

// f(list, form) with one tensor alone by itself.
template <class List, class Fn>
static void with_list(const List& l, Fn f) {
    if (l.n == 1) f(l.only(), std::integral_constant<int, 1>{});
    else f(l, std::integral_constant<int, kMuBatch>{});
}
template <class Fn>
static void with_form(int form, Fn f) {
    if (form == kMuLarge) f(std::integral_constant<int, kMuLarge>{});
    else if (form == kMuThreeQuarters) f(std::integral_constant<int, kMuThreeQuarters>{});
    else if (form == kMuMedium) f(std::integral_constant<int, kMuMedium>{});
    else f(std::integral_constant<int, kMuSmall>{});
}

void launch_mu_momentum(const MuTensors& t, const MuStepArgs& a, hipStream_t s) {
    with_list(t, [&](const auto& l, auto n) {
        hipLaunchKernelGGL(k_mu_momentum<decltype(n)::value>, dim3(t.blocks), dim3(kMuThreads), 0, s, l, a);
    });
}

void launch_mu_scatter(const MuTensors& t, const MuStepArgs& a, hipStream_t s) {
    with_list(t, [&](const auto& l, auto n) {
        hipLaunchKernelGGL(k_mu_scatter<decltype(n)::value>, dim3(t.blocks), dim3(kMuThreads), 0, s, l, a);
    });
}

void launch_mu_gram(const MuMatrices& m, int form, int src, hipStream_t s) {
    if (m.blocks == 0) return;
    with_list(m, [&](const auto& l, auto n) {
        with_form(form, [&](auto f) {
            hipLaunchKernelGGL((k_mu_gram<decltype(f)::value, decltype(n)::value>), dim3(m.blocks), dim3(kMuTileThreads), 0, s, l, src);
        });
    });
}

void launch_mu_join(const MuMatrices& m, hipStream_t s) {
    if (m.blocks == 0) return;
    with_list(m, [&](const auto& l, auto n) {
        hipLaunchKernelGGL(k_mu_join<decltype(n)::value>, dim3(m.blocks), dim3(kMuThreads), 0, s, l);
    });
}

void launch_mu_poly(const MuMatrices& m, int form, const MuPoly& p, hipStream_t s) {
    with_list(m, [&](const auto& l, auto n) {
        with_form(form, [&](auto f) {
            hipLaunchKernelGGL((k_mu_poly<decltype(f)::value, decltype(n)::value>), dim3(m.blocks), dim3(kMuTileThreads), 0, s, l, p);
        });
    });
}

void launch_mu_apply(const MuMatrices& m, int form, int src, float linear, const MuLast* last, hipStream_t s) {
    with_list(m, [&](const auto& l, auto n) {
        constexpr int N = decltype(n)::value;
        with_form(form, [&](auto f) {
            constexpr int F = decltype(f)::value;
            const dim3 g(m.blocks), t(kMuTileThreads);
            if (!last) {
                hipLaunchKernelGGL((k_mu_apply<F, N, MuNone>), g, t, 0, s, l, src, linear, MuNone{});
            } else if constexpr (N == 1) {
                const MuLastOf<1> z{last->t.only(), last->decay, last->update};
                hipLaunchKernelGGL((k_mu_apply<F, N, MuLastOf<1>>), g, t, 0, s, l, src, linear, z);
            } else {
                hipLaunchKernelGGL((k_mu_apply<F, N, MuLast>), g, t, 0, s, l, src, linear, *last);
            }
        });
    });
}

}  // namespace meo
