// Orthogonalization and the Muon step of matrices with few rows (a shorter side of at most 64), where
// each pass of muon.hip over such a matrix is a launch of 3 to 5 us, 17 and more of them.
//
// The mathematics is muon.hip's, but X, A and B are held as two fp16 parts in every product (hi hi +
// hi lo + lo hi: 22 bits): products are what such matrices have little of, and small ones would lose
// more to fp16 than large ones do (gaussian 16 x 16: 1.2e-3 of the result with one part, 3e-7 so,
// 7e-7 in float32).
//
// The longer side goes by blocks of 32 columns, a strip of 16 (64 rows: 8) to a thread block, each
// wave's its own: the step X' = a X + B X needs nothing else of X. A = X X^T is summed over the waves
// through LDS, over strips through the workspace. In an accumulator of a symmetric matrix a lane holds
// four consecutive rows of a column, which are four consecutive values of the contraction of that column
// as an operand: A, A^2 and B go from product to product as they are, in registers (16 rows) or through
// LDS by 16 bytes. A matrix of one strip is one launch, with the iterate in LDS; one of more strips is a
// launch per step and two before them.
//
// What bounds it: latencies (launches, barriers, LDS, dependent products). The work per value is some
// 8 vector instructions a step, too many for one CU from 16 x 1024 on: 16 x 4096 in one block took
// 59 us (in 8 strips 29), 4096 x 16 87 (31).
#include "muon_device.h"

namespace meo {

namespace {

typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) u32x2 L2;
typedef __attribute__((address_space(3))) u32x4 L4;
typedef __attribute__((address_space(3))) f32x4 F4;
typedef __attribute__((address_space(3))) float F1;
typedef __attribute__((address_space(3))) double D1;
typedef __attribute__((address_space(3))) uint16_t H1;

constexpr int kMuFewWaves = kMuFewThreads / 64;

// An LDS access of a wave to what its other lanes wrote is not moved over this.
__device__ __forceinline__ void mu_order() { __asm__ volatile("" ::: "memory"); }

// f(p) with p a constant, for registers that a loop indexes: a branch each. (An array indexed at run
// time became a selection over all of it; a loop written out in full, code that is read from memory
// once per launch.)
template <int N, class Fn>
__device__ __forceinline__ void mu_case(int p, Fn f) {
    if constexpr (N > 0) {
        if (p == N - 1) {
            f(std::integral_constant<int, N - 1>{});
            __asm__ volatile("; %0" ::"n"(N));  // (branches that end alike would be merged)
        } else {
            mu_case<N - 1>(p, f);
        }
    }
}

// X in LDS: blocks of 32 columns, R rows of 64 bytes in each, chunk c (16 bytes) of row r at position
// c ^ (r >> 2 & 3): rows read at one chunk touch every bank alike. The bytes of 4 values, chunk c8 >> 1:
__device__ __forceinline__ uint32_t mu_few_at(int r, int c8) {
    return r * 64 + (((c8 >> 1) ^ ((r >> 2) & 3)) << 4) + (c8 & 1) * 8;
}

// The products of a strip of R rows, its high parts at LDS address x, its low parts kBytes on. Accumulators: tiles of T x T, where a lane holds
// rows 8 v + 4 h + 0 .. 3 of its column, v < V. A block of 32 columns: SB parts of NT tiles.
template <int R>
struct MuFew {
    static constexpr int T = R == 16 ? 16 : 32, NT = R / T, V = T == 16 ? 1 : 4, SB = 32 / T;
    static constexpr int kStrip = mu_strip(R), NB = kStrip / 32 / kMuFewWaves;  // columns; blocks per wave
    static constexpr int kBytes = R * kStrip * 2;  // of one part of the strip
    // A's parts: by wave; R = 64: by pairs of waves, which have a column of tiles each.
    static constexpr int kParts = R == 64 ? kMuFewWaves / 2 : kMuFewWaves;
    static constexpr int kPart = R * R * 4, kSums = kParts * kPart;
    static constexpr int kLds = 2 * kBytes + kSums + 2 * R * 4;
    struct Acc { f32x4 v[V]; };
    struct Op { u32x2 v[V]; };  // T values of the contraction
    struct Ops { Op hi, lo; };
    typedef u32x2 Block[SB][NT][V];  // of the iterate, as accumulators have it

    uint32_t x, sums;
    int lane, wave, col, h;
    __device__ MuFew(uint32_t x_, uint32_t sums_) : x(x_), sums(sums_) {
        lane = threadIdx.x & 63;
        wave = uniform(threadIdx.x >> 6);
        col = lane & (T - 1);
        h = lane / T;
    }

    static __device__ __forceinline__ void mul(Acc& c, const Op& a, const Op& b) {
        if constexpr (T == 16) {
            c.v[0] = __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(half4, a.v[0]), __builtin_bit_cast(half4, b.v[0]), c.v[0], 0, 0, 0);
        } else {
            f32x16 w = __builtin_bit_cast(f32x16, c);
#pragma unroll
            for (int s = 0; s < 2; ++s)
                w = mfma_f16(u32x4{a.v[2 * s].x, a.v[2 * s].y, a.v[2 * s + 1].x, a.v[2 * s + 1].y},
                             u32x4{b.v[2 * s].x, b.v[2 * s].y, b.v[2 * s + 1].x, b.v[2 * s + 1].y}, w);
            c = __builtin_bit_cast(Acc, w);
        }
    }
    static __device__ __forceinline__ void mul(Acc& c, const Ops& a, const Ops& b) {
        mul(c, a.hi, b.lo);
        mul(c, a.lo, b.hi);
        mul(c, a.hi, b.hi);
    }
    static __device__ __forceinline__ void zero(Acc& c) {
#pragma unroll
        for (int v = 0; v < V; ++v) c.v[v] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // The n-th block of the wave, and where an accumulator's four values are in it.
    __device__ int block(int n) const { return n * kMuFewWaves + wave; }
    __device__ uint32_t place(int blk, int sb, int it, int v) const {
        return x + blk * (R * 64) + mu_few_at(it * T + col, T == 16 ? 4 * sb + h : 2 * v + h);
    }
    // f(sb, it, v) over a block.
    template <class Fn>
    static __device__ __forceinline__ void each(Fn f) {
#pragma unroll
        for (int sb = 0; sb < SB; ++sb)
#pragma unroll
            for (int it = 0; it < NT; ++it)
#pragma unroll
                for (int v = 0; v < V; ++v) f(sb, it, v);
    }

    // The wave's part of X X^T, of nb blocks, to `sums`. (R = 64: of blocks that two waves have.)
    __device__ __forceinline__ void gram(int nb) const {
        const int part = R == 64 ? wave >> 1 : wave, tj = R == 64 ? wave & 1 : 0;
        Acc g[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) zero(g[i]);
        for (int blk = part; blk < nb; blk += kParts) {
            const uint32_t o = x + blk * (R * 64);
            if constexpr (T == 16) {
                const half8 w = __builtin_bit_cast(half8, mu_lds(o + mu_few_at(col, 2 * h)));
                const half8 z = __builtin_bit_cast(half8, mu_lds(o + kBytes + mu_few_at(col, 2 * h)));
                g[0].v[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, z, g[0].v[0], 0, 0, 0);
                g[0].v[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(z, w, g[0].v[0], 0, 0, 0);
                g[0].v[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, w, g[0].v[0], 0, 0, 0);
            } else {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    u32x4 w[NT], z[NT];
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        w[i] = mu_lds(o + mu_few_at(i * T + col, 4 * c + 2 * h));
                        z[i] = mu_lds(o + kBytes + mu_few_at(i * T + col, 4 * c + 2 * h));
                    }
                    const u32x4 wj = NT == 1 || tj == 0 ? w[0] : w[NT - 1], zj = NT == 1 || tj == 0 ? z[0] : z[NT - 1];
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        f32x16 y = __builtin_bit_cast(f32x16, g[i]);
                        y = mfma_f16(w[i], zj, y);
                        y = mfma_f16(z[i], wj, y);
                        g[i] = __builtin_bit_cast(Acc, mfma_f16(w[i], wj, y));
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v)
                *(F4*)static_cast<uintptr_t>(sums + part * kPart + (((tj * NT + i) * V + v) * 64 + lane) * 16) = g[i].v[v];
    }
    // 16 bytes of the parts' sum, in order: chunks [column of tiles][row][v][lane].
    __device__ __forceinline__ f32x4 joined(int chunk) const {
        f32x4 w = *(const F4*)static_cast<uintptr_t>(sums + chunk * 16);
#pragma unroll
        for (int e = 1; e < kParts; ++e) w += *(const F4*)static_cast<uintptr_t>(sums + e * kPart + chunk * 16);
        return w;
    }

    // Four fp32 values as two fp16 parts.
    static __device__ __forceinline__ u32x2 parts(const f32x4& y, u32x2& lo) {
        const u32x2 w = mu_pack4(y.x, y.y, y.z, y.w);
        lo = mu_pack4(y.x - mu_half(w, 0), y.y - mu_half(w, 1), y.z - mu_half(w, 2), y.w - mu_half(w, 3));
        return w;
    }

    // A chunk of X X^T (times 4^12) becomes O's, 2^8 times, its two parts in the chunk's place;
    // the diagonal goes to diag().
    __device__ uint32_t diag() const { return sums + kSums; }
    __device__ uint32_t rows() const { return sums + kSums + R * 4; }  // q
    __device__ __forceinline__ void put_o(int chunk, f32x4 w, float un) const {
        const int z = chunk & 63, v = chunk / 64 % V, i = chunk / 64 / V % NT, j = chunk / 64 / V / NT;
        const int c = z & (T - 1), r = 8 * v + 4 * (z / T);
        w *= un;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i == j && r + e == c) {
                *(F1*)static_cast<uintptr_t>(diag() + (j * T + c) * 4) = w[e];
                w[e] = 0.0f;
            }
        u32x2 lo;
        const u32x2 hi = parts(w * kMuLift, lo);
        *(L4*)static_cast<uintptr_t>(sums + chunk * 16) = u32x4{hi.x, hi.y, lo.x, lo.y};
    }
    __device__ __forceinline__ Ops operand(uint32_t at, int j, int i) const {  // a tile of chunks
        Ops o;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const u32x4 w = mu_lds(at + (((j * NT + i) * V + v) * 64 + lane) * 16);
            o.hi.v[v] = u32x2{w.x, w.y};
            o.lo.v[v] = u32x2{w.z, w.w};
        }
        return o;
    }

    // From O (put_o, then a barrier): B, 2^8 times off the diagonal, as operands, and of the lane's columns
    // q = a + B_ii, 2^8 times. With 16 rows each wave forms B, with more a part of it each
    // (64 rows in every wave: 8 us of a step's arithmetic).
    Ops B[NT][NT];  // [column][row]
    float q[NT];
    __device__ __forceinline__ void poly(const MuPoly& p) {
        constexpr int kUnits = NT * NT * V, kPer = kUnits > kMuFewWaves ? kUnits / kMuFewWaves : 1;  // four values each
        const float cs = p.c * kMuUnlift;
        if (R == 16 || wave < kUnits) {
            const int tile = R == 16 ? 0 : wave * kPer / V, j = tile / NT, i = tile % NT;
            Ops a[NT], b[NT];
            Acc sq;
            zero(sq);
#pragma unroll
            for (int z = 0; z < NT; ++z) {
                a[z] = operand(sums, i, z);
                b[z] = NT == 1 ? a[z] : operand(sums, j, z);
                mul(sq, a[z], b[z]);
            }
            const float dj = *(const F1*)static_cast<uintptr_t>(diag() + (j * T + col) * 4);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (R != 16 && v / kPer != wave % (V / kPer)) continue;
                const f32x4 di = *(const F4*)static_cast<uintptr_t>(diag() + (i * T + 8 * v + 4 * h) * 4);
                const u32x4 o = mu_lds(sums + (((j * NT + i) * V + v) * 64 + lane) * 16);
                f32x4 y;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] = fmaf(mu_half(u32x2{o.x, o.y}, e) + mu_half(u32x2{o.z, o.w}, e), fmaf(p.c, di[e] + dj, p.b), sq.v[v][e] * cs);
                    if (i == j && 8 * v + 4 * h + e == col) {
                        *(F1*)static_cast<uintptr_t>(rows() + (j * T + col) * 4) =
                            (p.a + fmaf(p.b, dj, p.c * fmaf(dj, dj, sq.v[v][e] * (kMuUnlift * kMuUnlift)))) * kMuLift;
                        y[e] = 0.0f;
                    }
                }
                u32x2 lo;
                const u32x2 hi = parts(y, lo);
                if constexpr (R == 16) {
                    B[0][0].hi.v[0] = hi;
                    B[0][0].lo.v[0] = lo;
                } else {
                    *(L4*)static_cast<uintptr_t>(sums + kPart + (((j * NT + i) * V + v) * 64 + lane) * 16) = u32x4{hi.x, hi.y, lo.x, lo.y};
                }
            }
        }
        if (R == 16) {
            mu_order();  // (waves write the same q)
        } else {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < NT; ++i) B[j][i] = operand(sums + kPart, j, i);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) q[j] = *(const F1*)static_cast<uintptr_t>(rows() + (j * T + col) * 4);
    }

    // X' of a block of LDS: f(sb, it, v, four values, 2^8 times).
    template <class Fn>
    __device__ __forceinline__ void apply(int blk, Fn f) const {
        mu_order();
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) {
            Ops xt[NT];  // X^T's part: 4 rows of X of the lane's column each
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const uint32_t at = x + blk * (R * 64) + mu_few_at(i * T + 8 * v + 4 * h + ((lane >> 2) & 3),
                                                                       T == 16 ? 4 * sb + (lane & 3) : ((lane >> 4) & 1) * 4 + (lane & 3));
                    xt[i].hi.v[v] = mu_lds_tr(at);
                    xt[i].lo.v[v] = mu_lds_tr(at + kBytes);
                }
            mu_order();
#pragma unroll
            for (int it = 0; it < NT; ++it) {
                Acc c;
                zero(c);
#pragma unroll
                for (int i = 0; i < NT; ++i) mul(c, xt[i], B[it][i]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const uint32_t at = place(blk, sb, it, v);
                    const u32x2 xh = *(const L2*)static_cast<uintptr_t>(at), xl = *(const L2*)static_cast<uintptr_t>(at + kBytes);
                    f32x4 y;
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = fmaf(q[it], mu_half(xl, e), fmaf(q[it], mu_half(xh, e), c.v[v][e]));
                    f(sb, it, v, y);
                }
            }
        }
    }
    // As an iterate's parts, into LDS.
    __device__ __forceinline__ u32x2 split(int blk, int sb, int it, int v, const f32x4& y, u32x2& lo) const {
        const u32x2 w = parts(y * kMuUnlift, lo);
        const uint32_t at = place(blk, sb, it, v);
        *(L2*)static_cast<uintptr_t>(at) = w;
        *(L2*)static_cast<uintptr_t>(at + kBytes) = lo;
        return w;
    }
    // The first column, in a block, of four values.
    __device__ int column(int sb, int v) const { return (T == 16 ? 16 * sb : 0) + 8 * v + 4 * h; }
};

__device__ __forceinline__ void mu_few_clear(uint32_t at, uint32_t bytes) {
    for (uint32_t o = threadIdx.x * 16; o < bytes; o += kMuFewThreads * 16) *(L4*)static_cast<uintptr_t>(at + o) = u32x4{0u, 0u, 0u, 0u};
}
// 8 values of a row, and one, of a strip in LDS.
template <int R>
__device__ __forceinline__ void mu_few_put(uint32_t x, int r, int c, const uint32_t* hi, const uint32_t* lo) {
    const uint32_t at = x + (c >> 5) * (R * 64) + mu_few_at(r, (c & 31) >> 2);
    *(L4*)static_cast<uintptr_t>(at) = u32x4{hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, hi[4] | hi[5] << 16, hi[6] | hi[7] << 16};
    *(L4*)static_cast<uintptr_t>(at + MuFew<R>::kBytes) = u32x4{lo[0] | lo[1] << 16, lo[2] | lo[3] << 16, lo[4] | lo[5] << 16, lo[6] | lo[7] << 16};
}
template <int R>
__device__ __forceinline__ void mu_few_put1(uint32_t x, int r, int c, uint32_t hi, uint32_t lo) {
    const uint32_t at = x + (c >> 5) * (R * 64) + mu_few_at(r, (c & 31) >> 2) + (c & 3) * 2;
    *(H1*)static_cast<uintptr_t>(at) = static_cast<uint16_t>(hi);
    *(H1*)static_cast<uintptr_t>(at + MuFew<R>::kBytes) = static_cast<uint16_t>(lo);
}
// The sum over the block, in order; `at`: 8 bytes of LDS per wave.
__device__ __forceinline__ double mu_few_sum(double s, uint32_t at) {
    s = wave_sum(s);
    if ((threadIdx.x & 63) == 0) *(D1*)static_cast<uintptr_t>(at + (threadIdx.x >> 6) * 8) = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < kMuFewWaves; ++w) s += *(const D1*)static_cast<uintptr_t>(at + w * 8);
    return s;
}

// Four values of a row of X' (element (i, j), ..., (i, j + 3)) into the caller's tensor.
__device__ __forceinline__ void mu_few_store(const MuTensor& t, bool update, float decay, int64_t first, int i, int j, const f32x4& y) {
    const int short_side = t.tall ? t.cols : t.rows, long_side = t.tall ? t.rows : t.cols;
    if (i >= short_side || j >= long_side) return;
    typedef u32x2 u32x2_any __attribute__((aligned(2)));
    const int valid = min(4, long_side - j);
    if (!t.tall && valid == 4) {
        const int64_t at = first + static_cast<int64_t>(i) * t.ldx + j;
        f32x4 v = y;
        if (t.xbf16) {
            uint16_t* const p = static_cast<uint16_t*>(t.x) + at;
            if (update) {
                const u32x2 w = *gld<u32x2_any>(p);
                v = f32x4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)} * decay - t.coef * y;
            }
            *gst<u32x2_any>(p) = u32x2{bf16_bits(v.x) | bf16_bits(v.y) << 16, bf16_bits(v.z) | bf16_bits(v.w) << 16};
        } else {
            float* const p = static_cast<float*>(t.x) + at;
            if (update) v = *gld<f32x4_any>(p) * decay - t.coef * y;
            *gst<f32x4_any>(p) = v;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (e >= valid) break;
        const int64_t at = first + (t.tall ? static_cast<int64_t>(j + e) * t.ldx + i : static_cast<int64_t>(i) * t.ldx + j + e);
        float v = y[e];
        if (t.xbf16) {
            uint16_t* const p = static_cast<uint16_t*>(t.x) + at;
            if (update) v = bf16_lo(*gld<uint16_t>(p)) * decay - t.coef * v;
            *gst<uint16_t>(p) = static_cast<uint16_t>(bf16_bits(v));
        } else {
            float* const p = static_cast<float*>(t.x) + at;
            if (update) v = *gld<float>(p) * decay - t.coef * v;
            *gst<float>(p) = v;
        }
    }
}

// A matrix of one strip per block, all steps. In a captured graph: 16 x 16 8.8 us, 32 x 64 13.8, 64 x 64
// 24.9 (five steps; in tiles, 17 launches, 32 x 64 took 64).
template <int R, int N>
__global__ __launch_bounds__(kMuFewThreads, 2) void k_mu_few(MuListOf<MuFewTensor, N> l, MuFewArgs a) {
    using M = MuFew<R>;
    constexpr int kTurn = kMuFewThreads * kVec, kTurns = R * M::kStrip / kTurn;
    __shared__ __attribute__((aligned(16))) uint8_t lds[M::kLds];
    const int k = mu_find(l, blockIdx.x);
    const int b = static_cast<int>(mu_item(l, k, blockIdx.x));
    const MuFewTensor& s = l.d[k];
    MuTensor t;
    t.g = s.g; t.m = s.m; t.ms = s.ms; t.x = s.x;
    t.ldg = s.ldg; t.ldx = s.ldx;
    t.rows = s.rows; t.cols = s.cols;
    t.coef = s.coef;
    t.gbf16 = s.gbf16; t.xbf16 = s.xbf16; t.mkind = s.mkind;
    t.tall = s.rows > s.cols;
    const int size = t.rows * t.cols;
    const int nb = uniform((max(t.rows, t.cols) + 31) / 32);
    const uint32_t x0 = uniform(static_cast<int>(lds_addr(lds)));
    M m(x0, x0 + 2 * M::kBytes);

    // the directions and their squares' sum
    mu_few_clear(x0, nb * R * 64);
    mu_few_clear(x0 + M::kBytes, nb * R * 64);
    const int turns = uniform((size + kTurn - 1) / kTurn);
    float u[kTurns][kVec];
    double sum = 0.0;
#pragma unroll 1
    for (int p = 0; p < turns; ++p) {
        const int i = p * kTurn + threadIdx.x * kVec;
        float w[kVec];
        mu_take8(t, a.step, b, static_cast<int64_t>(b) * size, i, clamp_valid(static_cast<int64_t>(size) - i), w);
#pragma unroll
        for (int e = 0; e < kVec; ++e) sum += static_cast<double>(w[e]) * static_cast<double>(w[e]);
        mu_case<kTurns>(p, [&](auto q) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) u[q][e] = w[e];
        });
    }
    const double f = mu_factor_of(mu_few_sum(sum, m.sums), a.step.eps);

    // X0 in two parts
#pragma unroll 1
    for (int p = 0; p < turns; ++p) {
        const int i = p * kTurn + threadIdx.x * kVec;
        float z[kVec];
        mu_case<kTurns>(p, [&](auto q) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) z[e] = u[q][e];
        });
        uint32_t hi[kVec], lo[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) mu_split(static_cast<float>(z[e] * f), hi[e], lo[e]);
        if (i >= size) continue;
        int row = static_cast<uint32_t>(i) / static_cast<uint32_t>(t.cols), col = i - row * t.cols;
        if (!t.tall && col % kVec == 0 && col + kVec <= t.cols) {
            mu_few_put<R>(x0, row, col, hi, lo);
            continue;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            if (i + e < size) mu_few_put1<R>(x0, t.tall ? col : row, t.tall ? row : col, hi[e], lo[e]);
            if (++col == t.cols) {
                col = 0;
                ++row;
            }
        }
    }
    __syncthreads();

    constexpr float un = kMuGramUnlift, out = kMuXUnlift * kMuUnlift;
    const int64_t first = static_cast<int64_t>(b) * t.rows * t.ldx;
#pragma unroll 1
    for (int step = 0; step < a.steps; ++step) {
        m.gram(nb);
        __syncthreads();
        for (int c = threadIdx.x; c < M::kPart / 16; c += kMuFewThreads) m.put_o(c, m.joined(c), un);
        __syncthreads();
        m.poly(a.poly[step]);
        if (step + 1 == a.steps) {
#pragma unroll 1
            for (int blk = m.wave; blk < nb; blk += kMuFewWaves)
                m.apply(blk, [&](int sb, int it, int v, const f32x4& y) {
                    mu_few_store(t, a.update, a.decay, first, it * M::T + m.col, 32 * blk + m.column(sb, v), y * out);
                });
            return;
        }
#pragma unroll 1
        for (int blk = m.wave; blk < nb; blk += kMuFewWaves)
            m.apply(blk, [&](int sb, int it, int v, const f32x4& y) {
                u32x2 lo;
                m.split(blk, sb, it, v, y, lo);
            });
        mu_order();
        __syncthreads();  // A's sums have been read; R = 64: X' is read by two waves
    }
}

// Strips: X0 of one, into the workspace as accumulators have it, and its part of A. Four of 16 x 4096 and
// 4096 x 16: 7 us.
template <int R, int N>
__global__ __launch_bounds__(kMuFewThreads, 2) void k_mu_strip_start(MuListOf<MuTensor, N> l, MuStepArgs a) {
    using M = MuFew<R>;
    __shared__ __attribute__((aligned(16))) uint8_t lds[M::kLds];
    const int k = mu_find(l, blockIdx.x);
    const MuTensor& t = l.d[k];
    const uint32_t item = mu_item(l, k, blockIdx.x);
    const int strips = t.np / M::kStrip, b = uniform(static_cast<int>(item / strips)), strip = uniform(static_cast<int>(item % strips));
    const uint32_t x0 = uniform(static_cast<int>(lds_addr(lds)));
    M m(x0, x0 + 2 * M::kBytes);
    mu_few_clear(x0, 2 * M::kBytes);
    double sum = 0.0;
    const double* p = t.norm + static_cast<int64_t>(b) * t.parts;
    for (int i = threadIdx.x; i < t.parts; i += kMuFewThreads) sum += *gld<double>(p + i);
    const double f = mu_factor_of(mu_few_sum(sum, m.sums), a.eps);
    const int c0 = strip * M::kStrip, per = t.tall ? (t.cols + kVec - 1) / kVec : M::kStrip / kVec;  // 8 values each of a row
    const int rows = t.tall ? min(M::kStrip, t.rows - c0) : t.rows;
#pragma unroll 2
    for (int e0 = threadIdx.x; e0 < rows * per; e0 += kMuFewThreads) {
        const int r = e0 / per, c = e0 % per * kVec;
        const int row = t.tall ? c0 + r : r, col = t.tall ? c : c0 + c;
        const int valid = clamp_valid(static_cast<int64_t>(t.cols) - col);
        if (valid <= 0) continue;
        float u[kVec], g[kVec], w[kVec];
        const int64_t i = (static_cast<int64_t>(b) * t.rows + row);
        load_any8(t.g, i * t.ldg + col, valid, t.gbf16, g);
        if (t.m) {
            mu_load_m(t, i * t.cols + col, valid, w);
            mu_direction(a, g, w, u);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) u[e] = g[e];
        }
        uint32_t hi[kVec], lo[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) mu_split(e < valid ? static_cast<float>(u[e] * f) : 0.0f, hi[e], lo[e]);
        if (!t.tall) {
            mu_few_put<R>(x0, r, c, hi, lo);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (e < valid) mu_few_put1<R>(x0, c + e, r, hi[e], lo[e]);
        }
    }
    __syncthreads();
    const MuStripPlace at(t.mp, t.np, strips);
    uint8_t* const ws = t.ws + b * t.stride;
#pragma unroll
    for (int n = 0; n < M::NB; ++n) {
        const int blk = m.block(n);
        uint8_t* const w = ws + strip * M::kBytes + blk * (R * 64) + m.lane * 8;
        M::each([&](int sb, int it, int v) {
            const int64_t o = ((sb * M::NT + it) * M::V + v) * 512;
            const uint32_t z = m.place(blk, sb, it, v);
            *gst<u32x2>(w + o) = *(const L2*)static_cast<uintptr_t>(z);
            *gst<u32x2>(w + at.lo + o) = *(const L2*)static_cast<uintptr_t>(z + M::kBytes);
        });
    }
    m.gram(M::kStrip / 32);
    __syncthreads();
    float* const o = reinterpret_cast<float*>(ws + at.part) + static_cast<int64_t>(strip) * R * R;
    for (int c = threadIdx.x; c < M::kPart / 16; c += kMuFewThreads) *gst<f32x4>(o + c * 4) = m.joined(c);
}

// One step of a strip: A from all strips' parts (buffer src), X', its part of the next A; the last
// step's X' goes to the caller's tensors. Every strip joins all parts, which costs less than a launch for
// it: 16 x 4096 (8 parts of 1 KB) 4.3 us a step, 64 x 4096 (16 of 16 KB) 10.8.
template <int R, int N>
__global__ __launch_bounds__(kMuFewThreads, 2) void k_mu_strip_step(MuListOf<MuTensor, N> l, MuPoly poly, int src, int last, int update,
                                                                    float decay) {
    using M = MuFew<R>;
    __shared__ __attribute__((aligned(16))) uint8_t lds[M::kLds];
    const int k = mu_find(l, blockIdx.x);
    const MuTensor& t = l.d[k];
    const uint32_t item = mu_item(l, k, blockIdx.x);
    const int strips = t.np / M::kStrip, b = uniform(static_cast<int>(item / strips)), strip = uniform(static_cast<int>(item % strips));
    const uint32_t x0 = uniform(static_cast<int>(lds_addr(lds)));
    M m(x0, x0 + 2 * M::kBytes);
    const MuStripPlace at(t.mp, t.np, strips);
    uint8_t* const ws = t.ws + b * t.stride;
    uint8_t* const w = ws + strip * M::kBytes + m.lane * 8;
    typename M::Block high[M::NB], low[M::NB];
#pragma unroll
    for (int n = 0; n < M::NB; ++n)
        M::each([&](int sb, int it, int v) {
            const int64_t o = m.block(n) * (R * 64) + ((sb * M::NT + it) * M::V + v) * 512;
            high[n][sb][it][v] = *gld<u32x2>(w + o);
            low[n][sb][it][v] = *gld<u32x2>(w + at.lo + o);
        });
    constexpr float un = kMuGramUnlift;
    // the parts' sums, in order of groups of parts
    constexpr int kChunks = M::kPart / 16, kGroups = kChunks < kMuFewThreads ? kMuFewThreads / kChunks : 1;
    const float* const parts = reinterpret_cast<const float*>(ws + at.part) + static_cast<int64_t>(src) * strips * R * R;
    const int group = threadIdx.x / kChunks;  // (one group: 0 .. 0)
#pragma unroll
    for (int c = threadIdx.x % kChunks; c < kChunks; c += kMuFewThreads) {
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int e = group; e < strips; e += kGroups) s += *gld<f32x4>(parts + static_cast<int64_t>(e) * R * R + c * 4);
        if (kGroups > 1) *(F4*)static_cast<uintptr_t>(m.sums + group * M::kPart + c * 16) = s;
        else m.put_o(c, s, un);
    }
#pragma unroll
    for (int n = 0; n < M::NB; ++n)
        M::each([&](int sb, int it, int v) {
            const uint32_t z = m.place(m.block(n), sb, it, v);
            *(L2*)static_cast<uintptr_t>(z) = high[n][sb][it][v];
            *(L2*)static_cast<uintptr_t>(z + M::kBytes) = low[n][sb][it][v];
        });
    __syncthreads();
    if (kGroups > 1) {
        if (threadIdx.x < kChunks) {
            f32x4 s = *(const F4*)static_cast<uintptr_t>(m.sums + threadIdx.x * 16);
#pragma unroll
            for (int e = 1; e < kGroups; ++e) s += *(const F4*)static_cast<uintptr_t>(m.sums + e * M::kPart + threadIdx.x * 16);
            m.put_o(threadIdx.x, s, un);
        }
        __syncthreads();
    }
    m.poly(poly);
    if (last) {
        const int64_t first = static_cast<int64_t>(b) * t.rows * t.ldx;
#pragma unroll
        for (int n = 0; n < M::NB; ++n)
            m.apply(m.block(n), [&](int sb, int it, int v, const f32x4& y) {
                mu_few_store(t, update, decay, first, it * M::T + m.col, strip * M::kStrip + 32 * m.block(n) + m.column(sb, v),
                             y * (kMuXUnlift * kMuUnlift));
            });
        return;
    }
#pragma unroll
    for (int n = 0; n < M::NB; ++n)
        m.apply(m.block(n), [&](int sb, int it, int v, const f32x4& y) {
            const int64_t o = m.block(n) * (R * 64) + ((sb * M::NT + it) * M::V + v) * 512;
            u32x2 lo;
            *gst<u32x2>(w + o) = m.split(m.block(n), sb, it, v, y, lo);
            *gst<u32x2>(w + at.lo + o) = lo;
        });
    mu_order();
    __syncthreads();  // A's sums have been read; R = 64: X' is read by two waves
    m.gram(M::kStrip / 32);
    __syncthreads();
    float* const o = reinterpret_cast<float*>(ws + at.part) + static_cast<int64_t>((src ^ 1) * strips + strip) * R * R;
    for (int c = threadIdx.x; c < M::kPart / 16; c += kMuFewThreads) *gst<f32x4>(o + c * 4) = m.joined(c);
}

template <class Fn>
void with_rows(int rows, Fn f) {
    if (rows == 16) f(std::integral_constant<int, 16>{});
    else if (rows == 32) f(std::integral_constant<int, 32>{});
    else f(std::integral_constant<int, 64>{});
}

}  // namespace

void launch_mu_few(const MuFewTensors& t, int rows, const MuFewArgs& a, hipStream_t s) {
    with_rows(rows, [&](auto r) {
        const dim3 g(t.blocks), n(kMuFewThreads);
        if (t.n == 1) hipLaunchKernelGGL((k_mu_few<decltype(r)::value, 1>), g, n, 0, s, t.only(), a);
        else hipLaunchKernelGGL((k_mu_few<decltype(r)::value, kMuFewBatch>), g, n, 0, s, t, a);
    });
}

void launch_mu_strip_start(const MuTensors& t, int rows, const MuStepArgs& a, hipStream_t s) {
    with_rows(rows, [&](auto r) {
        const dim3 g(t.blocks), n(kMuFewThreads);
        if (t.n == 1) hipLaunchKernelGGL((k_mu_strip_start<decltype(r)::value, 1>), g, n, 0, s, t.only(), a);
        else hipLaunchKernelGGL((k_mu_strip_start<decltype(r)::value, kMuBatch>), g, n, 0, s, t, a);
    });
}

void launch_mu_strip_step(const MuTensors& t, int rows, const MuPoly& p, int src, bool last, bool update, float decay, hipStream_t s) {
    with_rows(rows, [&](auto r) {
        const dim3 g(t.blocks), n(kMuFewThreads);
        if (t.n == 1) hipLaunchKernelGGL((k_mu_strip_step<decltype(r)::value, 1>), g, n, 0, s, t.only(), p, src, last, update, decay);
        else hipLaunchKernelGGL((k_mu_strip_step<decltype(r)::value, kMuBatch>), g, n, 0, s, t, p, src, last, update, decay);
    });
}

}  // namespace meo
