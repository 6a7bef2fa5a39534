// Orthogonalization and the Muon step of matrices with few values, one block each, all steps in
// one launch: the mathematics and roundings of muon.hip (there each pass over such a matrix is a
// launch of 3 to 5 us, 15 and more in all).
//
// The iterate stays on the CU: its high parts in LDS, its low parts in the registers of the lanes
// that form them. The longer side goes by blocks of 32 columns; a wave's blocks are its own: the step
// X' = a X + B X needs nothing else of X. A = X X^T is summed over them through LDS.
// Every wave then forms B for itself: in an accumulator of a symmetric matrix a lane holds four
// consecutive rows of a column, which are four consecutive values of the contraction of that
// column as an operand, so A, A^2 and B go from product to product in registers.
//
// What bounds it: latencies (barriers, LDS, dependent products) and, for the largest, one CU's way
// to memory.
#include "muon_device.h"

namespace meo {

namespace {

typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) u32x2 L2;
typedef __attribute__((address_space(3))) u32x4 L4;
typedef __attribute__((address_space(3))) f32x4 F4;

constexpr int kMuFewWaves = kMuFewThreads / 64;

// An LDS access of a wave to what its other lanes wrote is not moved over this.
__device__ __forceinline__ void mu_order() { __asm__ volatile("" ::: "memory"); }

// A matrix of R rows. Accumulators: tiles of T x T, where a lane holds rows 8 v + 4 h + 0 .. 3 of its
// column, v < V.
template <int R>
struct MuFew {
    static constexpr int T = R == 16 ? 16 : 32, NT = R / T, V = T == 16 ? 1 : 4, SB = 32 / T;
    static constexpr int kValues = R == 64 ? 49152 : 65536;
    static constexpr int kBlocks = kValues / R / 32 / kMuFewWaves;  // of 32 columns per wave, at most
    static constexpr int kLow = SB * NT * V * 2;  // registers of a block's low parts
    static constexpr int kX = kValues * 2;  // bytes of X
    // A's parts: by wave; R = 64: by pairs of waves, which have a column of tiles each.
    static constexpr int kParts = R == 64 ? kMuFewWaves / 2 : kMuFewWaves;
    static constexpr int kPart = R * R * 4;
    static constexpr int kLds = kX + kParts * kPart * (R == 16 ? 2 : 1);
    typedef uint32_t Low __attribute__((ext_vector_type(R == 16 ? 16 : R == 32 ? 8 : 4)));
    static_assert(kBlocks <= static_cast<int>(sizeof(Low) / 4), "a wave's blocks");
    struct Acc { f32x4 v[V]; };
    struct Op { u32x2 v[V]; };  // T values of the contraction

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
    static __device__ __forceinline__ void zero(Acc& c) {
#pragma unroll
        for (int v = 0; v < V; ++v) c.v[v] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
};

// X in LDS: blocks of 32 columns, R rows of 64 bytes in each, chunk c (16 bytes) of row r at position
// c ^ (r >> 2 & 3): rows read at one chunk touch every bank alike. The bytes of 4 values, chunk c8 >> 1:
__device__ __forceinline__ uint32_t mu_few_at(int r, int c8) {
    return r * 64 + (((c8 >> 1) ^ ((r >> 2) & 3)) << 4) + (c8 & 1) * 8;
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

template <int R, int N>
__global__ __launch_bounds__(kMuFewThreads, 2) void k_mu_few(MuListOf<MuFewTensor, N> l, MuFewArgs a) {
    using M = MuFew<R>;
    constexpr int T = M::T, NT = M::NT, V = M::V, SB = M::SB;
    using Acc = typename M::Acc;
    using Op = typename M::Op;
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
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint32_t x0 = uniform(static_cast<int>(lds_addr(lds))), s0 = x0 + M::kX;

    // the directions and their squares' sum
    for (uint32_t o = threadIdx.x * 16; o < static_cast<uint32_t>(nb) * R * 64; o += kMuFewThreads * 16)
        *(L4*)static_cast<uintptr_t>(x0 + o) = u32x4{0u, 0u, 0u, 0u};
    constexpr int kTurn = kMuFewThreads * kVec;
    static_assert(M::kValues <= 16 * kTurn, "a thread's values");
    const int turns = uniform((size + kTurn - 1) / kTurn);
    u32x16 u[kVec];  // [e][turn]; turns and blocks are indexed at run time, which keeps the code short
    double sum = 0.0;
#pragma unroll 1
    for (int p = 0; p < turns; ++p) {
        const int i = p * kTurn + threadIdx.x * kVec;
        float w[kVec];
        mu_take8(t, a.step, b, static_cast<int64_t>(b) * size, i, clamp_valid(static_cast<int64_t>(size) - i), w);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            sum += static_cast<double>(w[e]) * static_cast<double>(w[e]);
            u[e][p] = __float_as_uint(w[e]);
        }
    }
    sum = wave_sum(sum);
    typedef __attribute__((address_space(3))) double D1;
    if (lane == 0) *(D1*)static_cast<uintptr_t>(s0 + wave * 8) = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < kMuFewWaves; ++w) sum += *(const D1*)static_cast<uintptr_t>(s0 + w * 8);
    const double f = mu_factor_of(sum, a.step.eps, s.lift);

    // X0 in two parts: the low ones through LDS to the lanes that keep them, then the high ones
    auto scatter = [&](bool low) {
#pragma unroll 1
        for (int p = 0; p < turns; ++p) {
            const int i = p * kTurn + threadIdx.x * kVec;
            uint32_t w[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                uint32_t hi, lo;
                mu_split(static_cast<float>(__uint_as_float(u[e][p]) * f), hi, lo);
                w[e] = low ? lo : hi;
            }
            if (i >= size) continue;
            int row = static_cast<uint32_t>(i) / static_cast<uint32_t>(t.cols), col = i - row * t.cols;
            if (!t.tall && col % kVec == 0 && col + kVec <= t.cols) {
                *(L4*)static_cast<uintptr_t>(x0 + (col >> 5) * (R * 64) + mu_few_at(row, (col & 31) >> 2)) =
                    u32x4{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
                continue;
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const int r = t.tall ? col : row, c = t.tall ? row : col;
                if (i + e < size)
                    *(__attribute__((address_space(3))) uint16_t*)static_cast<uintptr_t>(
                        x0 + (c >> 5) * (R * 64) + mu_few_at(r, (c & 31) >> 2) + (c & 3) * 2) = static_cast<uint16_t>(w[e]);
                if (++col == t.cols) {
                    col = 0;
                    ++row;
                }
            }
        }
    };
    scatter(true);
    __syncthreads();
    const int col = lane & (T - 1), h = lane / T;
    // of an accumulator's (or its low part's) four values v in block `blk`, part sb, tile it
    auto place = [&](int blk, int sb, int it, int v) {
        return x0 + blk * (R * 64) + mu_few_at(it * T + col, T == 16 ? 4 * sb + h : 2 * v + h);
    };
    const int mine = uniform((nb - wave + kMuFewWaves - 1) / kMuFewWaves);  // (nb < wave: 0)
    typename M::Low low[M::kLow];  // [..][block]
#pragma unroll 1
    for (int n = 0; n < mine; ++n)
#pragma unroll
        for (int sb = 0; sb < SB; ++sb)
#pragma unroll
            for (int it = 0; it < NT; ++it)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const u32x2 w = *(const L2*)static_cast<uintptr_t>(place(n * kMuFewWaves + wave, sb, it, v));
                    const int e = ((sb * NT + it) * V + v) * 2;
                    low[e][n] = w.x;
                    low[e + 1][n] = w.y;
                }
    __syncthreads();
    scatter(false);
    __syncthreads();

    const float lift = ldexpf(1.0f, s.lift), un = 1.0f / (lift * lift), out = 1.0f / lift * kMuUnlift;
    const int64_t first = static_cast<int64_t>(b) * t.rows * t.ldx;
    const int part = R == 64 ? wave >> 1 : wave;
#pragma unroll 1
    for (int step = 0; step < a.steps; ++step) {
        const MuPoly p = a.poly[step];
        // A over the wave's blocks
        const uint32_t sp = s0 + (R == 16 ? (step & 1) * M::kParts * M::kPart : 0);
        {
            Acc g[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) M::zero(g[i]);
            for (int blk = part; blk < nb; blk += M::kParts) {
                const uint32_t o = x0 + blk * (R * 64);
                if constexpr (T == 16) {
                    const half8 w = __builtin_bit_cast(half8, mu_lds(o + mu_few_at(col, 2 * h)));
                    g[0].v[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, w, g[0].v[0], 0, 0, 0);
                } else {
                    const int tj = R == 64 ? wave & 1 : 0;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        u32x4 w[NT];
#pragma unroll
                        for (int i = 0; i < NT; ++i) w[i] = mu_lds(o + mu_few_at(i * T + col, 4 * c + 2 * h));
                        const u32x4 z = NT == 1 || tj == 0 ? w[0] : w[NT - 1];
#pragma unroll
                        for (int i = 0; i < NT; ++i) g[i] = __builtin_bit_cast(Acc, mfma_f16(w[i], z, __builtin_bit_cast(f32x16, g[i])));
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    *(F4*)static_cast<uintptr_t>(sp + part * M::kPart + ((((R == 64 ? wave & 1 : 0) * NT + i) * V + v) * 64 + lane) * 16) = g[i].v[v];
        }
        __syncthreads();
        // the parts' sums, in order: [column of tiles][row][v][lane]
        auto joined = [&](int chunk) {
            f32x4 w = *(const F4*)static_cast<uintptr_t>(sp + chunk * 16);
#pragma unroll
            for (int e = 1; e < M::kParts; ++e) w += *(const F4*)static_cast<uintptr_t>(sp + e * M::kPart + chunk * 16);
            return w;
        };
        Acc A[NT][NT];  // [column][row]
        if constexpr (R == 16) {
            A[0][0].v[0] = joined(lane);
        } else {
            for (int c = threadIdx.x; c < M::kPart / 16; c += kMuFewThreads) {
                const f32x4 w = joined(c);
                *(F4*)static_cast<uintptr_t>(sp + c * 16) = w;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int v = 0; v < V; ++v) A[j][i].v[v] = *(const F4*)static_cast<uintptr_t>(sp + (((j * NT + i) * V + v) * 64 + lane) * 16);
        }
        // O 2^8 times and the diagonal d of the lane's columns
        const int holder = col + T * ((col >> 2) & (64 / T - 1));  // the lane with the diagonal of column `col`
        Op O[NT][NT], B[NT][NT];
        float d[NT], q[NT], tl[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float own = 0.0f;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    f32x4 w = A[j][i].v[v] * un;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (i == j && 8 * v + 4 * h + e == col) {
                            own = w[e];
                            w[e] = 0.0f;
                        }
                    w *= kMuLift;
                    O[j][i].v[v] = mu_pack4(w.x, w.y, w.z, w.w);
                }
            d[j] = __shfl(own, holder, 64);
        }
        // B 2^8 times off the diagonal, q = a + B_ii
        const float cs = p.c * kMuUnlift;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            f32x4 di[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < 4; ++e) di[v][e] = __shfl(d[i], 8 * v + 4 * h + e, 64);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                Acc sq;
                M::zero(sq);
#pragma unroll
                for (int z = 0; z < NT; ++z) M::mul(sq, O[i][z], O[j][z]);
                float own = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] = fmaf(mu_half(O[j][i].v[v], e), fmaf(p.c, di[v][e] + d[j], p.b), sq.v[v][e] * cs);
                        if (i == j && 8 * v + 4 * h + e == col) {
                            own = p.a + fmaf(p.b, d[j], p.c * fmaf(d[j], d[j], sq.v[v][e] * (kMuUnlift * kMuUnlift)));
                            y[e] = 0.0f;
                        }
                    }
                    B[j][i].v[v] = mu_pack4(y[0], y[1], y[2], y[3]);
                }
                if (i == j) {
                    const float al = p.a * kMuLift;
                    q[j] = __shfl(own, holder, 64) * kMuLift;
                    tl[j] = fmaf(q[j] - al, fminf(d[j] * d[j], 1.0f), al);
                }
            }
        }
        // X' of the wave's blocks
        const bool last = step + 1 == a.steps;
#pragma unroll 1
        for (int n = 0; n < mine; ++n) {
            const int blk = n * kMuFewWaves + wave;
            mu_order();
#pragma unroll
            for (int sb = 0; sb < SB; ++sb) {
                Op x[NT];  // X^T's part: 4 rows of X of the lane's column each
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        x[i].v[v] = mu_lds_tr(x0 + blk * (R * 64) + mu_few_at(i * T + 8 * v + 4 * h + ((lane >> 2) & 3),
                                                                           T == 16 ? 4 * sb + (lane & 3) : ((lane >> 4) & 1) * 4 + (lane & 3)));
                mu_order();
#pragma unroll
                for (int it = 0; it < NT; ++it) {
                    Acc c;
                    M::zero(c);
#pragma unroll
                    for (int i = 0; i < NT; ++i) M::mul(c, x[i], B[it][i]);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const uint32_t at = place(blk, sb, it, v);
                        const int reg = ((sb * NT + it) * V + v) * 2;
                        const u32x2 xh = *(const L2*)static_cast<uintptr_t>(at), xl = {low[reg][n], low[reg + 1][n]};
                        f32x4 y;  // 2^8 X'
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = fmaf(tl[it], mu_half(xl, e), fmaf(q[it], mu_half(xh, e), c.v[v][e]));
                        if (last) {
                            mu_few_store(t, a.update, a.decay, first, it * T + col, 32 * blk + 16 * (T == 16 ? sb : 0) + 8 * v + 4 * h, y * out);
                        } else {
                            y *= kMuUnlift;
                            const u32x2 w = mu_pack4(y.x, y.y, y.z, y.w);
                            *(L2*)static_cast<uintptr_t>(at) = w;
                            const u32x2 z = mu_pack4(y.x - mu_half(w, 0), y.y - mu_half(w, 1), y.z - mu_half(w, 2), y.w - mu_half(w, 3));
                            low[reg][n] = z.x;
                            low[reg + 1][n] = z.y;
                        }
                    }
                }
            }
        }
        mu_order();
        if (R != 16) __syncthreads();  // (A's sums have been read; R = 64: X' is read by two waves)
    }
}

}  // namespace

void launch_mu_few(const MuFewTensors& t, int rows, const MuFewArgs& a, hipStream_t s) {
    const dim3 g(t.blocks), n(kMuFewThreads);
    auto go = [&](auto r) {
        constexpr int R = decltype(r)::value;
        if (t.n == 1) hipLaunchKernelGGL((k_mu_few<R, 1>), g, n, 0, s, t.only(), a);
        else hipLaunchKernelGGL((k_mu_few<R, kMuFewBatch>), g, n, 0, s, t, a);
    };
    if (rows == 16) go(std::integral_constant<int, 16>{});
    else if (rows == 32) go(std::integral_constant<int, 32>{});
    else go(std::integral_constant<int, 64>{});
}

}  // namespace meo
