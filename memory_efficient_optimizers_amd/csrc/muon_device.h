// What the kernels of muon.hip and muon_small.hip share: the caller's tensors, fp16 values, LDS.
#pragma once
#include "muon.h"
#include "mx4_tile.h"

namespace meo {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));

constexpr float kMuLift = 256.0f;        // of O and B
constexpr float kMuUnlift = 1.0f / 256;

__device__ __forceinline__ f32x16 mfma_f16(const u32x4& a, const u32x4& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

// The tensor of block `id`. Kernel arguments are a microsecond away, so all counts are read at
// once, and a tensor alone (N = 1) needs none.
template <class T, int N>
__device__ __forceinline__ int mu_find(const MuListOf<T, N>& l, uint32_t id) {
    int k = 0;
#pragma unroll
    for (int i = 1; i < N; ++i) k += id >= l.first[i];
    return k;
}
// Its number among the tensor's blocks.
template <class T, int N>
__device__ __forceinline__ uint32_t mu_item(const MuListOf<T, N>& l, int k, uint32_t id) {
    return N == 1 ? id : id - l.first[k];
}

// Element (r, c) of a matrix of `cols` columns in the workspace.
__device__ __forceinline__ int64_t mu_at(int r, int c, int cols) {
    return (static_cast<int64_t>(r >> 6) * (cols >> 5) + (c >> 5)) * 2048 + (r & 63) * 32 + (c & 31);
}

// ----------------------------------------------------------------------------- the caller's tensors

// 8 values of matrix b of the gradient (or input) from element i of its rows on, the first
// `valid` of them.
__device__ __forceinline__ void mu_load_g(const MuTensor& t, int b, int64_t i, int valid, float* f) {
    const int64_t at = static_cast<int64_t>(b) * t.rows * t.ldg;
    if (t.ldg == t.cols) {
        load_any8(t.g, at + i, valid, t.gbf16, f);
        return;
    }
    const int64_t r = i / t.cols;
    const int c = static_cast<int>(i - r * t.cols);
    if (c + kVec <= t.cols) {
        load_any8(t.g, at + r * t.ldg + c, valid, t.gbf16, f);
        return;
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        f[e] = 0.0f;
        if (e >= valid) continue;
        const int64_t re = (i + e) / t.cols, j = at + re * t.ldg + (i + e - re * t.cols);
        f[e] = t.gbf16 ? __uint_as_float(static_cast<uint32_t>(*gld<uint16_t>(static_cast<const uint16_t*>(t.g) + j)) << 16)
                       : *gld<float>(static_cast<const float*>(t.g) + j);
    }
}

// 8 values of the momentum at element i of the whole tensor.
__device__ __forceinline__ void mu_load_m(const MuTensor& t, int64_t i, int valid, float* f) {
    if (t.mkind != 2) {
        load_any8(t.m, i, valid, t.mkind == 1, f);
        return;
    }
    const int8_t* p = static_cast<const int8_t*>(t.m) + i;
    typedef u32x2 u32x2_any __attribute__((aligned(1)));
    u32x2 w = {0u, 0u};
    if (valid == kVec) {
        w = *gld<u32x2_any>(p);
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            if (e < valid) w[e >> 2] |= static_cast<uint32_t>(*gld<uint8_t>(p + e)) << (8 * (e & 3));
    }
    const float s0 = valid > 0 ? *gld<float>(t.ms + (i >> 7)) : 0.0f;
    const float s1 = valid > 0 ? *gld<float>(t.ms + ((i + valid - 1) >> 7)) : 0.0f;  // 8 values touch two groups at most
#pragma unroll
    for (int e = 0; e < kVec; ++e)
        f[e] = static_cast<float>(static_cast<int8_t>(w[e >> 2] >> (8 * (e & 3)))) * (((i + e) >> 7) == (i >> 7) ? s0 : s1);
}

// As quant_i8x8, with the scale as max|m| times the float32 1/127, which is what torch makes of a division by a
// number on the GPU (4.7% of quotients by 127 differ from it in the last bit): a momentum quantized with elementary
// torch operations then has the same codes, those next to a border too.
__device__ __forceinline__ void mu_quantize8(float* m, uint32_t& lo, uint32_t& hi, float& scale) {
    float a = 0.0f;
#pragma unroll
    for (int e = 0; e < kVec; ++e) a = max_nan(a, fabsf(m[e]));
    a = max_nan(a, dpp<0xb1>(a));   // over the 16 lanes of a group: swap neighbours,
    a = max_nan(a, dpp<0x4e>(a));   // swap pairs,
    a = max_nan(a, dpp<0x141>(a));  // mirror halves,
    a = max_nan(a, dpp<0x140>(a));  // mirror the row
    scale = a * (1.0f / 127.0f);
    const bool ok = scale > 0.0f && scale <= 3.402823466e38f;  // finite and nonzero
    if (!(scale <= 3.402823466e38f)) scale = __builtin_nanf("");
    lo = hi = 0u;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        const float q = fminf(fmaxf(ok ? rintf(m[e] / scale) : 0.0f, -128.0f), 127.0f);
        const uint32_t byte = static_cast<uint32_t>(static_cast<int32_t>(q)) & 0xffu;
        if (e < 4) lo |= byte << (8 * e); else hi |= byte << (8 * (e - 4));
        m[e] = q * scale;
    }
}

// The direction from the gradient and the stored momentum.
__device__ __forceinline__ void mu_direction(const MuStepArgs& a, const float* g, const float* m, float* u) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) u[e] = a.nesterov ? g[e] * a.omb + m[e] * a.beta : m[e];
}

// 8 values of matrix b from element i of it on, the first `valid` of them: the momentum's update
// (every lane of the wave calls it) and the direction, or the values themselves. base: the matrix'
// first element.
__device__ __forceinline__ void mu_take8(const MuTensor& t, const MuStepArgs& a, int b, int64_t base, int64_t i, int valid, float* u) {
    float g[kVec];
    if (valid > 0) mu_load_g(t, b, i, valid, g);
    else
#pragma unroll
        for (int e = 0; e < kVec; ++e) g[e] = 0.0f;
    if (!t.m) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) u[e] = g[e];
        return;
    }
    float m[kVec];
    mu_load_m(t, base + i, valid, m);
#pragma unroll
    for (int e = 0; e < kVec; ++e) m[e] = m[e] * a.beta + g[e] * a.omb;
    if (t.mkind == 2) {
        uint32_t lo, hi;
        float scale;
        mu_quantize8(m, lo, hi, scale);
        store_i8x8(t.m, t.ms, base + i, valid, (reinterpret_cast<uintptr_t>(t.m) & 7) == 0, lo, hi, scale);
    } else if (valid > 0) {
        if (t.mkind == 1)
#pragma unroll
            for (int e = 0; e < kVec; ++e) m[e] = round_bf16(m[e]);
        store_any8(t.m, base + i, valid, t.mkind == 1, m);
    }
    mu_direction(a, g, m, u);
}

// 2^12 / max(norm, eps); a norm that is not finite gives NaN, one of zero 0 (1 / eps need not be finite).
__device__ __forceinline__ double mu_factor_of(double squares, double eps) {
    const double norm = sqrt(squares), top = norm > eps ? norm : eps;
    return !(norm <= 1.7976931348623157e308) ? __builtin_nan("") : norm > 0.0 ? static_cast<double>(kMuXLift) / top : 0.0;
}

// What the low parts add to a row's norm: 2 sum of hi lo (lo^2 is 2^-24 of hi^2 and less), X times 2^12, in
// fixed point: integers, so that neither the order of the sum nor the tiles change it. Of d at most 64 it
// is 2^-10 and less, here 2^27; a summand is rounded by 2^-33 of X's own unit. (Of a row with a NaN: anything
// finite, the product has the NaN.)
constexpr float kMuFixed = 256.0f;  // of hi lo
__device__ __forceinline__ int mu_fix(float v) {
    return static_cast<int>(rintf(fminf(fmaxf(v * kMuFixed, -1073741824.0f), 1073741824.0f)));
}
__device__ __forceinline__ float mu_unfix(int v) { return static_cast<float>(v) * (2.0f / kMuFixed); }
// Lanes 0 .. 31: the sum with lane + 32.
__device__ __forceinline__ uint32_t mu_halves(uint32_t v) {
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return p[0] + p[1];
}
__device__ __forceinline__ void mu_fixed_add(int32_t* p, uint32_t v) {
    __hip_atomic_fetch_add(gst<uint32_t>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ----------------------------------------------------------------------------- fp16 values, LDS

__device__ __forceinline__ void mu_split(float v, uint32_t& hi, uint32_t& lo) {
    const _Float16 h = static_cast<_Float16>(v);
    const _Float16 r = static_cast<_Float16>(v - static_cast<float>(h));
    hi = __builtin_bit_cast(uint16_t, h);
    lo = __builtin_bit_cast(uint16_t, r);
}

// Four consecutive values as fp16, and one of such a word pair. The values are rounded to fp32
// first: an instruction that multiplies, adds and rounds to fp16 at once, which the compiler takes
// in some variants of a kernel and not in others, made results depend on the tile form.
__device__ __forceinline__ u32x2 mu_pack4(float a, float b, float c, float d) {
    typedef _Float16 half4 __attribute__((ext_vector_type(4)));
    __asm__("" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
    return __builtin_bit_cast(u32x2, half4{static_cast<_Float16>(a), static_cast<_Float16>(b), static_cast<_Float16>(c),
                                           static_cast<_Float16>(d)});
}
__device__ __forceinline__ float mu_half(const u32x2& w, int e) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)))));
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 mu_lds_tr(uint32_t a) {  // 4 rows of a column (16-bit values)
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)static_cast<uintptr_t>(a)));
}
__device__ __forceinline__ u32x4 mu_lds(uint32_t a) {
    return *(const __attribute__((address_space(3))) u32x4*)static_cast<uintptr_t>(a);
}

}  // namespace meo
