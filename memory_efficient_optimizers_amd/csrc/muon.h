// Orthogonalization by Newton-Schulz steps and the Muon step: descriptors and launchers
// shared by muon.hip and the C ABI.
#pragma once
#include "internal.h"

namespace meo {

constexpr int kMuPad = 64;         // both sides of a matrix in the workspace are multiples of it
constexpr int kMuBatch = 16;       // tensors per launch (their descriptors are kernel arguments)
constexpr int kMuThreads = 256;    // momentum and scatter passes
constexpr int kMuTile = 64;        // scatter pass: square tiles of the matrix in the workspace
constexpr int64_t kMuPart = 2048;  // values per part of the momentum pass, up to kMuMaxParts of them
constexpr int64_t kMuMaxParts = 1024;
constexpr int64_t kMuMaxSide = 1 << 22;  // longer side of a matrix (32-bit offsets in a tile)
// The workspace holds X times 2^12. Its entries are at most 8, as its singular values are (check_ns_hp in
// abi.cpp refuses coefficients otherwise), so 2^15 there, below fp16's 65504. Two fp16 parts, whose
// smallest step is 2^-24, then hold X to 2^-37: 22 bits of an entry above 2^-14. (With a smaller power,
// entries from 1/8 of an orthonormal matrix' down lost bits, and every step multiplies what is lost by the
// linear coefficient: 64 x 64 with one strong entry over 1e-6 of noise, times 2^3, was 9.8e-5 off, 2.4e-3 after
// ten steps.)
constexpr float kMuXLift = 4096.0f, kMuXUnlift = 1.0f / 4096, kMuGramUnlift = kMuXUnlift * kMuXUnlift;
constexpr double kMuMaxSingular = 8.0, kMuMinSingular = 1.0 / 64;  // of the largest singular value, between steps
static_assert(kMuXLift * kMuMaxSingular <= 32768.0, "half of fp16's range, for roundings");

// What the passes over the caller's tensors need of one of them ([batch] matrices).
struct MuTensor {
    const void* g;    // gradient, or the matrices to orthogonalize
    void* m;          // momentum (null: orthogonalize)
    float* ms;        // scales of an 8-bit momentum
    void* x;          // parameter, or the result
    uint8_t* ws;      // workspace of the first matrix
    double* norm;     // [batch][parts] sums of squares
    int64_t ldg, ldx; // elements between rows of g and x
    int64_t stride;   // bytes of workspace per matrix
    int32_t rows, cols, batch;
    int32_t mp, np;   // padded shorter and longer side
    int32_t parts, tiles_per_part;  // of the momentum pass: kMuPart values per tile
    float coef;       // Muon: lr times the scale of the matrix' shape
    int16_t gbf16, xbf16, mkind;  // mkind: Storage of m (0 fp32, 1 bf16, 2 int8)
    int16_t tall;     // rows > cols: the workspace holds the transpose
};

// What a product needs of one tensor.
struct MuMatrix {
    uint8_t* ws;
    int64_t stride;
    int32_t mp, np, batch;
    int32_t parts, steps;  // A = X X^T: parts of the contraction, steps of 64 in each
};

// The blocks of a launch, by tensor: those before tensor i > 0 in first[i] (past the last one
// nothing is reached: 2^32 - 1), all in `blocks`. N = 1: one tensor alone (kernels are compiled for
// it too, see mu_find).
template <class T, int N>
struct MuListOf {
    int32_t n;
    uint32_t blocks;
    uint32_t first[N];
    T d[N];
    MuListOf<T, 1> only() const { return MuListOf<T, 1>{1, blocks, {0}, {d[0]}}; }
};
using MuTensors = MuListOf<MuTensor, kMuBatch>;
using MuMatrices = MuListOf<MuMatrix, kMuBatch>;

// Matrices in the workspace lie in blocks of 64 rows x 32 columns, 4 KB each, the blocks of a row of
// blocks one after the other: what a tile takes of 32 values of the contraction is then whole
// kilobytes, along rows and down columns. (Row-major, a transfer touched 16 rows, each in a page of
// its own where they are long.) Elements before row r (a multiple of 32) of column 0:
__host__ __device__ constexpr int64_t mu_rows(int64_t r, int64_t cols) { return (r / 64 * (cols / 32) * 64 + r % 64) * 32; }

// A matrix in the workspace (offsets in bytes): two buffers of X's high parts and one of the
// low parts ([mp][np] fp16), off-diagonal A and B ([mp][mp] fp16), the diagonal of A and
// the row factors a + B_ii ([mp] fp32), what the low parts add to the diagonal (two buffers of [mp] int32,
// mu_fix), partial sums of A.
struct MuPlace {
    int64_t x, lo, a, b, d, q, e, part, total;
    __host__ __device__ MuPlace(int64_t mp, int64_t np, int64_t parts) {
        const int64_t s = mp * mp * 2;
        x = mp * np * 2;
        lo = 2 * x;
        a = 3 * x;
        b = a + s;
        d = b + s;
        q = d + mp * 4;
        e = q + mp * 4;
        part = (e + 2 * mp * 4 + 255) / 256 * 256;
        total = part + (parts > 1 ? parts * mp * mp * 4 : 0);
    }
    __host__ __device__ int64_t hi(int buffer) const { return buffer ? x : 0; }
    __host__ __device__ int64_t low(int buffer, int64_t mp) const { return e + buffer * mp * 4; }  // of the diagonal, beside hi(buffer)
};

struct MuStepArgs {   // momentum pass and scatter
    float beta, omb;  // momentum weight and 1 - it
    int32_t nesterov;
    double eps;
};

struct MuPoly {       // X <- a X + (b A + c A^2) X
    float a, b, c;
};

// Square tiles of a product.
enum MuForm { kMuSmall = 0, kMuMedium, kMuThreeQuarters, kMuLarge, kMuForms };
constexpr int kMuFormTile[kMuForms] = {64, 128, 192, 256};
constexpr int kMuTileThreads = 256;

template <int N>
struct MuLastOf {     // the last step's results go to the caller's tensors
    MuListOf<MuTensor, N> t;
    float decay;      // 1 - lr wd
    int32_t update;   // a parameter's update (else bf16 results)
};
using MuLast = MuLastOf<kMuBatch>;

// ---- matrices with few rows

// A matrix whose shorter side is at most 64 takes 16, 32 or 64 rows, and its longer side strips of
// mu_strip columns, one to a thread block: of one strip, all steps are one launch; of up to 64 (32 of
// 64 rows), a launch each. The rows; 0: the matrix is worked on in tiles. From the matrix
// alone: its result does not depend on the list.
__host__ __device__ constexpr int mu_strip(int rows) { return rows == 64 ? 256 : 512; }
__host__ __device__ constexpr int mu_few(int64_t m, int64_t n) {
    return m <= 16 && n <= 64 * mu_strip(16) ? 16 : m <= 32 && n <= 64 * mu_strip(32) ? 32 : m <= 64 && n <= 32 * mu_strip(64) ? 64 : 0;
}
// The workspace of one in strips (np: whole strips): the iterate's high and low parts, and two buffers
// of the strips' parts of A.
struct MuStripPlace {
    int64_t lo, part, total;
    __host__ __device__ MuStripPlace(int64_t rows, int64_t np, int64_t strips) {
        lo = rows * np * 2;
        part = 2 * lo;
        total = part + 2 * strips * rows * rows * 4;
    }
};
constexpr int kMuFewBatch = 48;     // tensors per launch
constexpr int kMuFewThreads = 512;

struct MuFewTensor {  // fields as MuTensor's
    const void* g;
    void* m;
    float* ms;
    void* x;
    int32_t ldg, ldx, rows, cols, batch;
    float coef;
    int16_t gbf16, xbf16, mkind;
};
using MuFewTensors = MuListOf<MuFewTensor, kMuFewBatch>;

struct MuFewArgs {
    MuStepArgs step;
    float decay;
    int32_t update, steps;
    MuPoly poly[16];
};

// rows: 16, 32 or 64, the same for all. Of one strip; of several (after the momentum pass: X0 and its
// A, then the steps; src: the buffer of A's parts).
void launch_mu_few(const MuFewTensors& t, int rows, const MuFewArgs& a, hipStream_t s);
void launch_mu_strip_start(const MuTensors& t, int rows, const MuStepArgs& a, hipStream_t s);
void launch_mu_strip_step(const MuTensors& t, int rows, const MuPoly& p, int src, bool last, bool update, float decay, hipStream_t s);

void launch_mu_momentum(const MuTensors& t, const MuStepArgs& a, hipStream_t s);
void launch_mu_scatter(const MuTensors& t, const MuStepArgs& a, hipStream_t s);
// A's off-diagonal part and diagonal from X (buffer src); with parts (kMuSmall only), their sums
// and the join.
void launch_mu_gram(const MuMatrices& m, int form, int src, hipStream_t s);
void launch_mu_join(const MuMatrices& m, hipStream_t s);
// B = b A + c A^2 off the diagonal, a + B_ii on it.
void launch_mu_poly(const MuMatrices& m, int form, const MuPoly& p, hipStream_t s);
// X' = a X + B X, into the other buffer or, `last` given, the caller's tensors. linear: a.
void launch_mu_apply(const MuMatrices& m, int form, int src, float linear, const MuLast* last, hipStream_t s);

}  // namespace meo
