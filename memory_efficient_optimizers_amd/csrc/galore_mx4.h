// GaLore's step with MX4 projectors: descriptors and launchers shared by galore_mx4.hip and the C ABI.
#pragma once
#include "galore.h"

namespace meo {

// A projected tensor whose projector is held in MX4 (one copy, [r][d], blocks along d);
// u and ut are unused by its step. The gradient is bf16 (g, gs NULL) or MX4 [D][d] with
// blocks along d (g: its codes, gs: its scales). The planes of N have rows of rp >= r
// values, zero past r.
struct GxDesc : GDesc {
    const uint8_t* uc;  // projector codes [r][16 nb]
    const uint8_t* us;  // projector scales [r][nb]
    const uint8_t* gs;
    int32_t nb;         // blocks along d
    int32_t rp;         // r rounded up to 32: two of the back-projection's sub-steps
    int32_t form;       // projection: GxForm; of an MX4 gradient MxForm
    int32_t tpi;        // back-projection: 64-row tiles of N per item
    float* part;        // kitems > 1: the sums of R's parts, [ks][D][rp]
    int32_t ks, kper;   // parts of the contraction, and steps of kGxStep in each but the last
    int32_t kitem, kitems;  // parts per item, items per tile
};

struct GxTable {
    const GxDesc* desc;
    const int2* items;
};

// Projection with an MX4 projector: tiles of kGxFormRows rows of R, both sides in one launch
// (descriptors [0, nright) right-side ones). kGxAny: bf16 gradients of any shape and alignment;
// kGxDirect: of every tensor d is a multiple of 128 and the rows of the gradient and of the
// scales are aligned (four 4096 x 4096 matrices at rank 256 73 us, in the other form 78). An
// MX4 gradient takes the product's forms (MxForm).
enum GxForm { kGxAny = 0, kGxDirect, kGxForms };
constexpr int kGxFormRows[kGxForms] = {64, 64};
constexpr int kGxStep = 128;  // contraction step
// Items of a tensor: y = tile * kitems + item, of kitem of its ks parts each. Where there are several
// to a tile, R is summed by launch_gx_join (items of kGxJoinChunks times 8 columns of a row), whose
// epilogue is then the projection's.
constexpr int kGxJoinChunks = 256;
void launch_gx_project(const GxTable& t, int64_t n, int nright, const GaArgs& a, int form, hipStream_t s);
void launch_gx_join(const GxTable& t, int64_t n, const GaArgs& a, hipStream_t s);
void launch_gx_project_mx4(const GxTable& t, int64_t n, const GaArgs& a, int form, hipStream_t s);
// Back-projection with an MX4 projector: the U-register kernel for any shape, parameters
// of one dtype; item y = band * btj + chunk, chunks of tpi tiles of N.
void launch_gx_back(const GxTable& t, int64_t n, int nright, const GaArgs& a, bool xbf16, hipStream_t s);

}  // namespace meo
