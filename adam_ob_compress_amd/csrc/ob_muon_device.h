// ob_muon_device.h -- what the kernels of the Muon step share.
#pragma once

#include "ob_any.h"
#include "ob_mfma.h"
#include "ob_muon_kernels.h"

namespace ob {
namespace {

typedef _Float16 h4v __attribute__((ext_vector_type(4)));

// The iteration's polynomial, and the powers of two that its matrices are held times: X in fp16 times 2^9, A and
// B = b A + c A^2 times 2^10.  |X| <= 1.3, |A| <= 1.5 and |B| < 12 throughout, so nothing overflows, and values down to 2^-14 / 2^9 of X keep all
// their bits.  fp16 rounds eight times finer than bf16 at the same rate: X after five iterations is off by 1.2e-3 to 4e-3 (2-norm), in
// bf16 by 1e-2 to 3e-2.
constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScaleX = 512.0f;
constexpr float kGram = 1.0f / 256.0f;      // sums of X X^T (2^18) to A (2^10)
constexpr float kUp = 1.0f / 1024.0f;       // sums of A A (2^20) to 2^10, of B X (2^19) to 2^9

__device__ __forceinline__ bool skips(const MuonCall& c) { return c.control && c.control->skip != 0; }
__device__ __forceinline__ float grad_scale(const MuonCall& c) { return c.control ? c.control->grad_scale : 1.0f; }

// u from the scaled gradient and the new momentum
__device__ __forceinline__ float direction(const MuonCall& c, float g, float m)
{
    return c.nesterov ? static_cast<float>((1.0 - c.momentum) * static_cast<double>(g) + c.momentum * static_cast<double>(m)) : m;
}

__device__ __forceinline__ f4 load4u(const float* p, int64_t i) { return *reinterpret_cast<const f4e*>(p + i); }

// Rate, decay and scale of a matrix's update.
struct Rates {
    float l, d, sx;
    // the new parameter from the old one and 2^9 X
    __device__ __forceinline__ float update(float was, float x) const { return fmaf(-l, fmaf(d, was, sx * x), was); }
};
__device__ __forceinline__ Rates rates_of(const MuonCall& c, const MuonMatrix& mt)
{
    const double R = mt.rows, C = mt.cols, big = R > C ? R : C;
    const double scale = c.scale == OB_MUON_MATCH_RMS ? 0.2 * sqrt(big) : c.scale == OB_MUON_SHAPE && R > C ? sqrt(R / C) : 1.0;
    Rates q;
    q.l = static_cast<float>(c.lr * static_cast<double>(mt.lr_mult) * (c.control ? static_cast<double>(c.control->lr_scale) : 1.0));
    q.d = static_cast<float>(c.wd * static_cast<double>(mt.wd_mult));
    q.sx = static_cast<float>(scale / static_cast<double>(kScaleX));
    return q;
}

}  // namespace
}  // namespace ob
