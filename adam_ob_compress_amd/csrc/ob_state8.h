// ob_state8.h -- device side of the 8-bit state format (the rules are in ob_adam.h) and of gradients
// at any alignment.
//
// The codes are square-law: an m is c|c| q, a v is (k^2 q)^2.  Decoding costs two to three products; the
// root that encoding needs is one v_sqrt_f32 per value.  That root is good to a few ulp, so it gives the
// code or the one below it (its argument is lowered by 2^-13, far above its error and far below the
// distance of two borders), and one comparison with the next border, which is an fp32 number by the format's rule,
// settles which.  All values here are fp32 in single IEEE operations, so the codes are the same
// wherever they are computed.
#pragma once

#include "ob_adamw.h"
#include "ob_device.h"

namespace ob {
namespace {

constexpr float kQuantM = 1.0f / 16129.0f;   // 1 / 127^2, rounded to fp32
constexpr float kQuantV = 1.0f / 65025.0f;   // 1 / 255^2
constexpr uint32_t kTinyBits = 0x0f800000u;  // 2^-96
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr float kBelow = 1.0f / 8192.0f;

// Largest value over the wave's 64 lanes, in every lane (a scalar register): maxima over pairs, quads,
// half rows and rows by DPP, then rows joined by row broadcasts into lane 63.  All lanes active.
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
#define OB_DPP_MAX(ctrl, rows)                                                                             \
    {                                                                                                      \
        const uint32_t y = static_cast<uint32_t>(                                                          \
            __builtin_amdgcn_update_dpp(static_cast<int>(x), static_cast<int>(x), ctrl, rows, 0xF, false)); \
        x = x > y ? x : y;                                                                                 \
    }
    OB_DPP_MAX(0xB1, 0xF)    // quad_perm [1,0,3,2]
    OB_DPP_MAX(0x4E, 0xF)    // quad_perm [2,3,0,1]
    OB_DPP_MAX(0x141, 0xF)   // row_half_mirror
    OB_DPP_MAX(0x140, 0xF)   // row_mirror
    OB_DPP_MAX(0x142, 0xA)   // row_bcast:15 into rows 1 and 3
    OB_DPP_MAX(0x143, 0xC)   // row_bcast:31 into rows 2 and 3
#undef OB_DPP_MAX
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), 63));
}

// Single operations, never fused with a neighbour: the format's rules round each of them.
__device__ __forceinline__ float mul(float a, float b)
{
#pragma clang fp contract(off)
    return a * b;
}

__device__ __forceinline__ float sub(float a, float b)
{
#pragma clang fp contract(off)
    return a - b;
}

// The format's scale from the bits of the block's largest magnitude.  (top as unsigned bits: NaN above
// infinity above every number, so neither is lost in the maximum.)
template <bool V>
__device__ __forceinline__ float block_scale(uint32_t top)
{
    const float t = __uint_as_float(top);
    const float q = V ? mul(sqrtf(t), kQuantV) : mul(t, kQuantM);
    return top >= kInfBits ? __uint_as_float(0x7fc00000u) : top < kTinyBits ? 0.0f : q;
}

// 1/q for the first guess of a code (0 where the block has no codes)
__device__ __forceinline__ float guess_scale(float q) { return q > 0.0f ? __builtin_amdgcn_rcpf(q) : 0.0f; }

// value of code k >= 0 (also of the half-way borders k - 1/2)
template <bool V>
__device__ __forceinline__ float code_value(float k, float q)
{
    const float r = mul(mul(k, k), q);
    return V ? mul(r, r) : r;
}

// |code| of x >= 0 as a float; rq: guess_scale(q); bits: 16 random bits (SR).  root_x: about sqrt(x) (V).
template <bool V, bool SR>
__device__ __forceinline__ float encode(float x, float root_x, float q, float rq, uint32_t bits)
{
    constexpr float most = V ? 255.0f : 127.0f;
    const float y = __builtin_amdgcn_sqrtf(V ? root_x * rq : x * rq);
    float k;
    if (!SR) {
        k = floorf(y + (0.5f - kBelow));
        k += x >= code_value<V>(k + 0.5f, q) ? 1.0f : 0.0f;
    } else {
        k = fmaxf(floorf(y - kBelow), 0.0f);
        float low = code_value<V>(k, q), high = code_value<V>(k + 1.0f, q);
        if (x >= high) {
            k += 1.0f;
            low = high;
            high = code_value<V>(k + 1.0f, q);
        }
        const float u = static_cast<float>(bits);
        k += mul(u, sub(high, low)) < mul(sub(x, low), 65536.0f) ? 1.0f : 0.0f;
        k = fminf(k, most);
    }
    if (V) k = x > 0.0f ? fmaxf(k, 1.0f) : 0.0f;
    return q > 0.0f ? k : 0.0f;
}

__device__ __forceinline__ float decode_m(uint32_t biased_byte, float q)
{
    const float c = static_cast<float>(biased_byte) - 128.0f;
    return mul(c * fabsf(c), q);
}

__device__ __forceinline__ float decode_v(uint32_t byte, float q) { return code_value<true>(static_cast<float>(byte), q); }

// m codes are int8; the bytes are handled with 128 added (one exclusive-or per four of them)
constexpr uint32_t kBias4 = 0x80808080u;

__device__ __forceinline__ uint32_t byte_of(uint32_t w, int j) { return (w >> (8 * j)) & 0xffu; }

__device__ __forceinline__ uint32_t put_byte(float k, int j, uint32_t w)
{
    return __builtin_amdgcn_cvt_pk_u8_f32(k, j, w);
}

}  // namespace
}  // namespace ob
