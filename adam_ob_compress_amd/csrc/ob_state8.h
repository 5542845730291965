// ob_state8.h -- device side of the 8-bit state format (the rules are in ob_adam.h) and of gradients
// at any alignment.
//
// The codes are square-law: an m is c|c| q, a v is (k^2 q)^2, and the borders between codes are fp32 numbers by the
// format's rule, so the codes are the same wherever they are computed.  Taken by comparing with the borders they
// made the vector ALU the bound of the 8-bit step (1e9 bf16 parameters 1867 us, 1690 now, then by HBM; by chance 3131
// and 2527, still by the ALU), so a code is first taken from the hardware's roots, rounded, together with its
// distance from the next border.  Only where a block has an element closer to a border than the roots' error could reach (a
// few blocks in a hundred), or a scale so small that a root may be lost, are its codes settled by the borders themselves.
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
// How close to a border the first guess of a code is not trusted, in codes.  The guess y is off by y times the
// relative error of its parts (1/q and root 1 ulp each, product half an ulp, under a root that halves them; for v
// one root more; the borders' own roundings): at most 3.8e-5 for m (y <= 127) and 8e-5 for v (y <= 255).
constexpr float kNearM = 1.0f / 16384.0f, kNearV = 1.0f / 8192.0f;
// The same for chance, in units of the 16 random bits, around the circle of 65536 of them: below 1.6 for m and 4.2 for v.
constexpr float kNearChanceM = 4.0f, kNearChanceV = 8.0f;
// Scales of v below 2^-63 are settled as well by chance: their code 1 stands for a subnormal q^2, and the hardware's root of
// a subnormal v, which may be due code 2, is 0.  (To nearest that v has code 1: the border to 2 is 5 q^2 > 2^-126.)
constexpr uint32_t kSmallScaleBits = 0x20000000u;  // 2^-63

typedef float f4e __attribute__((ext_vector_type(4), aligned(4)));

// A wave takes spans of S = kSpan state blocks (the step on short lists: of one), four elements of each block per
// lane.  A span's 2 S largest magnitudes (of m and of v) are reduced together: each exchange of half-waves
// or rows leaves half as many registers, so eight values over 64 lanes cost 20 operations.
constexpr int kSpan = 4;
constexpr int kSpanElems = kSpan * kStateBlock;

__device__ __forceinline__ uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }

// a over lanes 0..31 (pairs with the upper half) next to b over lanes 32..63
__device__ __forceinline__ uint32_t fold32(uint32_t a, uint32_t b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    return max_u(r[0], r[1]);
}

// rows (16 lanes) of a: 0, 2 and of b: 1, 3, each with its neighbouring row folded in
__device__ __forceinline__ uint32_t fold16(uint32_t a, uint32_t b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    return max_u(r[0], r[1]);
}

// the largest of each row of 16 lanes, in all of them
__device__ __forceinline__ uint32_t row_max(uint32_t x)
{
#define OB_DPP_MAX(ctrl) \
    x = max_u(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), ctrl, 0xF, 0xF, true)));
    OB_DPP_MAX(0xB1)    // quad_perm [1,0,3,2]
    OB_DPP_MAX(0x4E)    // quad_perm [2,3,0,1]
    OB_DPP_MAX(0x141)   // row_half_mirror
    OB_DPP_MAX(0x140)   // row_mirror
#undef OB_DPP_MAX
    return x;
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

// The root of t in [2^-96, 2^128), correctly rounded: the hardware's root is within one unit, and the residuals
// with its neighbours say which of the three is nearest.
__device__ __forceinline__ float exact_root(float t)
{
    const float s = __builtin_amdgcn_sqrtf(t);
    const float down = __uint_as_float(__float_as_uint(s) - 1u), up = __uint_as_float(__float_as_uint(s) + 1u);
    float r = fmaf(-down, s, t) <= 0.0f ? down : s;
    return fmaf(-up, s, t) > 0.0f ? up : r;
}

// The scales of a span's blocks.  tm, tv: per block the lane's largest magnitude as unsigned bits (NaN above
// infinity above every number, so neither is lost in a maximum).  Two registers hold the eight scales, each in
// a row of 16 lanes: rows 0, 1 of a the m of blocks 0, 1, rows 2, 3 their v; b blocks 2, 3.  (One block: its m in
// rows 0, 1 of a, its v in rows 2, 3.)
struct SpanScales {
    float a, b;
    __device__ __forceinline__ float get(int j, bool v) const   // uniform
    {
        return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(j < 2 ? a : b), (v ? 32 : 0) + 16 * (j & 1)));
    }
};

__device__ __forceinline__ float block_scale(uint32_t top, bool v)
{
    const float t = __uint_as_float(top);
    const float q = v ? mul(exact_root(t), kQuantV) : mul(t, kQuantM);
    return top >= kInfBits ? __uint_as_float(0x7fc00000u) : top < kTinyBits ? 0.0f : q;
}

template <int S>
__device__ __forceinline__ SpanScales span_scales(const uint32_t tm[S], const uint32_t tv[S])
{
    static_assert(S == 1 || S == 4, "spans of one or four blocks");
    const bool v = (threadIdx.x & 32) != 0;
    const uint32_t first = fold32(tm[0], tv[0]);
    SpanScales s{};
    s.a = block_scale(row_max(fold16(first, S == 1 ? first : fold32(tm[S / 4], tv[S / 4]))), v);
    if (S == 4) s.b = block_scale(row_max(fold16(fold32(tm[S / 2], tv[S / 2]), fold32(tm[S - 1], tv[S - 1]))), v);
    return s;
}

// value of code k >= 0 (also of the half-way borders k - 1/2)
template <bool V>
__device__ __forceinline__ float code_value(float k, float q)
{
    const float r = mul(mul(k, k), q);
    return V ? mul(r, r) : r;
}

// Philox4x32-10 (ob_device.h) at the counter (blk, t) with blk = base + lane: base is uniform and a multiple of 64, lane below
// 64, so the counter's high word and all that depends on it alone stay in scalar registers.
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) { return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96); }

__device__ __forceinline__ u4 philox_lanes(uint64_t seed, uint64_t t, int64_t base, uint32_t lane)
{
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
    uint32_t c0 = static_cast<uint32_t>(base) + lane, c1 = static_cast<uint32_t>(static_cast<uint64_t>(base) >> 32);
    uint32_t c2 = static_cast<uint32_t>(t), c3 = static_cast<uint32_t>(t >> 32);
#pragma unroll
    for (int round = 0; round < 10; ++round) {
        const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0, p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
        const uint32_t h0 = static_cast<uint32_t>(p0 >> 32), h1 = static_cast<uint32_t>(p1 >> 32);
        // the first two rounds' scalar parts by plain xors
        c0 = round < 1 ? h1 ^ c1 ^ k0 : xor3(h1, c1, k0);
        c2 = round < 1 ? h0 ^ (c3 ^ k1) : xor3(h0, c3, k1);
        c1 = static_cast<uint32_t>(p1);
        c3 = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u4{{c0, c1, c2, c3}};
}

// |code| of x >= 0 as a float, by the rule, for a block with q > 0.  rq: about 1/q; root: about sqrt(x) (V
// only); bits: 16 random bits (SR).
template <bool V, bool SR>
__device__ __forceinline__ float code_by_rule(float x, float root, float q, float rq, uint32_t bits)
{
    constexpr float most = V ? 255.0f : 127.0f;
    const float y = __builtin_amdgcn_sqrtf((V ? root : x) * rq);
    float k;
    if (!SR) {
        const float h = floorf(y + (0.5f - kBelow)) + 0.5f;   // the next border
        k = h + (x >= code_value<V>(h, q) ? 0.5f : -0.5f);
    } else {
        k = fmaxf(floorf(y - kBelow), 0.0f);
        k += x >= code_value<V>(k + 1.0f, q) ? 1.0f : 0.0f;
        const float low = code_value<V>(k, q), high = code_value<V>(k + 1.0f, q);
        const float u = static_cast<float>(bits);
        k += mul(u, sub(high, low)) < mul(sub(x, low), 65536.0f) ? 1.0f : 0.0f;
        k = fminf(k, most);
    }
    return V && x > 0.0f ? fmaxf(k, 1.0f) : k;
}

// The codes of a lane's four elements of one block, as stored (int8 codes of m, uint8 of v).
template <bool V, bool SR>
__device__ __forceinline__ uint32_t encode4(const float x[4], const float root[4], float q, const u4& w)
{
    const float rq = __builtin_amdgcn_rcpf(q);
    uint32_t r = 0;
    auto put = [&](float code, int k) {
        r = __builtin_amdgcn_cvt_pk_u8_f32(V ? code : copysignf(code, x[k]) + 128.0f, k, r);   // rounds to nearest
    };
    auto bits = [&](int k) { return V ? w.x[k] >> 16 : w.x[k] & 0xffffu; };
    bool near = false;
    if (!SR) {
        float d = 1.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float y = __builtin_amdgcn_sqrtf((V ? root[k] : fabsf(x[k])) * rq);
            d = fminf(d, fabsf(__builtin_amdgcn_fractf(y) - 0.5f));
            put(V ? fmaxf(y, x[k] > 0.0f ? 1.0f : 0.0f) : y, k);
        }
        near = d < (V ? kNearV : kNearM);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // x in units of q (V: its root), its code k + f, the value between the codes' as a share of the gap: up
            // where the random bits are below that share.  num and gap are x - value(k) and value(k+1) - value(k)
            // over q (V: q^2).
            const float t = (V ? root[k] : fabsf(x[k])) * rq;
            const float c = floorf(__builtin_amdgcn_sqrtf(t)), odd = fmaf(2.0f, c, 1.0f);
            float num, gap;
            if (V) {
                const float c2 = c * c;
                num = (t - c2) * (t + c2);
                gap = odd * fmaf(2.0f, c2, odd);
            } else {
                num = fmaf(-c, c, t);
                gap = odd;
            }
            const float e = fmaf(num, 65536.0f, -static_cast<float>(bits(k)) * gap);
            // Near: |e| close to 0, or to 65536 gaps, where a value so close to a code may have been counted from
            // the wrong side of it and the bits are at the other end of their range.
            near = near || fabsf(fmaf(gap, -32768.0f, fabsf(e))) > (32768.0f - (V ? kNearChanceV : kNearChanceM)) * gap;
            const float up = c + fminf(fmaxf(e * 0x1p100f, 0.0f), 1.0f);   // one above where e > 0
            put(V ? fmaxf(up, x[k] > 0.0f ? 1.0f : 0.0f) : up, k);
        }
    }
    const bool small = V && SR && __float_as_uint(q) - 1u < kSmallScaleBits - 1u;   // 0 < q < 2^-63
    if (small || __builtin_amdgcn_ballot_w64(near) != 0) {
        r = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) put(code_by_rule<V, SR>(fabsf(x[k]), V ? root[k] : 0.0f, q, rq, bits(k)), k);
    }
    return q > 0.0f ? (V ? r : r ^ 0x80808080u) : 0u;
}

// The values of four stored codes.
template <bool V>
__device__ __forceinline__ void decode4(uint32_t w, float q, float x[4])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t b = w >> (8 * k);
        const float c = V ? static_cast<float>(b & 0xffu) : static_cast<float>(static_cast<int8_t>(b));
        x[k] = V ? code_value<true>(c, q) : mul(c * fabsf(c), q);
    }
}

// A lane's four codes, `cnt` of them in the tensor (4 or more: all); NT: nontemporal.
template <bool FULL, bool NT>
__device__ __forceinline__ uint32_t load_codes(const void* codes, int64_t i, int cnt)
{
    const uint8_t* c = static_cast<const uint8_t*>(codes) + i;
    if (FULL || cnt >= 4) return ldv<NT>(reinterpret_cast<const uint32_t*>(c));
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < cnt) w |= static_cast<uint32_t>(c[k]) << (8 * k);
    return w;
}

template <bool FULL>
__device__ __forceinline__ void store_codes(void* codes, int64_t i, int cnt, uint32_t w)
{
    uint8_t* c = static_cast<uint8_t*>(codes) + i;
    if (FULL || cnt >= 4) {
        __builtin_nontemporal_store(w, reinterpret_cast<uint32_t*>(c));
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < cnt) c[k] = static_cast<uint8_t>(w >> (8 * k));
}

// Scales of a span's blocks, the first `blocks` of them there; sb: the first block.
template <int S, bool FULL>
__device__ __forceinline__ f4 load_scales(const float* q, int64_t sb, int blocks)
{
    if (FULL && S == 4) return *reinterpret_cast<const f4e*>(q + sb);
    f4 r{};
#pragma unroll
    for (int j = 0; j < S; ++j)
        if (FULL || j < blocks) r[j] = q[sb + j];
    return r;
}

template <int S, bool FULL>
__device__ __forceinline__ void store_scales(float* mq, float* vq, int64_t sb, int blocks, const SpanScales& s)
{
    const int lane = static_cast<int>(threadIdx.x) & 63, j = (lane >> 4) & 1;
    if ((lane & (S == 1 ? 31 : 15)) != 0) return;
    float* q = (lane < 32 ? mq : vq) + sb + j;
    if (FULL || j < blocks) q[0] = s.a;
    if (S == 4 && (FULL || j + 2 < blocks)) q[2] = s.b;
}

}  // namespace
}  // namespace ob
