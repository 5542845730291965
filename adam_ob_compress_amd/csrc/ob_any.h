// ob_any.h -- loads and stores of elements of any of the list types, shared by the kernels over lists of tensors.
#pragma once

#include "ob_device.h"
#include "ob_state8.h"

namespace ob {
namespace {

// ------------------------------------------------------------------------------------------------
// loads and stores of four consecutive elements at the alignment of one
// ------------------------------------------------------------------------------------------------

typedef uint32_t u2e __attribute__((ext_vector_type(2), aligned(2)));

// type of elements: 0 fp32, 1 bf16, 2 fp16
template <int D>
__device__ __forceinline__ float widen16(uint32_t h)
{
    return D == 1 ? __uint_as_float(h << 16) : ErrF16::widen(h);
}

template <int D>
__device__ __forceinline__ f4 load_any4(const void* __restrict__ p, int64_t i)
{
    if (D == 0) return __builtin_nontemporal_load(reinterpret_cast<const f4e*>(static_cast<const float*>(p) + i));
    const u2e u = __builtin_nontemporal_load(reinterpret_cast<const u2e*>(static_cast<const uint16_t*>(p) + i));
    f4 r;
    r.x = widen16<D>(u.x & 0xffffu);
    r.y = widen16<D>(u.x >> 16);
    r.z = widen16<D>(u.y & 0xffffu);
    r.w = widen16<D>(u.y >> 16);
    return r;
}

template <int D>
__device__ __forceinline__ float load_any1(const void* __restrict__ p, int64_t i)
{
    return D == 0 ? static_cast<const float*>(p)[i] : widen16<D>(static_cast<const uint16_t*>(p)[i]);
}

// The 16-bit pattern of fp32 x rounded to the type: to nearest even, or (SR) up in magnitude where the 16 random
// bits r are below what is cut off.
template <int D, bool SR>
__device__ __forceinline__ uint32_t round16(float x, uint32_t r)
{
    if (D == 1 && SR) {
        // the cut-off bits plus 65535 - r carry exactly then; infinities have none, a NaN is kept a NaN
        const uint32_t u = __float_as_uint(x);
        return (x != x ? u | 0x00400000u : u + (r ^ 0xffffu)) >> 16;
    }
    if (D == 1) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
    return ErrF16::bits(SR ? ErrF16::rounded_sr(x, r) : ErrF16::rounded(x));
}

// Two values as elements of the type, in one word.
template <int D, bool SR>
__device__ __forceinline__ uint32_t round16x2(float x, float y, uint32_t r, uint32_t s)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    if (D == 1 && !SR) return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{x, y}, b2));
    return round16<D, SR>(x, r) | (round16<D, SR>(y, s) << 16);
}

// Four values as elements of the type; w: their random words (SR).
template <int D, bool SR>
__device__ __forceinline__ void store_any4(void* __restrict__ p, int64_t i, f4 x, const u4& w)
{
    if (D == 0) {
        __builtin_nontemporal_store(static_cast<f4e>(x), reinterpret_cast<f4e*>(static_cast<float*>(p) + i));
        return;
    }
    u2e u;
    u.x = round16x2<D, SR>(x.x, x.y, w.x[0] >> 16, w.x[1] >> 16);
    u.y = round16x2<D, SR>(x.z, x.w, w.x[2] >> 16, w.x[3] >> 16);
    __builtin_nontemporal_store(u, reinterpret_cast<u2e*>(static_cast<uint16_t*>(p) + i));
}

template <int D, bool SR>
__device__ __forceinline__ void store_any1(void* __restrict__ p, int64_t i, float x, uint32_t w)
{
    if (D == 0)
        static_cast<float*>(p)[i] = x;
    else
        static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(round16<D, SR>(x, w >> 16));
}

// ------------------------------------------------------------------------------------------------
// sums of squares of a list's gradients: squares and sums in double
// ------------------------------------------------------------------------------------------------

typedef uint32_t u4e __attribute__((ext_vector_type(4), aligned(2)));

template <int G>
__device__ __forceinline__ float load_grad1(const void* g, int64_t i)
{
    if (G == 0) return static_cast<const float*>(g)[i];
    const uint32_t h = static_cast<const uint16_t*>(g)[i];
    return G == 1 ? __uint_as_float(h << 16) : ErrF16::widen(h);
}

__device__ __forceinline__ void add_square(float x, double& s) { s = fma(static_cast<double>(x), static_cast<double>(x), s); }

// Sum of the squares in 16 bytes of gradients into two sums (the second shortens the chain of additions).
template <int G>
__device__ __forceinline__ void add_squares(u4e u, double s[2])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (G == 0) {
            add_square(__uint_as_float(u[k]), s[k & 1]);
        } else {
            add_square(G == 1 ? __uint_as_float(u[k] << 16) : ErrF16::widen(u[k] & 0xffffu), s[0]);
            add_square(G == 1 ? __uint_as_float(u[k] & 0xffff0000u) : ErrF16::widen(u[k] >> 16), s[1]);
        }
    }
}

// The squares of an item's elements, by a block of kListBlock threads.
template <int G, bool NT>
__device__ __forceinline__ void item_squares(const void* grad, const ListItem& it, double s[2])
{
    constexpr int V = G == 0 ? 4 : 8, U = 8, kTrip = V * kListBlock * U;
    const char* g = static_cast<const char*>(grad) + it.start * (16 / V);
    const int tid = static_cast<int>(threadIdx.x);
    int base = 0;
    for (; base + kTrip <= it.len; base += kTrip) {
        u4e x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const u4e* at = reinterpret_cast<const u4e*>(g + int64_t(base) * (16 / V)) + u * kListBlock + tid;
            x[u] = NT ? __builtin_nontemporal_load(at) : *at;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) add_squares<G>(x[u], s);
    }
    for (; base < it.len; base += V * kListBlock) {   // a tensor's last item
        const int at = base + V * tid, cnt = it.len - at;
        if (cnt >= V) {
            add_squares<G>(*reinterpret_cast<const u4e*>(g + int64_t(at) * (16 / V)), s);
        } else {
            for (int k = 0; k < cnt; ++k) add_square(load_grad1<G>(g, at + k), s[0]);
        }
    }
}

}  // namespace
}  // namespace ob
