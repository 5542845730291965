// ob_state8.hip -- the global gradient norm of a list of tensors with the control block that the steps
// read, and the 8-bit state format to and from fp32.
#include "ob_state8.h"

namespace ob {
namespace {

// ------------------------------------------------------------------------------------------------
// gradient norm: squares and sums in double (their order is fixed by the list and the grid); one pass
// over the gradients, then one block over the partial sums
// ------------------------------------------------------------------------------------------------

typedef float f4e __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u2e __attribute__((ext_vector_type(2), aligned(2)));

template <int G>
__device__ __forceinline__ float load_grad1(const void* g, int64_t i)
{
    if (G == 0) return static_cast<const float*>(g)[i];
    const uint32_t h = static_cast<const uint16_t*>(g)[i];
    return G == 1 ? __uint_as_float(h << 16) : ErrF16::widen(h);
}

template <int G>
__device__ __forceinline__ f4 load_grad4(const void* g, int64_t i)
{
    if (G == 0) return *reinterpret_cast<const f4e*>(static_cast<const float*>(g) + i);
    const u2e u = *reinterpret_cast<const u2e*>(static_cast<const uint16_t*>(g) + i);
    f4 r;
    if (G == 1) {
        r.x = __uint_as_float(u.x << 16);
        r.y = __uint_as_float(u.x & 0xffff0000u);
        r.z = __uint_as_float(u.y << 16);
        r.w = __uint_as_float(u.y & 0xffff0000u);
    } else {
        r.x = ErrF16::widen(u.x & 0xffffu);
        r.y = ErrF16::widen(u.x >> 16);
        r.z = ErrF16::widen(u.y & 0xffffu);
        r.w = ErrF16::widen(u.y >> 16);
    }
    return r;
}

template <int G>
__global__ __launch_bounds__(kListBlock) void k_grad_sumsq(ListLaunch L, NormPtrs ptrs, int first,
                                                           double* __restrict__ partials)
{
    __shared__ double lds[kListBlock / 64];
    double s = 0.0;
    for (int64_t b = blockIdx.x; b < L.n_items; b += gridDim.x) {
        const ListItem it = L.items[b];
        const void* g = ptrs.g[it.tensor - L.tensor0];
        if (g == nullptr) continue;
        for (int base = 0; base < it.len; base += kListTile) {
            const int at = base + 4 * static_cast<int>(threadIdx.x);
            const int cnt = it.len - at;
            if (cnt >= 4) {
                const f4 x = load_grad4<G>(g, it.start + at);
#pragma unroll
                for (int k = 0; k < 4; ++k) s = fma(static_cast<double>(x[k]), static_cast<double>(x[k]), s);
            } else {
                for (int k = 0; k < cnt; ++k) {
                    const double x = static_cast<double>(load_grad1<G>(g, it.start + at + k));
                    s = fma(x, x, s);
                }
            }
        }
    }
    s = block_sum(s, lds);
    if (threadIdx.x == 0) partials[blockIdx.x] = first ? s : partials[blockIdx.x] + s;
}

__global__ __launch_bounds__(kListBlock) void k_grad_control(ob_control* ctl, int grid, NormParams np)
{
    __shared__ double lds[kListBlock / 64];
    const double* partials = reinterpret_cast<const double*>(ctl + 1);
    double s = 0.0;
    for (int b = threadIdx.x; b < grid; b += kListBlock) s += partials[b];
    s = block_sum(s, lds);
    if (threadIdx.x != 0) return;
    const double norm = fabs(np.g_mult) * sqrt(s);
    double f = 1.0;
    if (np.clip) {
        f = np.max_norm / (norm + 1e-6);
        f = f > 1.0 ? 1.0 : f;   // NaN stays
    }
    ctl->norm = static_cast<float>(norm);
    ctl->grad_scale = static_cast<float>(np.g_mult * f);
    const bool ok = (__float_as_uint(static_cast<float>(norm)) & 0x7fffffffu) < kInfBits;
    ctl->skip = ok ? 0 : 1;
    if (!np.advance) return;
    if (!ok) {
        ctl->skipped += 1;
        return;
    }
    const int64_t t = ctl->step + 1;
    ctl->step = t;
    ctl->bc1 = 1.0 - pow(np.beta1, static_cast<double>(t));
    ctl->bc2 = 1.0 - pow(np.beta2, static_cast<double>(t));
}

// ------------------------------------------------------------------------------------------------
// the 8-bit format: one state block per wave and trip
// ------------------------------------------------------------------------------------------------

template <bool V>
__device__ __forceinline__ void encode_block(int64_t at, int64_t cnt, int lane, const float* __restrict__ x,
                                             uint8_t* __restrict__ codes, float* __restrict__ scales)
{
    float e[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t i = at + 4 * lane;
    const int64_t left = cnt - 4 * lane;
    if (left >= 4) {
        const f4 r = ld4<true>(x, i);
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = r[k];
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < left) e[k] = x[i + k];
    }
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t b = __float_as_uint(e[k]);
        if (V && b > 0x80000000u) b = kInfBits + 1;   // a negative v counts as NaN (-0 does not)
        b &= 0x7fffffffu;
        top = top > b ? top : b;
    }
    const float q = block_scale<V>(wave_max(top));
    const float rq = guess_scale(q);
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (V) {
            w = put_byte(encode<true, false>(e[k], __builtin_amdgcn_sqrtf(e[k]), q, rq, 0), k, w);
        } else {
            const float c = encode<false, false>(fabsf(e[k]), 0.0f, q, rq, 0);
            w = put_byte(copysignf(c, e[k]) + 128.0f, k, w);
        }
    }
    if (!V) w ^= kBias4;
    if (lane == 0) scales[at / kStateBlock] = q;
    if (left >= 4) {
        *reinterpret_cast<uint32_t*>(codes + i) = w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < left) codes[i + k] = static_cast<uint8_t>(byte_of(w, k));
    }
}

template <bool V>
__device__ __forceinline__ void decode_block(int64_t at, int64_t cnt, int lane, const uint8_t* __restrict__ codes,
                                             const float* __restrict__ scales, float* __restrict__ x)
{
    const int64_t i = at + 4 * lane;
    const int64_t left = cnt - 4 * lane;
    const float q = scales[at / kStateBlock];
    if (left >= 4) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + i) ^ (V ? 0u : kBias4);
        f4 r;
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = V ? decode_v(byte_of(w, k), q) : decode_m(byte_of(w, k), q);
        st4<true>(x, i, r);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k >= left) continue;
            const uint32_t b = codes[i + k];
            x[i + k] = V ? decode_v(b, q) : decode_m(b ^ 0x80u, q);
        }
    }
}

// A block of the launch takes kSpan state blocks per wave, of m and of v.
constexpr int kSpan = 4;

__global__ __launch_bounds__(kListBlock) void k_state8_encode(int64_t n, const float* m, const float* v, uint8_t* mc,
                                                              float* mq, uint8_t* vc, float* vq)
{
    const int wave = static_cast<int>(threadIdx.x) >> 6, lane = static_cast<int>(threadIdx.x) & 63;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kListBlock / 64) + wave) * kSpan * kStateBlock;
    for (int j = 0; j < kSpan; ++j) {
        const int64_t at = first + j * kStateBlock, cnt = n - at;
        if (cnt <= 0) return;
        if (m) encode_block<false>(at, cnt, lane, m, mc, mq);
        if (v) encode_block<true>(at, cnt, lane, v, vc, vq);
    }
}

__global__ __launch_bounds__(kListBlock) void k_state8_decode(int64_t n, const uint8_t* mc, const float* mq,
                                                              const uint8_t* vc, const float* vq, float* m, float* v)
{
    const int wave = static_cast<int>(threadIdx.x) >> 6, lane = static_cast<int>(threadIdx.x) & 63;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kListBlock / 64) + wave) * kSpan * kStateBlock;
    for (int j = 0; j < kSpan; ++j) {
        const int64_t at = first + j * kStateBlock, cnt = n - at;
        if (cnt <= 0) return;
        if (m) decode_block<false>(at, cnt, lane, mc, mq, m);
        if (v) decode_block<true>(at, cnt, lane, vc, vq, v);
    }
}

unsigned state8_grid(int64_t n)
{
    constexpr int64_t per = int64_t(kListBlock / 64) * kSpan * kStateBlock;
    return static_cast<unsigned>((n + per - 1) / per);
}

}  // namespace

hipError_t launch_grad_sumsq(const ListLaunch& L, const NormPtrs& ptrs, int g_dtype, int grid, int first,
                             double* partials, hipStream_t s)
{
    switch (g_dtype) {
    case OB_BF16: hipLaunchKernelGGL(k_grad_sumsq<1>, dim3(grid), dim3(kListBlock), 0, s, L, ptrs, first, partials); break;
    case OB_F16: hipLaunchKernelGGL(k_grad_sumsq<2>, dim3(grid), dim3(kListBlock), 0, s, L, ptrs, first, partials); break;
    default: hipLaunchKernelGGL(k_grad_sumsq<0>, dim3(grid), dim3(kListBlock), 0, s, L, ptrs, first, partials);
    }
    return hipGetLastError();
}

hipError_t launch_grad_control(ob_control* ctl, int grid, const NormParams& np, hipStream_t s)
{
    hipLaunchKernelGGL(k_grad_control, dim3(1), dim3(kListBlock), 0, s, ctl, grid, np);
    return hipGetLastError();
}

hipError_t launch_state8_encode(int64_t n, const float* m, const float* v, int8_t* mc, float* mq, uint8_t* vc,
                                float* vq, hipStream_t s)
{
    hipLaunchKernelGGL(k_state8_encode, dim3(state8_grid(n)), dim3(kListBlock), 0, s, n, m, v,
                       reinterpret_cast<uint8_t*>(mc), mq, vc, vq);
    return hipGetLastError();
}

hipError_t launch_state8_decode(int64_t n, const int8_t* mc, const float* mq, const uint8_t* vc, const float* vq,
                                float* m, float* v, hipStream_t s)
{
    hipLaunchKernelGGL(k_state8_decode, dim3(state8_grid(n)), dim3(kListBlock), 0, s, n,
                       reinterpret_cast<const uint8_t*>(mc), mq, vc, vq, m, v);
    return hipGetLastError();
}

}  // namespace ob
