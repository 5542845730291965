// ob_state8.hip -- the global gradient norm of a list of tensors with the control block that the steps
// read, and the 8-bit state format to and from fp32.
#include "ob_state8.h"

namespace ob {
namespace {

// ------------------------------------------------------------------------------------------------
// gradient norm: squares and sums in double (their order is fixed by the list and the grid); one pass
// over the gradients, then one block over the partial sums
// ------------------------------------------------------------------------------------------------

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
    const double bc1 = 1.0 - pow(np.beta1, static_cast<double>(t)), bc2 = 1.0 - pow(np.beta2, static_cast<double>(t));
    ctl->step = t;
    ctl->bc1 = bc1;
    ctl->bc2 = bc2;
    ctl->inv_bc1 = static_cast<float>(1.0 / bc1);
    ctl->inv_root_bc2 = static_cast<float>(1.0 / sqrt(bc2));
}

// ------------------------------------------------------------------------------------------------
// the 8-bit format: one state block per wave and trip
// ------------------------------------------------------------------------------------------------

// The lane's four elements of x that are in the array; zeros behind it.
template <bool FULL>
__device__ __forceinline__ void load4(const float* __restrict__ x, int64_t i, int64_t left, float e[4])
{
    if (FULL || left >= 4) {
        const f4 r = ld4<true>(x, i);
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = r[k];
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) e[k] = k < left ? x[i + k] : 0.0f;
}

template <bool FULL>
__device__ __forceinline__ void encode_span(int64_t n, int64_t at, const float* m, const float* v, uint8_t* mc, float* mq,
                                            uint8_t* vc, float* vq)
{
    const int lane4 = 4 * (static_cast<int>(threadIdx.x) & 63);
    const int left = FULL ? kSpanElems : static_cast<int>(n - at), blocks = (left + kStateBlock - 1) / kStateBlock;
    float me[kSpan][4] = {}, ve[kSpan][4] = {}, root[kSpan][4];
    uint32_t tm[kSpan] = {}, tv[kSpan] = {};
#pragma unroll
    for (int j = 0; j < kSpan; ++j) {
        const int o = j * kStateBlock + lane4;
        if (m) load4<FULL>(m, at + o, left - o, me[j]);
        if (v) load4<FULL>(v, at + o, left - o, ve[j]);
    }
#pragma unroll
    for (int j = 0; j < kSpan; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            tm[j] = max_u(tm[j], __float_as_uint(me[j][k]) & 0x7fffffffu);
            ve[j][k] += 0.0f;                              // -0 becomes +0, so that
            tv[j] = max_u(tv[j], __float_as_uint(ve[j][k]));   // a set sign is a negative v or a NaN
            root[j][k] = __builtin_amdgcn_sqrtf(ve[j][k]);
        }
    }
    const SpanScales q = span_scales(tm, tv);
    const int lane = static_cast<int>(threadIdx.x) & 63;
    if (lane < 32 ? m != nullptr : v != nullptr) store_scales<FULL>(mq, vq, at / kStateBlock, blocks, q);
#pragma unroll
    for (int j = 0; j < kSpan; ++j) {
        const int o = j * kStateBlock + lane4;
        if (m) store_codes<FULL>(mc, at + o, left - o, encode4<false, false>(me[j], nullptr, q.get(j, false), u4{}));
        if (v) store_codes<FULL>(vc, at + o, left - o, encode4<true, false>(ve[j], root[j], q.get(j, true), u4{}));
    }
}

template <bool FULL, bool V>
__device__ __forceinline__ void decode_span(int64_t n, int64_t at, const uint8_t* codes, const float* scales, float* x)
{
    const int lane4 = 4 * (static_cast<int>(threadIdx.x) & 63);
    const int left = FULL ? kSpanElems : static_cast<int>(n - at), blocks = (left + kStateBlock - 1) / kStateBlock;
    const f4 q = load_scales<FULL>(scales, at / kStateBlock, blocks);
    uint32_t w[kSpan];
#pragma unroll
    for (int j = 0; j < kSpan; ++j) w[j] = load_codes<FULL>(codes, at + j * kStateBlock + lane4, left - j * kStateBlock - lane4);
#pragma unroll
    for (int j = 0; j < kSpan; ++j) {
        const int o = j * kStateBlock + lane4;
        float e[4];
        decode4<V>(w[j], q[j], e);
        if (FULL || left - o >= 4) {
            const f4 r = {e[0], e[1], e[2], e[3]};
            st4<true>(x, at + o, r);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < left - o) x[at + o + k] = e[k];
        }
    }
}

constexpr int64_t kState8Elems = int64_t(kListBlock / 64) * kSpanElems;   // per block of the launch

__device__ __forceinline__ int64_t span_start()
{
    return static_cast<int64_t>(blockIdx.x) * kState8Elems +
           __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6) * kSpanElems;
}

__global__ __launch_bounds__(kListBlock) void k_state8_encode(int64_t n, const float* m, const float* v, uint8_t* mc,
                                                              float* mq, uint8_t* vc, float* vq)
{
    const int64_t at = span_start();
    if (n - at >= kSpanElems)
        encode_span<true>(n, at, m, v, mc, mq, vc, vq);
    else if (n > at)
        encode_span<false>(n, at, m, v, mc, mq, vc, vq);
}

__global__ __launch_bounds__(kListBlock) void k_state8_decode(int64_t n, const uint8_t* mc, const float* mq,
                                                              const uint8_t* vc, const float* vq, float* m, float* v)
{
    const int64_t at = span_start();
    if (n - at >= kSpanElems) {
        if (m) decode_span<true, false>(n, at, mc, mq, m);
        if (v) decode_span<true, true>(n, at, vc, vq, v);
    } else if (n > at) {
        if (m) decode_span<false, false>(n, at, mc, mq, m);
        if (v) decode_span<false, true>(n, at, vc, vq, v);
    }
}

unsigned state8_grid(int64_t n) { return static_cast<unsigned>((n + kState8Elems - 1) / kState8Elems); }

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
