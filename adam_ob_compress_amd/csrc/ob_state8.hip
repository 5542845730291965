// ob_state8.hip -- the global gradient norm of a list of tensors with the control block that the steps
// read, and the 8-bit state format to and from fp32.
#include "ob_state8.h"

namespace ob {
namespace {

// ------------------------------------------------------------------------------------------------
// gradient norm: squares and sums in double (their order is fixed by the list and the grid); one pass
// over the gradients, then one block over the partial sums
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

// What the norm's last block writes into the control block: s is the sum of all squares.  Threads 0 and 1
// take one bias correction each; both are lanes of one wave.
__device__ __forceinline__ void write_control(ob_control* ctl, double s, const NormParams& np)
{
    if (threadIdx.x > 1) return;
    const double norm = fabs(np.g_mult) * sqrt(s);
    const bool ok = (__float_as_uint(static_cast<float>(norm)) & 0x7fffffffu) < kInfBits;
    const int64_t t = ctl->step + 1;
    const double bc = np.advance ? 1.0 - pow(threadIdx.x == 0 ? np.beta1 : np.beta2, static_cast<double>(t)) : 1.0;
    const double bc2 = __shfl(bc, 1, 64);
    if (threadIdx.x == 1) {
        if (np.advance && ok) ctl->bc2 = bc;
        return;
    }
    double f = 1.0;
    if (np.clip) {
        f = np.max_norm / (norm + 1e-6);
        f = f > 1.0 ? 1.0 : f;   // NaN stays
    }
    ctl->norm = static_cast<float>(norm);
    ctl->grad_scale = static_cast<float>(np.g_mult * f);
    ctl->skip = ok ? 0 : 1;
    if (!np.advance) return;
    if (ok) {
        ctl->step = t;
        ctl->bc1 = bc;
        ctl->root_factor = static_cast<float>(bc / sqrt(bc2));
    } else {
        ctl->skipped += 1;
    }
}

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

// Bound by HBM's reads: 1.56e9 bf16 gradients 444 us, 7.0 TB/s (8-byte loads, one item's tile at a time: 575 us).
// A block takes every gridDim-th item, a lane 16 bytes of every 4 KB of it, eight of them in flight.  With np.ticket
// the block that finishes last (by a ticket in the control block, which it sets back to zero) also finishes
// the norm; the grid has at most kListBlock blocks then.
template <int G>
__global__ __launch_bounds__(kListBlock) void k_grad_sumsq(ListLaunch L, NormPtrs ptrs, int64_t nt_items, ob_control* ctl,
                                                           NormParams np)
{
    __shared__ double lds[kListBlock / 64];
    __shared__ bool last;
    double* partials = reinterpret_cast<double*>(ctl + 1);
    double s[2] = {0.0, 0.0};
    for (int64_t b = blockIdx.x; b < L.n_items; b += gridDim.x) {
        const ListItem it = L.items[b];
        const void* g = ptrs.g[it.tensor - L.tensor0];
        if (g == nullptr) continue;
        if (b < nt_items)
            item_squares<G, true>(g, it, s);
        else
            item_squares<G, false>(g, it, s);
    }
    const double t = block_sum(s[0] + s[1], lds);
    if (threadIdx.x == 0) {
        double* mine = partials + blockIdx.x;
        __hip_atomic_store(mine, np.first ? t : *mine + t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = np.ticket && __hip_atomic_fetch_add(&ctl->ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                                gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    if (threadIdx.x == 0) ctl->ticket = 0;
    const double a = threadIdx.x < gridDim.x
                         ? __hip_atomic_load(partials + threadIdx.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                         : 0.0;
    write_control(ctl, block_sum(a, lds), np);
}

// The control block from the partial sums of a larger grid.
__global__ __launch_bounds__(kListBlock) void k_grad_control(ob_control* ctl, int grid, NormParams np)
{
    __shared__ double lds[kListBlock / 64];
    const double* partials = reinterpret_cast<const double*>(ctl + 1);
    double a[OB_CONTROL_PARTIALS / kListBlock];
#pragma unroll
    for (int k = 0; k < OB_CONTROL_PARTIALS / kListBlock; ++k) {
        const int b = k * kListBlock + static_cast<int>(threadIdx.x);
        a[k] = b < grid ? partials[b] : 0.0;
    }
#pragma unroll
    for (int k = 1; k < OB_CONTROL_PARTIALS / kListBlock; ++k) a[0] += a[k];
    write_control(ctl, block_sum(a[0], lds), np);
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

template <bool FULL, bool V>
__device__ __forceinline__ void encode_span(int64_t n, int64_t at, const float* x, uint8_t* codes, float* scales)
{
    const int lane = static_cast<int>(threadIdx.x) & 63, lane4 = 4 * lane;
    const int left = FULL ? kSpanElems : static_cast<int>(n - at), blocks = (left + kStateBlock - 1) / kStateBlock;
    float e[kSpan][4], root[kSpan][4];
    uint32_t top[kSpan] = {};
#pragma unroll
    for (int j = 0; j < kSpan; ++j) load4<FULL>(x, at + j * kStateBlock + lane4, left - j * kStateBlock - lane4, e[j]);
#pragma unroll
    for (int j = 0; j < kSpan; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (V) e[j][k] += 0.0f;   // -0 becomes +0, so that a set sign is a negative v or a NaN: not finite below
            top[j] = max_u(top[j], __float_as_uint(e[j][k]) & (V ? 0xffffffffu : 0x7fffffffu));
            root[j][k] = V ? __builtin_amdgcn_sqrtf(e[j][k]) : 0.0f;
        }
    }
    // the four scales, one in each row of 16 lanes: of blocks 0, 2, 1, 3
    const float q = block_scale(row_max(fold16(fold32(top[0], top[1]), fold32(top[2], top[3]))), V);
    auto row = [](int j) { return (j & 1) * 2 + (j >> 1); };
    const int mine = row(lane >> 4);   // the same exchange of two bits backwards
    if ((lane & 15) == 0 && (FULL || mine < blocks)) scales[at / kStateBlock + mine] = q;
#pragma unroll
    for (int j = 0; j < kSpan; ++j) {
        const float qj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(q), 16 * row(j)));
        const int o = j * kStateBlock + lane4;
        store_codes<FULL>(codes, at + o, left - o, encode4<V, false>(e[j], root[j], qj, u4{}));
    }
}

template <bool FULL, bool V>
__device__ __forceinline__ void decode_span(int64_t n, int64_t at, const uint8_t* codes, const float* scales, float* x)
{
    const int lane4 = 4 * (static_cast<int>(threadIdx.x) & 63);
    const int left = FULL ? kSpanElems : static_cast<int>(n - at), blocks = (left + kStateBlock - 1) / kStateBlock;
    const f4 q = load_scales<kSpan, FULL>(scales, at / kStateBlock, blocks);
    uint32_t w[kSpan];
#pragma unroll
    for (int j = 0; j < kSpan; ++j) w[j] = load_codes<FULL, false>(codes, at + j * kStateBlock + lane4, left - j * kStateBlock - lane4);
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

// Bound by HBM's reads: 1e9 elements 1620 us, 6.2 TB/s.
// The blocks of a launch's first row encode m, those of the second v.  (Both moments in each block: 1e9
// elements 1714 us against 1614.  The decoder does not gain by it.)
__global__ __launch_bounds__(kListBlock) void k_state8_encode(int64_t n, const float* m, const float* v, uint8_t* mc,
                                                              float* mq, uint8_t* vc, float* vq)
{
    const int64_t at = span_start();
    const bool whole = n - at >= kSpanElems;
    if (n <= at) return;
    if (blockIdx.y == 0) {
        if (m == nullptr) return;
        if (whole)
            encode_span<true, false>(n, at, m, mc, mq);
        else
            encode_span<false, false>(n, at, m, mc, mq);
    } else {
        if (v == nullptr) return;
        if (whole)
            encode_span<true, true>(n, at, v, vc, vq);
        else
            encode_span<false, true>(n, at, v, vc, vq);
    }
}

// Bound by HBM's writes (8 of 10 bytes an element): 1e9 elements 1.76 ms, 5.7 TB/s, where a fill of one of its
// outputs runs at 6.6.  The codes by nontemporal loads: 1.83 ms; ordinary stores: the same; several spans per wave one
// after the other: 1 to 6 percent slower.
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

hipError_t launch_grad_sumsq(const ListLaunch& L, const NormPtrs& ptrs, int g_dtype, int grid, int64_t nt_items,
                             ob_control* ctl, const NormParams& np, hipStream_t s)
{
    const auto k = g_dtype == OB_BF16 ? k_grad_sumsq<1> : g_dtype == OB_F16 ? k_grad_sumsq<2> : k_grad_sumsq<0>;
    hipLaunchKernelGGL(k, dim3(grid), dim3(kListBlock), 0, s, L, ptrs, nt_items, ctl, np);
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
    hipLaunchKernelGGL(k_state8_encode, dim3(state8_grid(n), 2), dim3(kListBlock), 0, s, n, m, v,
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
