// ob_clip.hip -- norms of the tensors of a list and of all together, and the gradients times a factor that clips them.
#include "ob_any.h"
#include "ob_clip.h"

namespace ob {
namespace {

// What is reduced: a sum of squares, or a largest magnitude.  Both in double; a NaN stays.
template <bool MAX>
__device__ __forceinline__ double join(double a, double b)
{
    if (!MAX) return a + b;
    return b > a || b != b ? b : a;
}

template <bool MAX>
__device__ __forceinline__ double join_wave(double v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = join<MAX>(v, __shfl_xor(v, off, 64));
    return v;
}

// Over the block in a fixed order; every thread returns the same value.
template <bool MAX, int WAVES>
__device__ __forceinline__ double join_block(double v, double* lds)
{
    v = join_wave<MAX>(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = lds[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s = join<MAX>(s, lds[w]);
    return s;
}

// The largest magnitude in 16 bytes of gradients, as the bits of a non-negative fp32: they compare as the values do, with
// NaN on top.
template <int G>
__device__ __forceinline__ uint32_t max_bits(u4e u, uint32_t m)
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (G == 0) {
            m = max_u(m, u[k] & 0x7fffffffu);
        } else {
            const float a = G == 1 ? __uint_as_float(u[k] << 16) : ErrF16::widen(u[k] & 0xffffu);
            const float b = G == 1 ? __uint_as_float(u[k] & 0xffff0000u) : ErrF16::widen(u[k] >> 16);
            m = max_u(max_u(m, __float_as_uint(a) & 0x7fffffffu), __float_as_uint(b) & 0x7fffffffu);
        }
    }
    return m;
}

template <int G, bool NT>
__device__ __forceinline__ uint32_t item_max(const void* grad, const ListItem& it)
{
    constexpr int V = G == 0 ? 4 : 8;
    const char* g = static_cast<const char*>(grad) + it.start * (16 / V);
    uint32_t m = 0;
    for (int at = V * static_cast<int>(threadIdx.x); at < it.len; at += V * kListBlock) {
        if (it.len - at >= V) {
            const u4e* p = reinterpret_cast<const u4e*>(g + int64_t(at) * (16 / V));
            m = max_bits<G>(NT ? __builtin_nontemporal_load(p) : *p, m);
        } else {
            for (int k = at; k < it.len; ++k) m = max_u(m, __float_as_uint(load_grad1<G>(g, k)) & 0x7fffffffu);
        }
    }
    return m;
}

// One work group for each item (16 K elements of one tensor).  Bound by HBM's reads: 1e9 bf16 gradients 290 us, 6.9 TB/s.
template <int G, bool MAX>
__global__ __launch_bounds__(kListBlock) void k_item_norms(ListLaunch L, NormPtrs ptrs, int64_t nt_items, double* partials)
{
    __shared__ double lds[kListBlock / 64];
    const int64_t b = blockIdx.x;
    const ListItem it = L.items[b];
    const void* g = ptrs.g[it.tensor - L.tensor0];
    double v = 0.0;
    if (g != nullptr) {
        if (MAX) {
            v = static_cast<double>(__uint_as_float(b < nt_items ? item_max<G, true>(g, it) : item_max<G, false>(g, it)));
        } else {
            double s[2] = {0.0, 0.0};
            if (b < nt_items)
                item_squares<G, true>(g, it, s);
            else
                item_squares<G, false>(g, it, s);
            v = s[0] + s[1];
        }
    }
    v = join_block<MAX, kListBlock / 64>(v, lds);
    if (threadIdx.x == 0) partials[b] = v;
}

constexpr int kNormBlock = 1024;

// fp32 norm from a reduced value
template <bool MAX>
__device__ __forceinline__ float norm_of(double v, double g_mult)
{
    return static_cast<float>(fabs(g_mult) * (MAX ? v : sqrt(v)));
}

// A tensor's partial results, by `threads` threads of which this is number `at`.
template <bool MAX>
__device__ __forceinline__ double tensor_part(const NormTables& t, int64_t place, int at, int threads)
{
    double v = 0.0;
    for (int64_t i = t.first[place] + at; i < t.first[place + 1]; i += threads) v = join<MAX>(v, t.partials[i]);
    return v;
}

// One work group for each tensor.
template <bool MAX>
__global__ __launch_bounds__(kNormBlock) void k_tensor_norms(NormTables t, double g_mult, float* norms)
{
    __shared__ double lds[kNormBlock / 64];
    const double v = join_block<MAX, kNormBlock / 64>(tensor_part<MAX>(t, blockIdx.x, static_cast<int>(threadIdx.x), kNormBlock), lds);
    if (threadIdx.x != 0) return;
    norms[t.order[blockIdx.x]] = norm_of<MAX>(v, g_mult);
    t.partials[t.items + blockIdx.x] = v;
}

// The norm of all from the tensors'.  SMALL: the tensors' too, a wave for each in turn.
template <bool MAX, bool SMALL>
__global__ __launch_bounds__(kNormBlock) void k_total_norm(NormTables t, double g_mult, float* norms)
{
    __shared__ double lds[kNormBlock / 64];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
    double all = 0.0;
    if (SMALL) {
        for (int64_t k = tid >> 6; k < t.tensors; k += kNormBlock / 64) {
            const double v = join_wave<MAX>(tensor_part<MAX>(t, k, lane, 64));
            if (lane == 0) {
                norms[t.order[k]] = norm_of<MAX>(v, g_mult);
                all = join<MAX>(all, v);
            }
        }
    } else {
        for (int64_t k = tid; k < t.tensors; k += kNormBlock) all = join<MAX>(all, t.partials[t.items + k]);
    }
    all = join_block<MAX, kNormBlock / 64>(all, lds);
    if (tid == 0) norms[t.tensors] = norm_of<MAX>(all, g_mult);
}

// The norms of a short list in one launch: a wave for each tensor in turn.
template <int G, bool MAX>
__global__ __launch_bounds__(kNormBlock) void k_short_norms(ListLaunch L, NormPtrs ptrs, NormTables t, double g_mult, float* norms)
{
    constexpr int V = G == 0 ? 4 : 8, U = 4;   // elements of a load, loads in flight
    __shared__ double lds[kNormBlock / 64];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
    double all = 0.0;
    for (int64_t k = tid >> 6; k < t.tensors; k += kNormBlock / 64) {
        const char* g = static_cast<const char*>(ptrs.g[k]);
        double s[2] = {0.0, 0.0};
        uint32_t m = 0;
        if (g != nullptr && t.first[k] < t.first[k + 1]) {
            const int n = L.items[t.first[k]].len;   // a short tensor is one item
            for (int at = V * lane; at < n; at += 64 * V * U) {
                u4e x[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = at + 64 * V * u;
                    x[u] = u4e{};
                    if (i + V <= n) x[u] = *reinterpret_cast<const u4e*>(g + int64_t(i) * (16 / V));
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (MAX)
                        m = max_bits<G>(x[u], m);
                    else
                        add_squares<G>(x[u], s);
                }
            }
            const int rest = n / V * V + lane;   // less than a load's elements at the end
            if (rest < n) {
                const float e = load_grad1<G>(g, rest);
                m = max_u(m, __float_as_uint(e) & 0x7fffffffu);
                add_square(e, s[0]);
            }
        }
        const double v = join_wave<MAX>(MAX ? static_cast<double>(__uint_as_float(m)) : s[0] + s[1]);
        if (lane == 0) {
            norms[t.order[k]] = norm_of<MAX>(v, g_mult);
            all = join<MAX>(all, v);
        }
    }
    all = join_block<MAX, kNormBlock / 64>(all, lds);
    if (tid == 0) norms[t.tensors] = norm_of<MAX>(all, g_mult);
}

// Eight elements from element i on, widened, and back.
template <int G>
__device__ __forceinline__ void load8(const void* g, int64_t i, float x[8])
{
    if (G == 0) {
        const f4 a = load_any4<0>(g, i), b = load_any4<0>(g, i + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = a[e];
            x[4 + e] = b[e];
        }
    } else {
        const u4e u = __builtin_nontemporal_load(reinterpret_cast<const u4e*>(static_cast<const uint16_t*>(g) + i));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = widen16<G>(u[e] & 0xffffu);
            x[2 * e + 1] = widen16<G>(u[e] >> 16);
        }
    }
}
template <int D>
__device__ __forceinline__ void store8(void* out, int64_t i, const float x[8])
{
    if (D == 0) {
        store_any4<0, false>(out, i, f4{x[0], x[1], x[2], x[3]}, u4{});
        store_any4<0, false>(out, i + 4, f4{x[4], x[5], x[6], x[7]}, u4{});
    } else {
        u4e u;
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = round16x2<D, false>(x[2 * e], x[2 * e + 1], 0, 0);
        __builtin_nontemporal_store(u, reinterpret_cast<u4e*>(static_cast<uint16_t*>(out) + i));
    }
}

// out = g * f.  The items in reverse: the norms read the list's end last, and what the last-level cache holds of it is met first.
// Bound by HBM.  A work group takes an item (4096 elements), a lane 16 bytes of 16-bit gradients at a time, two in flight, and forms the
// factor once: 1e9 bf16 elements into bf16 633 us, 6.3 TB/s (four elements a lane and group, a factor for each: 985 us).
template <int G, int D>
__global__ __launch_bounds__(kListBlock) void k_clip(ListLaunch L, ListPtrs ptrs, ClipParams cp)
{
    constexpr int kParts = kStepTiles * kListTile / (8 * kListBlock);
    const ListItem it = L.items[L.n_items - 1 - blockIdx.x];
    const void* g = ptrs.g[it.tensor - L.tensor0];
    if (g == nullptr) return;
    void* out = ptrs.p[it.tensor - L.tensor0];
    const int tid = static_cast<int>(threadIdx.x);
    const bool whole = it.len == 8 * kListBlock * kParts;
    float x[kParts][8];
    if (whole) {
#pragma unroll
        for (int k = 0; k < kParts; ++k) load8<G>(g, it.start + 8 * (k * kListBlock + tid), x[k]);
    }
    const double norm = static_cast<double>(cp.norms[cp.order ? cp.order[it.tensor] : cp.total]);
    double f = 1.0;
    if (cp.clip) {
        f = cp.max_norm / (norm + 1e-6);
        f = f > 1.0 ? 1.0 : f;
    }
    f = isfinite(norm) ? f * cp.g_mult : __builtin_nan("");
    const float scale = static_cast<float>(f);
    if (G == D && out == g && scale == 1.0f) return;
    if (whole) {
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] = mul(x[k][e], scale);
            store8<D>(out, it.start + 8 * (k * kListBlock + tid), x[k]);
        }
        return;
    }
    // a tensor's last item: four elements at a time, and what is left
    for (int at = 4 * tid; at < it.len; at += kListTile) {
        const int64_t i = it.start + at;
        if (it.len - at >= 4) {
            f4 v = load_any4<G>(g, i);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = mul(v[e], scale);
            store_any4<D, false>(out, i, v, u4{});
        } else {
            for (int e = at; e < it.len; ++e) store_any1<D, false>(out, it.start + e, mul(load_any1<G>(g, it.start + e), scale), 0);
        }
    }
}

// Lists up to which one work group takes the tensors' norms and the total: a tensor per wave and turn.
constexpr int64_t kSmallTensors = 64, kSmallItems = 1024;

template <bool MAX>
hipError_t tensor_norms(const NormTables& t, double g_mult, float* norms, hipStream_t s)
{
    if (t.tensors <= kSmallTensors && t.items <= kSmallItems) {
        hipLaunchKernelGGL((k_total_norm<MAX, true>), dim3(1), dim3(kNormBlock), 0, s, t, g_mult, norms);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((k_tensor_norms<MAX>), dim3(static_cast<unsigned>(t.tensors)), dim3(kNormBlock), 0, s, t, g_mult, norms);
    if (hipError_t e = hipGetLastError()) return e;
    hipLaunchKernelGGL((k_total_norm<MAX, false>), dim3(1), dim3(kNormBlock), 0, s, t, g_mult, norms);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_item_norms(const ListLaunch& L, const NormPtrs& ptrs, int g_dtype, int kind, int64_t nt_items, double* partials,
                             hipStream_t s)
{
    const bool max = kind == OB_NORM_MAX;
    const auto k = g_dtype == OB_BF16  ? (max ? k_item_norms<1, true> : k_item_norms<1, false>)
                   : g_dtype == OB_F16 ? (max ? k_item_norms<2, true> : k_item_norms<2, false>)
                                       : (max ? k_item_norms<0, true> : k_item_norms<0, false>);
    hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(L.n_items)), dim3(kListBlock), 0, s, L, ptrs, nt_items, partials);
    return hipGetLastError();
}

hipError_t launch_short_norms(const ListLaunch& L, const NormPtrs& ptrs, int g_dtype, int kind, const NormTables& t, double g_mult,
                              float* norms, hipStream_t s)
{
    const bool max = kind == OB_NORM_MAX;
    const auto k = g_dtype == OB_BF16  ? (max ? k_short_norms<1, true> : k_short_norms<1, false>)
                   : g_dtype == OB_F16 ? (max ? k_short_norms<2, true> : k_short_norms<2, false>)
                                       : (max ? k_short_norms<0, true> : k_short_norms<0, false>);
    hipLaunchKernelGGL(k, dim3(1), dim3(kNormBlock), 0, s, L, ptrs, t, g_mult, norms);
    return hipGetLastError();
}

hipError_t launch_tensor_norms(const NormTables& t, int kind, double g_mult, float* norms, hipStream_t s)
{
    return kind == OB_NORM_MAX ? tensor_norms<true>(t, g_mult, norms, s) : tensor_norms<false>(t, g_mult, norms, s);
}

hipError_t launch_clip(const ListLaunch& L, const ListPtrs& ptrs, int g, int d, const ClipParams& cp, hipStream_t s)
{
    static constexpr void (*kernels[3][3])(ListLaunch, ListPtrs, ClipParams) = {
        {k_clip<0, 0>, k_clip<0, 1>, k_clip<0, 2>}, {k_clip<1, 0>, k_clip<1, 1>, k_clip<1, 2>}, {k_clip<2, 0>, k_clip<2, 1>, k_clip<2, 2>}};
    hipLaunchKernelGGL(kernels[g][d], dim3(static_cast<unsigned>(L.n_items)), dim3(kListBlock), 0, s, L, ptrs, cp);
    return hipGetLastError();
}

}  // namespace ob
