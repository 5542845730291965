// ob_matmul.hip -- matrix products with a residual; compiled once per operand type (OB_MM_BF16: 0 fp16, 1 bf16).
#include "ob_any.h"
#include "ob_matmul.h"
#include "ob_mfma.h"

#ifndef OB_MM_BF16
#error "OB_MM_BF16 selects the operands' type"
#endif

namespace ob {
namespace {

// Row and column of a matrix's tile `t`.  All: panels of eight rows of tiles, column after column, so that the
// work groups that run together share rows and columns in their XCD's L2.  Symmetric: row after row below the diagonal.
__device__ __forceinline__ void tile_at(const ProductArgs& p, int64_t t, int& i, int& j)
{
    if (p.symmetric) {
        i = static_cast<int>((sqrt(8.0 * static_cast<double>(t) + 1.0) - 1.0) * 0.5);
        while (static_cast<int64_t>(i) * (i + 1) / 2 > t) --i;
        while (static_cast<int64_t>(i + 1) * (i + 2) / 2 <= t) ++i;
        j = static_cast<int>(t - static_cast<int64_t>(i) * (i + 1) / 2);
        return;
    }
    const int64_t panel = static_cast<int64_t>(8) * p.tiles_n, q = t / panel;
    const int rows = min(8, p.tiles_m - static_cast<int>(q) * 8), r = static_cast<int>(t - q * panel);
    i = static_cast<int>(q) * 8 + r % rows;
    j = r / rows;
}

// Work groups go around the eight XCDs; give each XCD a range of consecutive tiles.
__device__ __forceinline__ int64_t by_xcd(int64_t b, int64_t n)
{
    const int64_t each = n / 8, more = n % 8, x = b % 8;
    return x * each + (x < more ? x : more) + b / 8;
}

// Four elements of type D as they are loaded, and widened.
template <int D>
struct Four {
    f4e v;
    __device__ __forceinline__ f4 wide() const { return v; }
};
template <>
struct Four<1> {
    u2e v;
    __device__ __forceinline__ f4 wide() const
    {
        return f4{widen16<1>(v.x & 0xffffu), widen16<1>(v.x >> 16), widen16<1>(v.y & 0xffffu), widen16<1>(v.y >> 16)};
    }
};
template <>
struct Four<2> {
    u2e v;
    __device__ __forceinline__ f4 wide() const
    {
        return f4{widen16<2>(v.x & 0xffffu), widen16<2>(v.x >> 16), widen16<2>(v.y & 0xffffu), widen16<2>(v.y >> 16)};
    }
};

// From element i on, `left` of them there.
template <int D>
__device__ __forceinline__ Four<D> load_four(const char* p, int64_t i, int left)
{
    Four<D> r{};
    if (left >= 4) {
        r.v = *reinterpret_cast<const decltype(r.v)*>(p + i * (D == 0 ? 4 : 2));
    } else if constexpr (D == 0) {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < left) r.v[e] = reinterpret_cast<const float*>(p)[i + e];
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < left) r.v[e >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i + e]) << (16 * (e & 1));
    }
    return r;
}

template <int D>
__device__ __forceinline__ void store_four(char* p, int64_t i, f4 x, int left)
{
    if (left >= 4) {
        if constexpr (D == 0) {
            *reinterpret_cast<f4e*>(p + i * 4) = x;
        } else {
            u2e u;
            u.x = round16x2<D, false>(x.x, x.y, 0, 0);
            u.y = round16x2<D, false>(x.z, x.w, 0, 0);
            *reinterpret_cast<u2e*>(p + i * 2) = u;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (e < left) store_any1<D, false>(p, i + e, x[e], 0);
}

// The result of a tile, WHOLE (all of it is there) or not.  mirror: what is below the diagonal goes above it too.
template <int D, bool WHOLE, class P>
__device__ __forceinline__ void finish_part(const ProductArgs& p, const P& tile, char* lds, int64_t batch, int m0, int n0, bool mirror, int only)
{
    constexpr int64_t kBytes = D == 0 ? 4 : 2;
    const char* c = static_cast<const char*>(p.c) + batch * p.batch_c * kBytes;
    char* d = static_cast<char*>(p.d) + batch * p.batch_d * kBytes;
    auto load = [&](int r, int col) {
        const int i = m0 + r, j = n0 + col;
        if (p.beta == 0.0f || (!WHOLE && (i >= p.m || j >= p.n))) return Four<D>{};
        return load_four<D>(c, i * p.ldc + j, WHOLE ? 4 : p.n - j);
    };
    tile.finish(
        lds, load,
        [&](int r, int col, f4v sum, const Four<D>& old) {
            const int i = m0 + r, j = n0 + col;
            f4v x;
            if (p.beta != 0.0f) {
                const f4 y = old.wide();
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = fmaf(p.alpha, sum[e], p.beta * y[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = p.alpha * sum[e];
            }
            if (WHOLE || (i < p.m && j < p.n)) store_four<D>(d, i * p.ldd + j, x, WHOLE ? 4 : p.n - j);
            return x;
        },
        mirror, [](int, int) { return 0; },
        [&](int r, int col, f4v x, int) {
            const int i = m0 + r, j = n0 + col;
            if (WHOLE || (i < p.m && j < p.n)) store_four<D>(d, j * p.ldd + i, x, WHOLE ? 4 : p.m - i);
        },
        only);
}

template <int D, int TM, class P>
__device__ __forceinline__ void finish_as(const ProductArgs& p, const P& tile, char* lds, int64_t batch, int m0, int n0, int only)
{
    const bool mirror = p.symmetric && m0 != n0;
    if (p.m - m0 >= TM && p.n - n0 >= TM)
        finish_part<D, true>(p, tile, lds, batch, m0, n0, mirror, only);
    else
        finish_part<D, false>(p, tile, lds, batch, m0, n0, mirror, only);
}

template <int TM, class P>
__device__ __forceinline__ void finish(const ProductArgs& p, const P& tile, char* lds, int64_t batch, int m0, int n0, int only)
{
    if (p.out_type == OB_F32)
        finish_as<0, TM>(p, tile, lds, batch, m0, n0, only);
    else if (p.out_type == OB_BF16)
        finish_as<1, TM>(p, tile, lds, batch, m0, n0, only);
    else
        finish_as<2, TM>(p, tile, lds, batch, m0, n0, only);
}

// Matrix, first row and first column of the launch's tile t.  The same in all lanes, which divisions and roots hide: so told,
// addresses stay in scalar registers.
__device__ __forceinline__ void tile_place(const ProductArgs& p, int64_t t, int size, int64_t& batch, int& m0, int& n0)
{
    const int64_t q = (p.first + t) / p.tiles;
    int ti, tj;
    tile_at(p, p.first + t - q * p.tiles, ti, tj);
    batch = __builtin_amdgcn_readfirstlane(static_cast<int>(q));
    m0 = __builtin_amdgcn_readfirstlane(ti) * size;
    n0 = __builtin_amdgcn_readfirstlane(tj) * size;
}

// Tiles of 256 (8 waves), 128 and 64 (4 waves).  fp16: 8192^3 1278 TFLOP/s both by K, 1270 both by rows, 1226 by columns; 4096^3 1245
// and 1189; tiles of 128 4096^3 875, tiles of 64 2048^3 622.  CHUNKS: 16-byte loads straight into LDS; else, for odd sizes, by way of registers
// (4096^3 on tiles of 128 743; 1531 x 1003 x 777 on tiles of 64 13.6 us).
template <int TM, int WM, int WN, bool AK, bool BK, bool CHUNKS>
__global__ __launch_bounds__(64 * (TM / WM) * (TM / WN)) void k_product(ProductArgs p)
{
    using P = TileProduct<TM, TM, WM, WN, OB_MM_BF16 != 0, AK, BK, CHUNKS>;
    __shared__ __attribute__((aligned(16))) char lds[P::kLds];
    const int64_t b = blockIdx.x;
    const bool whole = b < p.full;
    const int64_t q = whole ? 0 : by_xcd(b - p.full, gridDim.x - p.full);   // part of a tile
    int64_t batch;
    int m0, n0, k0 = 0, k = p.k;
    tile_place(p, whole ? by_xcd(b, p.full) : p.full + q / p.split, TM, batch, m0, n0);
    if (!whole) {
        const int64_t steps = (k + P::kTileK - 1) / P::kTileK, part = q % p.split;
        k0 = __builtin_amdgcn_readfirstlane(static_cast<int>(steps * part / p.split) * P::kTileK);
        const int64_t end = steps * (part + 1) / p.split * P::kTileK;
        k = __builtin_amdgcn_readfirstlane(static_cast<int>(end < p.k ? end : p.k)) - k0;
    }
    P tile;
    tile.run(Operand{p.a + batch * p.batch_a + (AK ? m0 * p.lda + k0 : k0 * p.lda + m0), p.lda, p.m - m0, k},
             Operand{p.b + batch * p.batch_b + (BK ? n0 * p.ldb + k0 : k0 * p.ldb + n0), p.ldb, p.n - n0, k}, lds);
    if (whole)
        finish<TM>(p, tile, lds, batch, m0, n0, -1);
    else
        tile.put(p.parts + q * P::kFloats);
}

#if OB_MM_BF16 == 0
// A turn (32 rows of each wave) of one of the tiles that several work groups shared: their sums in order.
template <int TM, int WM, int WN>
__global__ __launch_bounds__(64 * (TM / WM) * (TM / WN)) void k_product_join(ProductArgs p)
{
    using P = TileProduct<TM, TM, WM, WN, false, true, true, true>;
    __shared__ __attribute__((aligned(16))) char lds[P::kLdsOut];
    const int only = static_cast<int>(blockIdx.x % P::kTurnsOut);
    const int64_t t = blockIdx.x / P::kTurnsOut;
    int64_t batch;
    int m0, n0;
    tile_place(p, p.full + t, TM, batch, m0, n0);
    P tile;
    tile.clear();
    for (int s = 0; s < p.split; ++s) tile.add(p.parts + (t * p.split + s) * P::kFloats, only);
    finish<TM>(p, tile, lds, batch, m0, n0, only);
}

template <int TM, int WM, int WN>
hipError_t join(const ProductArgs& p, int64_t rest, hipStream_t s)
{
    hipLaunchKernelGGL((k_product_join<TM, WM, WN>), dim3(static_cast<unsigned>(rest * (WM / 32))), dim3(64 * (TM / WM) * (TM / WN)), 0,
                       s, p);
    return hipGetLastError();
}
#endif

template <int TM, int WM, int WN, bool CHUNKS>
hipError_t launch(const ProductArgs& p, bool ak, bool bk, int64_t count, hipStream_t s)
{
    const dim3 grid(static_cast<unsigned>(count)), block(64 * (TM / WM) * (TM / WN));
    if (ak && bk)
        hipLaunchKernelGGL((k_product<TM, WM, WN, true, true, CHUNKS>), grid, block, 0, s, p);
    else if (ak)
        hipLaunchKernelGGL((k_product<TM, WM, WN, true, false, CHUNKS>), grid, block, 0, s, p);
    else if (bk)
        hipLaunchKernelGGL((k_product<TM, WM, WN, false, true, CHUNKS>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((k_product<TM, WM, WN, false, false, CHUNKS>), grid, block, 0, s, p);
    return hipGetLastError();
}

}  // namespace

template <bool BF16>
hipError_t launch_product(const ProductArgs& p, int size, bool ak, bool bk, bool chunks, int64_t count, hipStream_t s)
{
    if (size == 0) return chunks ? launch<256, 128, 64, true>(p, ak, bk, count, s) : hipErrorInvalidValue;
    if (size == 1) return chunks ? launch<128, 64, 64, true>(p, ak, bk, count, s) : launch<128, 64, 64, false>(p, ak, bk, count, s);
    return chunks ? launch<64, 32, 32, true>(p, ak, bk, count, s) : launch<64, 32, 32, false>(p, ak, bk, count, s);
}

template hipError_t launch_product<OB_MM_BF16 != 0>(const ProductArgs&, int, bool, bool, bool, int64_t, hipStream_t);

#if OB_MM_BF16 == 0
hipError_t launch_product_join(const ProductArgs& p, int size, int64_t rest, hipStream_t s)
{
    return size == 0 ? join<256, 128, 64>(p, rest, s) : size == 1 ? join<128, 64, 64>(p, rest, s) : join<64, 32, 32>(p, rest, s);
}
#endif

}  // namespace ob
