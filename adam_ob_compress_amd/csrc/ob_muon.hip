// ob_muon.hip -- the Muon step over lists of matrices: momentum with the sums of squares, the normalised matrices in fp16, the
// products of the iterations, and the update in the last product's epilogue.
#include "ob_muon_device.h"

namespace ob {
namespace {

// m = mu m + (1-mu) g', and the sum of u^2 of an item.  One pass: g and m in, m out.  Bound by HBM: 2.0e8 bf16 gradients 355 us, 5.7 TB/s.
template <int G>
__global__ __launch_bounds__(kListBlock) void k_muon_momentum(MuonCall c, ListPtrs ptrs)
{
    __shared__ double lds[kListBlock / 64];
    if (skips(c)) return;
    const MuonItem it = c.items[blockIdx.x];
    const MuonMatrix& mt = c.matrices[it.matrix];
    const void* g = ptrs.g[mt.place - c.place0];
    if (g == nullptr) return;
    const float scale = grad_scale(c);
    const double mu = c.momentum;
    const int64_t gi = mt.elem + it.start;
    float* m = c.m + mt.state + it.start;
    double s = 0.0;
    auto one = [&](float x, float old) {
        const float y = mul(x, scale);
        const float now = static_cast<float>(mu * static_cast<double>(old) + (1.0 - mu) * static_cast<double>(y));
        add_square(direction(c, y, now), s);
        return now;
    };
    for (int at = 4 * static_cast<int>(threadIdx.x); at < it.len; at += kListTile) {
        if (it.len - at >= 4) {
            const f4 x = load_any4<G>(g, gi + at), old = load4u(m, at);
            f4 now;
#pragma unroll
            for (int e = 0; e < 4; ++e) now[e] = one(x[e], old[e]);
            *reinterpret_cast<f4e*>(m + at) = now;
        } else {
            for (int e = at; e < it.len; ++e) m[e] = one(load_any1<G>(g, gi + e), m[e]);
        }
    }
    s = block_sum(s, lds);
    if (threadIdx.x == 0) c.parts[blockIdx.x] = s;
}

// What u is multiplied with: 2^9 / (|u| + eps), one work group for each matrix.
__global__ __launch_bounds__(kListBlock) void k_muon_factor(MuonCall c)
{
    __shared__ double lds[kListBlock / 64];
    if (skips(c)) return;
    const MuonMatrix& mt = c.matrices[blockIdx.x];
    double s = 0.0;
    for (int i = static_cast<int>(threadIdx.x); i < mt.parts; i += kListBlock) s += c.parts[mt.part0 + i];
    s = block_sum(s, lds);
    if (threadIdx.x == 0) c.factor[blockIdx.x] = static_cast<float>(static_cast<double>(kScaleX) / (sqrt(s) + c.eps));
}

// A tile of X from g and m, smaller side first, zeros where the sides are rounded up.  A matrix with more rows than columns is
// turned over in LDS.  u is formed again from g and m (its norm is known only now): 2.0e8 elements 438 us, 3.7 TB/s, 3% of their step.
template <int G>
__global__ __launch_bounds__(kListBlock) void k_muon_write(MuonCall c, ListPtrs ptrs)
{
    constexpr int T = kMuonWriteTile;
    __shared__ float turned[T][T + 1];
    if (skips(c)) return;
    const MuonTile tl = c.write[blockIdx.x];
    const MuonMatrix& mt = c.matrices[tl.matrix];
    const void* g = ptrs.g[mt.place - c.place0];
    if (g == nullptr) return;
    const float scale = grad_scale(c), f = c.factor[tl.matrix];
    const bool tall = mt.rows > mt.cols;
    // the tile in the parameter's orientation
    const int row0 = (tall ? tl.j : tl.i) * T, col0 = (tall ? tl.i : tl.j) * T;
    const int tid = static_cast<int>(threadIdx.x), line = tid >> 4, q = (tid & 15) * 4;
    _Float16* x = reinterpret_cast<_Float16*>(c.half + mt.x[0]);
    const float* m = c.m + mt.state;
    // Four lines of 16 for a thread, all loads before the first store (64 experts of 512 x 1408 83 us; a line at a time 95).
    constexpr int kLines = T / 16;
    f4 gv[kLines], mv[kLines];
    const int col = col0 + q;
#pragma unroll
    for (int k = 0; k < kLines; ++k) {
        const int row = row0 + line + 16 * k;
        const int64_t at = static_cast<int64_t>(row) * mt.cols + col;
        gv[k] = mv[k] = f4{};
        if (row >= mt.rows) continue;
        if (col + 4 <= mt.cols) {
            gv[k] = load_any4<G>(g, mt.elem + at);
            mv[k] = load4u(m, at);
        } else {
            for (int e = 0; e < 3; ++e)
                if (col + e < mt.cols) {
                    gv[k][e] = load_any1<G>(g, mt.elem + at + e);
                    mv[k][e] = m[at + e];
                }
        }
    }
#pragma unroll
    for (int k = 0; k < kLines; ++k) {
        const int i = line + 16 * k, row = row0 + i;
        float v[4];   // zeros, where there is no element
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = row < mt.rows && col + e < mt.cols ? mul(direction(c, mul(gv[k][e], scale), mv[k][e]), f) : 0.0f;
        if (tall) {
#pragma unroll
            for (int e = 0; e < 4; ++e) turned[q + e][i] = v[e];
        } else if (row < mt.r && col < mt.k) {   // k is a multiple of 8
            const h4v h = {static_cast<_Float16>(v[0]), static_cast<_Float16>(v[1]), static_cast<_Float16>(v[2]), static_cast<_Float16>(v[3])};
            *reinterpret_cast<h4v*>(x + static_cast<int64_t>(row) * mt.k + col) = h;
        }
    }
    if (!tall) return;
    __syncthreads();
    for (int i = line; i < T; i += 16) {
        const int row = tl.i * T + i, col = tl.j * T + q;
        if (row >= mt.r || col >= mt.k) continue;
        const h4v h = {static_cast<_Float16>(turned[i][q]), static_cast<_Float16>(turned[i][q + 1]), static_cast<_Float16>(turned[i][q + 2]),
                      static_cast<_Float16>(turned[i][q + 3])};
        *reinterpret_cast<h4v*>(x + static_cast<int64_t>(row) * mt.k + col) = h;
    }
}

// The place of X in an iteration (both are loaded: an index would move the whole description out of the scalar registers).
__device__ __forceinline__ int64_t x_of(const MuonMatrix& mt, int turn) { return turn & 1 ? mt.x[1] : mt.x[0]; }

// The tile's sums for a product: rows from m0, columns from n0 on.
template <int PRODUCT, class P>
__device__ __forceinline__ void muon_sums(P& tile, const MuonCall& c, const MuonMatrix& mt, int turn, int m0, int n0, char* lds)
{
    const uint16_t* x = c.half + x_of(mt, turn);
    if constexpr (PRODUCT == MUON_GRAM)
        tile.run(Operand{x + static_cast<int64_t>(m0) * mt.k, mt.k, mt.r - m0, mt.k},
                 Operand{x + static_cast<int64_t>(n0) * mt.k, mt.k, mt.r - n0, mt.k}, lds);
    else if constexpr (PRODUCT == MUON_POLY)
        tile.run(Operand{c.half + mt.a + static_cast<int64_t>(m0) * mt.r, mt.r, mt.r - m0, mt.r},
                 Operand{c.half + mt.a + static_cast<int64_t>(n0) * mt.r, mt.r, mt.r - n0, mt.r}, lds);
    else
        tile.run(Operand{c.half + mt.b + static_cast<int64_t>(m0) * mt.r, mt.r, mt.r - m0, mt.r},
                 Operand{x + n0, mt.k, mt.k - n0, mt.r}, lds);
}

template <int TM, int WM, int WN, int PRODUCT>
using MuonProduct = TileProduct<TM, TM, WM, WN, false, true, PRODUCT != MUON_STEP, true>;

// One product of an iteration.  Seven matrices of 4096 x 4096 to 4096 x 11008: A 768 us, B 468, X 1506 (1100 TFLOP/s), bound by power and, in
// the symmetric ones, by a last round that fills 72% of the card, in X by a wait of the compiler's (Stage::fragment); 48 of 768 x 768: 50,
// 51 and 76 us, bound by the tiles' ends, X by that wait too.
template <int TM, int WM, int WN, int PRODUCT>
__global__ __launch_bounds__(64 * (TM / WM) * (TM / WN)) void k_muon_product(MuonCall c, const MuonTile* tiles, int turn)
{
    using P = MuonProduct<TM, WM, WN, PRODUCT>;
    __shared__ __attribute__((aligned(16))) char lds[P::kLds];
    if (skips(c)) return;
    const MuonTile tl = tiles[blockIdx.x];
    const MuonMatrix mt = c.matrices[tl.matrix];
    const int m0 = tl.i * TM, n0 = tl.j * TM;
    P tile;
    muon_sums<PRODUCT>(tile, c, mt, turn, m0, n0, lds);
    const _Float16* from = reinterpret_cast<const _Float16*>(c.half + (PRODUCT == MUON_STEP ? x_of(mt, turn) : mt.a));
    _Float16* to = reinterpret_cast<_Float16*>(c.half + (PRODUCT == MUON_GRAM ? mt.a : PRODUCT == MUON_POLY ? mt.b : x_of(mt, turn + 1)));
    const int64_t ld = PRODUCT == MUON_STEP ? mt.k : mt.r;
    const int cols = PRODUCT == MUON_STEP ? mt.k : mt.r;
    // both sides are multiples of 8; A is symmetric, and so is what is added to its sums
    tile.finish(
        lds,
        [&](int r, int col) {
            h4v old{};
            if (PRODUCT != MUON_GRAM && m0 + r < mt.r && n0 + col < cols) old = *reinterpret_cast<const h4v*>(from + (m0 + r) * ld + n0 + col);
            return old;
        },
        [&](int r, int col, f4v s, h4v old) {
            f4v x;
            h4v h;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float o = static_cast<float>(old[e]);
                x[e] = PRODUCT == MUON_GRAM ? s[e] * kGram : PRODUCT == MUON_POLY ? fmaf(kC * kUp, s[e], kB * o) : fmaf(kUp, s[e], kA * o);
                h[e] = static_cast<_Float16>(x[e]);
            }
            if (m0 + r < mt.r && n0 + col < cols) *reinterpret_cast<h4v*>(to + (m0 + r) * ld + n0 + col) = h;
            return x;
        },
        PRODUCT != MUON_STEP && tl.i != tl.j, [](int, int) { return 0; },
        [&](int r, int col, f4v x, int) {
            h4v h;
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = static_cast<_Float16>(x[e]);
            if (m0 + r < mt.r && n0 + col < cols) *reinterpret_cast<h4v*>(to + (n0 + col) * ld + m0 + r) = h;
        });
}

// The last X and the update, where the parameters' 2 to 10 bytes an element join the product's: seven matrices of 4096 x 4096 to 4096 x 11008
// with masters 1746 us, the same step without them 1506.
template <int TM, int WM, int WN, int PK>
__global__ __launch_bounds__(64 * (TM / WM) * (TM / WN)) void k_muon_last(MuonCall c, ListPtrs ptrs, const MuonTile* tiles, int turn)
{
    using P = MuonProduct<TM, WM, WN, MUON_STEP>;
    constexpr bool kMaster = PK == PK_MASTER_BF16 || PK == PK_MASTER_F16;
    constexpr int D = kMaster ? PK - 2 : PK;
    __shared__ __attribute__((aligned(16))) char lds[P::kLds];
    if (skips(c)) return;
    const MuonTile tl = tiles[blockIdx.x];
    const MuonMatrix mt = c.matrices[tl.matrix];
    if (ptrs.g[mt.place - c.place0] == nullptr) return;
    void* p = ptrs.p[mt.place - c.place0];
    const int m0 = tl.i * TM, n0 = tl.j * TM;
    P tile;
    muon_sums<MUON_STEP>(tile, c, mt, turn, m0, n0, lds);

    const Rates q = rates_of(c, mt);
    const bool tall = mt.rows > mt.cols;
    const int rows = tall ? mt.cols : mt.rows, cols = tall ? mt.rows : mt.cols;   // of X, without what was rounded up
    const _Float16* from = reinterpret_cast<const _Float16*>(c.half + x_of(mt, turn));
    float* master = kMaster ? c.master + mt.state : nullptr;
    // Four parameters behind each other from `at` on, `left` of them there: as they are, and updated.
    auto load = [&](int64_t at, int left) {
        f4 was{};
        if (left >= 4)
            was = kMaster ? load4u(master, at) : load_any4<D>(p, mt.elem + at);
        else
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < left) was[e] = kMaster ? master[at + e] : load_any1<D>(p, mt.elem + at + e);
        return was;
    };
    auto store = [&](int64_t at, f4 was, f4v x, int left) {
        f4 now;
#pragma unroll
        for (int e = 0; e < 4; ++e) now[e] = q.update(was[e], x[e]);
        if (left >= 4) {
            if (kMaster) *reinterpret_cast<f4e*>(master + at) = now;
            store_any4<D, false>(p, mt.elem + at, now, u4{});
            return;
        }
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            if (e >= left) continue;
            if (kMaster) master[at + e] = now[e];
            store_any1<D, false>(p, mt.elem + at + e, now[e], 0);
        }
    };
    struct Held {
        h4v x;
        f4 was;
    };
    // a matrix with more rows than columns is turned over: its parameters lie along X's columns
    tile.finish(
        lds,
        [&](int r, int col) {
            const int i = m0 + r, j = n0 + col;
            Held h{};
            if (i >= rows || j >= cols) return h;
            h.x = *reinterpret_cast<const h4v*>(from + static_cast<int64_t>(i) * mt.k + j);
            if (!tall) h.was = load(static_cast<int64_t>(i) * mt.cols + j, cols - j);
            return h;
        },
        [&](int r, int col, f4v s, const Held& h) {
            const int i = m0 + r, j = n0 + col;
            f4v x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = fmaf(kUp, s[e], kA * static_cast<float>(h.x[e]));
            if (!tall && i < rows && j < cols) store(static_cast<int64_t>(i) * mt.cols + j, h.was, x, cols - j);
            return x;
        },
        tall,
        [&](int r, int col) {
            const int i = m0 + r, j = n0 + col;
            return i < rows && j < cols ? load(static_cast<int64_t>(j) * mt.cols + i, rows - i) : f4{};
        },
        [&](int r, int col, f4v x, f4 was) {
            const int i = m0 + r, j = n0 + col;
            if (i < rows && j < cols) store(static_cast<int64_t>(j) * mt.cols + i, was, x, rows - i);
        });
}

template <int TM, int WM, int WN>
hipError_t product(const MuonCall& c, int product, const MuonTile* tiles, int64_t count, int turn, hipStream_t s)
{
    const dim3 grid(static_cast<unsigned>(count)), block(64 * (TM / WM) * (TM / WN));
    if (product == MUON_GRAM)
        hipLaunchKernelGGL((k_muon_product<TM, WM, WN, MUON_GRAM>), grid, block, 0, s, c, tiles, turn);
    else if (product == MUON_POLY)
        hipLaunchKernelGGL((k_muon_product<TM, WM, WN, MUON_POLY>), grid, block, 0, s, c, tiles, turn);
    else
        hipLaunchKernelGGL((k_muon_product<TM, WM, WN, MUON_STEP>), grid, block, 0, s, c, tiles, turn);
    return hipGetLastError();
}

template <int TM, int WM, int WN>
hipError_t last(const MuonCall& c, const ListPtrs& ptrs, const MuonTile* tiles, int64_t count, int turn, int pk, hipStream_t s)
{
    const dim3 grid(static_cast<unsigned>(count)), block(64 * (TM / WM) * (TM / WN));
    switch (pk) {
    case PK_F32: hipLaunchKernelGGL((k_muon_last<TM, WM, WN, PK_F32>), grid, block, 0, s, c, ptrs, tiles, turn); break;
    case PK_BF16: hipLaunchKernelGGL((k_muon_last<TM, WM, WN, PK_BF16>), grid, block, 0, s, c, ptrs, tiles, turn); break;
    case PK_F16: hipLaunchKernelGGL((k_muon_last<TM, WM, WN, PK_F16>), grid, block, 0, s, c, ptrs, tiles, turn); break;
    case PK_MASTER_BF16: hipLaunchKernelGGL((k_muon_last<TM, WM, WN, PK_MASTER_BF16>), grid, block, 0, s, c, ptrs, tiles, turn); break;
    case PK_MASTER_F16: hipLaunchKernelGGL((k_muon_last<TM, WM, WN, PK_MASTER_F16>), grid, block, 0, s, c, ptrs, tiles, turn); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_muon_momentum(const MuonCall& c, const ListPtrs& ptrs, int g, int64_t items, hipStream_t s)
{
    const auto k = g == OB_BF16 ? k_muon_momentum<1> : g == OB_F16 ? k_muon_momentum<2> : k_muon_momentum<0>;
    hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(items)), dim3(kListBlock), 0, s, c, ptrs);
    return hipGetLastError();
}

hipError_t launch_muon_factor(const MuonCall& c, int64_t matrices, hipStream_t s)
{
    hipLaunchKernelGGL(k_muon_factor, dim3(static_cast<unsigned>(matrices)), dim3(kListBlock), 0, s, c);
    return hipGetLastError();
}

hipError_t launch_muon_write(const MuonCall& c, const ListPtrs& ptrs, int g, int64_t tiles, hipStream_t s)
{
    const auto k = g == OB_BF16 ? k_muon_write<1> : g == OB_F16 ? k_muon_write<2> : k_muon_write<0>;
    hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(tiles)), dim3(kListBlock), 0, s, c, ptrs);
    return hipGetLastError();
}

hipError_t launch_muon_product(const MuonCall& c, int kind, const MuonTile* tiles, int64_t count, int tile, int turn, hipStream_t s)
{
    return tile == 0   ? product<256, 128, 64>(c, kind, tiles, count, turn, s)
           : tile == 1 ? product<128, 64, 64>(c, kind, tiles, count, turn, s)
                       : product<64, 32, 32>(c, kind, tiles, count, turn, s);
}

hipError_t launch_muon_last(const MuonCall& c, const ListPtrs& ptrs, const MuonTile* tiles, int64_t count, int tile, int turn, int pk,
                            hipStream_t s)
{
    return tile == 0   ? last<256, 128, 64>(c, ptrs, tiles, count, turn, pk, s)
           : tile == 1 ? last<128, 64, 64>(c, ptrs, tiles, count, turn, pk, s)
                       : last<64, 32, 32>(c, ptrs, tiles, count, turn, pk, s);
}

}  // namespace ob
