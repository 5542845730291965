// ob_muon_small.hip -- the Muon step for matrices that fit a compute unit's LDS: momentum, norm, all iterations and the update in
// one launch, one work group for each matrix.
#include "ob_muon_device.h"

#include <type_traits>

namespace ob {
namespace {

constexpr int kSmallThreads = 512, kSmallWaves = kSmallThreads / 64;

// The fragment of rows [row0, row0 + 16) of a matrix by K, k in [32 kk, 32 kk + 32): lane l holds row l % 16, eight k from 8 (l / 16) on.
__device__ __forceinline__ s8v by_k(const uint16_t* at, int ld, int row0, int kk)
{
    const int lane = static_cast<int>(threadIdx.x) & 63;
    return *reinterpret_cast<const s8v*>(at + (row0 + (lane & 15)) * ld + kk * 32 + (lane >> 4) * 8);
}
// The same of columns [col0, col0 + 16) of a matrix whose lines are the k.
__device__ __forceinline__ s8v by_columns(const uint16_t* at, int ld, int col0, int kk)
{
    const int lane = static_cast<int>(threadIdx.x) & 63, q = lane & 15;
    const uint16_t* p = at + (kk * 32 + (lane >> 4) * 8 + (q >> 2)) * ld + col0 + (q & 3) * 4;
    const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OB_LDS(s4v, const_cast<uint16_t*>(p)));
    const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OB_LDS(s4v, const_cast<uint16_t*>(p + 4 * ld)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int D>
__device__ __forceinline__ f4 load4_of(const void* p, int64_t i, int left)
{
    if (left >= 4) return load_any4<D>(p, i);
    f4 r{};
    for (int e = 0; e < left; ++e) r[e] = load_any1<D>(p, i + e);
    return r;
}

// f(type as a constant)
template <class F>
__device__ __forceinline__ void by_type(int d, F&& f)
{
    if (d == OB_F32)
        f(std::integral_constant<int, 0>{});
    else if (d == OB_BF16)
        f(std::integral_constant<int, 1>{});
    else
        f(std::integral_constant<int, 2>{});
}

// Block `id` of the lower half of a square of blocks, counted row by row.
__device__ __forceinline__ void block_at(int id, int& i, int& j)
{
    i = 0;
    while (id > i) id -= ++i;
    j = id;
}

// Bound by the waits between its parts (15 products, each behind a barrier), not by rates: eight matrices of 64 x 64 to 5 x 129 21.5 us.  By
// the launches for large matrices (18 of them) 80 us.
// X, A and B = b A + c A^2 stay in LDS (see MuonSmallLayout); a wave takes blocks of 16 x 16 of A and of B, below the diagonal, and
// strips of 16 columns of X, which it alone reads and writes in X = a X + B X.
template <int LDS>
__global__ __launch_bounds__(kSmallThreads) void k_muon_small(MuonCall c, ListPtrs ptrs, int gd, int pk, int iterations)
{
    __shared__ __attribute__((aligned(16))) uint16_t lds[kMuonSmallLds[LDS] / 2];
    if (skips(c)) return;
    const MuonMatrix mt = c.matrices[blockIdx.x];
    const void* g = ptrs.g[mt.place - c.place0];
    if (g == nullptr) return;
    void* p = ptrs.p[mt.place - c.place0];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool tall = mt.rows > mt.cols;
    const int r = tall ? mt.cols : mt.rows, k = tall ? mt.rows : mt.cols, n = mt.rows * mt.cols;

    // the layout: muon_small_layout() of (mt.r, mt.k)
    const int rows = (mt.r + 15) / 16 * 16, sums = (mt.r + 31) / 32 * 32, cols = (mt.k + 31) / 32 * 32;
    const int ldx = cols + 8, lda = sums + 8;
    uint16_t* x = lds;
    uint16_t* a = x + sums * ldx;
    uint16_t* b = a + rows * lda;
    const int end = static_cast<int>(b - lds) + rows * lda;
    float* scratch = reinterpret_cast<float*>(lds + end);                                           // rows <= 32
    double* reduce = reinterpret_cast<double*>(lds + end + (rows <= 32 ? kMuonSmallScratch : 0));   // a number for each wave
    for (int i = tid * 8; i < end; i += kSmallThreads * 8) *reinterpret_cast<u4v*>(lds + i) = u4v{};

    // momentum and the norm of u
    const float scale = grad_scale(c);
    const double mu = c.momentum;
    float* m = c.m + mt.state;
    double s = 0.0;
    by_type(gd, [&](auto type) {
        constexpr int G = decltype(type)::value;
        for (int at = 4 * tid; at < n; at += 4 * kSmallThreads) {
            const int left = n - at;
            const f4 gv = load4_of<G>(g, mt.elem + at, left);
            f4 old{};
            if (left >= 4)
                old = load4u(m, at);
            else
                for (int e = 0; e < left; ++e) old[e] = m[at + e];
            f4 now;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = mul(gv[e], scale);
                now[e] = static_cast<float>(mu * static_cast<double>(old[e]) + (1.0 - mu) * static_cast<double>(y));
                if (e < left) add_square(direction(c, y, now[e]), s);
            }
            if (left >= 4)
                *reinterpret_cast<f4e*>(m + at) = now;
            else
                for (int e = 0; e < left; ++e) m[at + e] = now[e];
        }
    });
    s = wave_sum(s);
    if (lane == 0) reduce[wave] = s;
    __syncthreads();
    s = reduce[0];
#pragma unroll
    for (int w = 1; w < kSmallWaves; ++w) s += reduce[w];
    const float f = static_cast<float>(static_cast<double>(kScaleX) / (sqrt(s) + c.eps));

    // X, smaller side first; a thread reads the momentum that it wrote
    by_type(gd, [&](auto type) {
        constexpr int G = decltype(type)::value;
        for (int at = 4 * tid; at < n; at += 4 * kSmallThreads) {
            const int left = n - at;
            const f4 gv = load4_of<G>(g, mt.elem + at, left);
            f4 mv{};
            if (left >= 4)
                mv = load4u(m, at);
            else
                for (int e = 0; e < left; ++e) mv[e] = m[at + e];
            int row = at / mt.cols, col = at - row * mt.cols;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (e < left) {
                    const _Float16 h = static_cast<_Float16>(mul(direction(c, mul(gv[e], scale), mv[e]), f));
                    x[tall ? col * ldx + row : row * ldx + col] = __builtin_bit_cast(uint16_t, h);
                }
                if (++col == mt.cols) {
                    col = 0;
                    ++row;
                }
            }
        }
    });
    __syncthreads();

    const int side = rows / 16, blocks = side * (side + 1) / 2;
    const int row_of = lane & 15, col_of = (lane >> 4) * 4;   // of a lane's four places in a block
    auto put = [&](uint16_t* to, int i, int j, h4v h) {       // a block of a symmetric matrix, and its mirror image
        *reinterpret_cast<h4v*>(to + (16 * i + row_of) * lda + 16 * j + col_of) = h;
        if (i != j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) reinterpret_cast<_Float16*>(to)[(16 * j + col_of + e) * lda + 16 * i + row_of] = h[e];
        }
    };
    const Rates rate = rates_of(c, mt);
    for (int turn = 0; turn < iterations; ++turn) {
        // A = X X'.  Few blocks: the waves share each one's sum.
        const int share = blocks == 1 ? kSmallWaves : blocks <= 3 ? 2 : 1;
        for (int id = wave / share; id < blocks; id += kSmallWaves / share) {
            int i, j;
            block_at(id, i, j);
            f4v sum{};
            const int steps = cols / 32, part = wave % share;
            for (int kk = steps * part / share; kk < steps * (part + 1) / share; ++kk)
                sum = mfma<false>(by_k(x, ldx, 16 * j, kk), by_k(x, ldx, 16 * i, kk), sum);
            if (share > 1) {   // one turn of this loop
                *reinterpret_cast<f4v*>(scratch + (wave * 64 + lane) * 4) = sum;
                continue;
            }
            h4v h;
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = static_cast<_Float16>(sum[e] * kGram);
            put(a, i, j, h);
        }
        if (share > 1) {
            __syncthreads();
            if (wave < blocks) {
                int i, j;
                block_at(wave, i, j);
                f4v sum{};
                for (int w = 0; w < share; ++w) sum += *reinterpret_cast<const f4v*>(scratch + ((wave * share + w) * 64 + lane) * 4);
                h4v h;
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = static_cast<_Float16>(sum[e] * kGram);
                put(a, i, j, h);
            }
        }
        __syncthreads();
        // B = b A + c A^2
        for (int id = wave; id < blocks; id += kSmallWaves) {
            int i, j;
            block_at(id, i, j);
            f4v sum{};
            for (int kk = 0; kk < sums / 32; ++kk) sum = mfma<false>(by_k(a, lda, 16 * j, kk), by_k(a, lda, 16 * i, kk), sum);
            const h4v old = *reinterpret_cast<const h4v*>(a + (16 * i + row_of) * lda + 16 * j + col_of);
            h4v h;
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = static_cast<_Float16>(fmaf(kC * kUp, sum[e], kB * static_cast<float>(old[e])));
            put(b, i, j, h);
        }
        __syncthreads();
        // X = a X + B X, or the update
        for (int strip = wave; strip < cols / 16; strip += kSmallWaves) {
            f4v sum[kMuonSmallBlocks] = {};
            for (int kk = 0; kk < sums / 32; ++kk) {
                const s8v right = by_columns(x, ldx, 16 * strip, kk);
#pragma unroll
                for (int i = 0; i < kMuonSmallBlocks; ++i)
                    if (i < side) sum[i] = mfma<false>(right, by_k(b, lda, 16 * i, kk), sum[i]);
            }
#pragma unroll
            for (int i = 0; i < kMuonSmallBlocks; ++i) {
                if (i >= side) continue;
                const int row = 16 * i + row_of, col = 16 * strip + col_of;
                h4v* at = reinterpret_cast<h4v*>(x + row * ldx + col);
                const h4v old = *at;
                f4v v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = fmaf(kUp, sum[i][e], kA * static_cast<float>(old[e]));
                if (turn + 1 < iterations) {
                    *at = h4v{static_cast<_Float16>(v[0]), static_cast<_Float16>(v[1]), static_cast<_Float16>(v[2]), static_cast<_Float16>(v[3])};
                    continue;
                }
                if (row >= r) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (col + e >= k) continue;
                    const int64_t q = tall ? static_cast<int64_t>(col + e) * mt.cols + row : static_cast<int64_t>(row) * mt.cols + col + e;
                    float* master = pk >= PK_MASTER_BF16 ? c.master + mt.state + q : nullptr;
                    by_type(pk >= PK_MASTER_BF16 ? pk - 2 : pk, [&](auto type) {
                        constexpr int D = decltype(type)::value;
                        const float now = rate.update(master ? *master : load_any1<D>(p, mt.elem + q), v[e]);
                        if (master) *master = now;
                        store_any1<D, false>(p, mt.elem + q, now, 0);
                    });
                }
            }
        }
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_muon_small(const MuonCall& c, const ListPtrs& ptrs, int64_t matrices, int g_dtype, int pk, int iterations, int lds,
                             hipStream_t s)
{
    const auto k = lds == 0 ? k_muon_small<0> : lds == 1 ? k_muon_small<1> : k_muon_small<2>;
    hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(matrices)), dim3(kSmallThreads), 0, s, c, ptrs, g_dtype, pk, iterations);
    return hipGetLastError();
}

}  // namespace ob
