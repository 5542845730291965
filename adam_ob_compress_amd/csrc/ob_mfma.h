// ob_mfma.h -- one tile of a matrix product on the matrix cores: D = L R for a tile of D, operands of 16 bits, sums in
// fp32.  Used by the products of ob_matmul.hip and by the iterations of ob_muon.hip, which add their epilogues.
//
// L is M x K, R is K x N; both are described by "rows" (of L: its rows; of R: its columns), so that each operand is
// rows x K.  An operand lies by K (K_MAJOR: element (row, k) at row*ld + k) or by rows (k*ld + row).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ob {
namespace {

typedef float f4v __attribute__((ext_vector_type(4)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));
typedef _Float16 h8v __attribute__((ext_vector_type(8)));
typedef __bf16 b8v __attribute__((ext_vector_type(8)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef uint32_t u4u __attribute__((ext_vector_type(4), aligned(2)));

#define OB_LDS(T, p) ((__attribute__((address_space(3))) T*)(p))

constexpr int kTileK = 64;    // K of a step: 128 bytes of a row

// D[n][m] += R[n][k] L[m][k] for a 16 x 16 x 32 block: with R as the first operand a lane ends up with four
// consecutive columns of one row of D, which is what a row-major D is stored by.
template <bool BF16>
__device__ __forceinline__ f4v mfma(s8v r, s8v l, f4v acc)
{
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8v, r), __builtin_bit_cast(b8v, l), acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, r), __builtin_bit_cast(h8v, l), acc, 0, 0, 0);
}

// An operand as a tile sees it: its rows [row0, row0 + extent) and K.
struct Operand {
    const uint16_t* p;   // at (row0, 0)
    int64_t ld;          // elements
    int rows;            // rows there are from row0 on (more than a tile's: all of them)
    int k;
};

// ROWS x kTileK elements of an operand in LDS, as 16-byte chunks whose places are permuted, so that neither the
// reads of fragments nor the writes meet the same bank twice:
//   K_MAJOR  a row's 8 chunks along K:  chunk c of row r at place c ^ (r & 7);
//   else     a k's ROWS / 8 chunks along the rows:  chunk c of k at place c ^ 2 f(k), f(k) = k & 3 | (k >> 3 & 3) << 2
//            (two chunks are the 16 rows of a fragment, and the 16 k of one read differ in f).
template <int ROWS, int THREADS, bool K_MAJOR, bool ASYNC>
struct Stage {
    static constexpr int kBytes = ROWS * kTileK * 2;
    static constexpr int kLoads = kBytes / 16 / THREADS;   // chunks per thread
    static constexpr int kLine = K_MAJOR ? 8 : ROWS / 8;   // chunks per line (row, or k)
    static_assert(kLoads * THREADS * 16 == kBytes, "every thread loads the same number of chunks");

    static __device__ __forceinline__ int swizzle(int line)
    {
        return K_MAJOR ? line & 7 : (((line & 3) | ((line >> 3 & 3) << 2)) << 1) & (kLine - 1);
    }

    u4v reg[ASYNC ? 1 : kLoads];
    uint32_t off[ASYNC ? kLoads : 1];   // byte offsets of the thread's chunks from the step's first byte

    // place of the thread's chunk j: line and chunk in it
    static __device__ __forceinline__ void place(int j, int& line, int& chunk)
    {
        const int q = j * THREADS + static_cast<int>(threadIdx.x);
        line = q / kLine;
        chunk = (q % kLine) ^ swizzle(line);
    }

    __device__ __forceinline__ void begin(const Operand& o)
    {
        if constexpr (ASYNC) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                int line, chunk;
                place(j, line, chunk);
                const bool in = (K_MAJOR ? line : chunk * 8) < o.rows;
                off[j] = in ? static_cast<uint32_t>(line * o.ld + chunk * 8) * 2u : kOutside;
            }
        }
    }

    // Load of step t into LDS at `to` (ASYNC) or into registers.
    __device__ __forceinline__ void load(const Operand& o, int t, char* to)
    {
        const int left = o.k - t * kTileK;   // k that there are from this step on
        const uint16_t* base = o.p + (K_MAJOR ? static_cast<int64_t>(t) * kTileK : static_cast<int64_t>(t) * kTileK * o.ld);
        if constexpr (ASYNC) {
            const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), 0, kInside, 0x00027000);
            const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                uint32_t v = off[j];
                if (left < kTileK) {
                    int line, chunk;
                    place(j, line, chunk);
                    if ((K_MAJOR ? chunk * 8 : line) >= left) v = kOutside;
                }
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, OB_LDS(void, to + (j * THREADS + wave * 64) * 16), 16,
                                                         static_cast<int>(v), 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                int line, chunk;
                place(j, line, chunk);
                const int along = (K_MAJOR ? left : o.rows) - chunk * 8;             // elements that there are from the chunk on
                const bool there = line < (K_MAJOR ? o.rows : left);
                const uint16_t* p = base + line * o.ld + chunk * 8;
                u4v v{};
                if (there && along >= 8) {
                    v = *reinterpret_cast<const u4u*>(p);
                } else if (there) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < along) v[e >> 1] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
                }
                reg[j] = v;
            }
        }
    }

    // What load() put into registers, into LDS.
    __device__ __forceinline__ void store(char* to)
    {
        if constexpr (!ASYNC) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                *reinterpret_cast<u4v*>(to + (j * THREADS + static_cast<int>(threadIdx.x)) * 16) = reg[j];
        }
    }

    // The fragment of rows [row0, row0 + 16) (row0 a multiple of 16) and k in [32 kk, 32 kk + 32): lane l holds row l % 16,
    // eight k from 8 (l / 16) on.
    static __device__ __forceinline__ s8v fragment(const char* at, int row0, int kk)
    {
        const int lane = static_cast<int>(threadIdx.x) & 63, r = lane & 15, g = lane >> 4;
        if constexpr (K_MAJOR) {
            return *reinterpret_cast<const s8v*>(at + (row0 + r) * 128 + ((kk * 4 + g) ^ (r & 7)) * 16);
        } else {
            // 16 lanes read four k of 16 rows, four rows each, and get four k of one row
            const int k = kk * 32 + g * 8 + (r >> 2);
            const int c = ((row0 >> 3) + (r >> 1 & 1)) ^ swizzle(k);
            const char* p = at + k * (kLine * 16) + c * 16 + (r & 1) * 8;
            const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OB_LDS(s4v, p));
            const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OB_LDS(s4v, p + 4 * kLine * 16));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

private:
    static constexpr uint32_t kOutside = 0x80000000u;   // beyond kInside: the load gives zeros
    static constexpr int kInside = 0x7fffffff;
};

// A tile of TM x TN by waves of WM x WN.
template <int TM, int TN, int WM, int WN, bool BF16, bool L_KMAJOR, bool R_KMAJOR, bool ASYNC>
struct TileProduct {
    static constexpr int kWavesN = TN / WN, kThreads = 64 * (TM / WM) * kWavesN;
    static constexpr int kFm = WM / 16, kFn = WN / 16;
    using SL = Stage<TM, kThreads, L_KMAJOR, ASYNC>;
    using SR = Stage<TN, kThreads, R_KMAJOR, ASYNC>;
    static constexpr int kStage = SL::kBytes + SR::kBytes;
    static constexpr int kLds = 2 * kStage;

    f4v acc[kFm][kFn];

    // first row and column of the wave's part
    static __device__ __forceinline__ int wave_m()
    {
        return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6) / kWavesN * WM;
    }
    static __device__ __forceinline__ int wave_n()
    {
        return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6) % kWavesN * WN;
    }

    __device__ __forceinline__ void fragments(const char* at, int kk, s8v (&l)[kFm], s8v (&r)[kFn])
    {
#pragma unroll
        for (int j = 0; j < kFn; ++j) r[j] = SR::fragment(at + SL::kBytes, wave_n() + 16 * j, kk);
#pragma unroll
        for (int i = 0; i < kFm; ++i) l[i] = SL::fragment(at, wave_m() + 16 * i, kk);
    }
    __device__ __forceinline__ void multiply(const s8v (&l)[kFm], const s8v (&r)[kFn])
    {
#pragma unroll
        for (int i = 0; i < kFm; ++i)
#pragma unroll
            for (int j = 0; j < kFn; ++j) acc[i][j] = mfma<BF16>(r[j], l[i], acc[i][j]);
    }

    // The sums over all of K; every thread of the group, lds: kLds bytes.
    __device__ __forceinline__ void run(const Operand& lo, const Operand& ro, char* lds)
    {
        SL sl;
        SR sr;
#pragma unroll
        for (int i = 0; i < kFm; ++i)
#pragma unroll
            for (int j = 0; j < kFn; ++j) acc[i][j] = f4v{};
        const int steps = (lo.k + kTileK - 1) / kTileK;
        if (steps == 0) return;
        sl.begin(lo);
        sr.begin(ro);
        sl.load(lo, 0, lds);
        sr.load(ro, 0, lds + SL::kBytes);
        sl.store(lds);
        sr.store(lds + SL::kBytes);
        __syncthreads();
        for (int t = 0; t < steps; ++t) {
            char* at = lds + (t & 1) * kStage;
            char* to = lds + (~t & 1) * kStage;
            if (t + 1 < steps) {
                sl.load(lo, t + 1, to);
                sr.load(ro, t + 1, to + SL::kBytes);
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                s8v l[kFm], r[kFn];
                fragments(at, kk, l, r);
                multiply(l, r);
            }
            if (t + 1 < steps) {
                sl.store(to);
                sr.store(to + SL::kBytes);
            }
            __syncthreads();
        }
    }

    // f(row, column, four sums of the row from the column on) for all of the lane's places in the tile.
    template <class F>
    __device__ __forceinline__ void each(F&& f) const
    {
        const int lane = static_cast<int>(threadIdx.x) & 63;
#pragma unroll
        for (int i = 0; i < kFm; ++i)
#pragma unroll
            for (int j = 0; j < kFn; ++j) f(wave_m() + 16 * i + (lane & 15), wave_n() + 16 * j + 4 * (lane >> 4), acc[i][j]);
    }
};

}  // namespace
}  // namespace ob
