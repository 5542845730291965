// ob_mfma.h -- one tile of a matrix product on the matrix cores: D = L R for a tile of D, operands of 16 bits, sums in
// fp32.  Used by the products of ob_matmul.hip and by the iterations of ob_muon.hip, which add their epilogues.
//
// L is M x K, R is K x N; both are described by "rows" (of L: its rows; of R: its columns), so that each operand is
// rows x K.  An operand lies by K (K_MAJOR: element (row, k) at row*ld + k) or by rows (k*ld + row).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ob_product.h"

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


// D[n][m] += R[n][k] L[m][k] for a 16 x 16 x 32 block: with R as the first operand a lane ends up with four consecutive
// columns of one row of D, which is what a row-major D is stored by.  Blocks of 32 x 32 x 16 take as many cycles (8192^3: 1.34e6
// and 1.35e6) but run at a lower clock, large products being bound by the power they draw: 931 us and 860.
constexpr int kMfma = 16, kMfmaK = 32;
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

// ROWS x KT elements (KT 64 or 32) of an operand in LDS, as 16-byte chunks whose places are permuted, so that the lanes that
// read fragments together (lanes 0-3, 12-15 and 20-27 of a 16-byte read, and so on) meet different banks:
//   K_MAJOR  a row's KT / 8 chunks along K:  chunk c of row r at place c ^ (r & 7), of four chunks at c ^ (r >> 1 & 3);
//   else     a k's ROWS / 8 chunks along the rows:  chunk c of k at place c ^ 2 f(k), f(k) = k & 3 | (k >> 3 & 3) << 2
//            (two chunks are the 16 rows of a fragment, and the 16 k of one read differ in f).
template <int ROWS, int KT, int THREADS, bool K_MAJOR, bool ASYNC>
struct Stage {
    static constexpr int kBytes = ROWS * KT * 2;
    static constexpr int kLoads = kBytes / 16 / THREADS;   // chunks per thread
    static constexpr int kLine = K_MAJOR ? KT / 8 : ROWS / 8;   // chunks per line (row, or k)
    static_assert(kLoads * THREADS * 16 == kBytes, "every thread loads the same number of chunks");

    static __device__ __forceinline__ int swizzle(int line)
    {
        if (K_MAJOR) return KT == 64 ? line & 7 : line >> 1 & 3;
        return (((line & 3) | ((line >> 3 & 3) << 2)) << 1) & (kLine - 1);
    }

    u4v reg[ASYNC ? 1 : kLoads];
    uint32_t off[ASYNC ? kLoads : 1];         // ASYNC: byte offsets of the thread's chunks from the step's first byte (product_reach())
    const uint16_t* at[ASYNC ? 1 : kLoads];   // else their addresses

    // place of the thread's chunk j: line and chunk in it
    static __device__ __forceinline__ void place(int j, int& line, int& chunk)
    {
        const int q = j * THREADS + static_cast<int>(threadIdx.x);
        line = q / kLine;
        chunk = (q % kLine) ^ swizzle(line);
    }

    __device__ __forceinline__ void begin(const Operand& o)
    {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            int line, chunk;
            place(j, line, chunk);
            const bool in = (K_MAJOR ? line : chunk * 8) < o.rows;
            if constexpr (ASYNC)
                off[j] = in ? static_cast<uint32_t>(line * o.ld + chunk * 8) * 2u : kOutside;
            else   // a row that is not there: another one, whose sums nobody stores
                at[j] = o.p + (K_MAJOR ? (in ? line : 0) * o.ld + chunk * 8 : line * o.ld + (in ? chunk * 8 : 0));
        }
    }

    // Load of step t into LDS at `to` (ASYNC) or into registers.
    __device__ __forceinline__ void load(const Operand& o, int t, char* to)
    {
        const int left = o.k - t * KT;   // k that there are from this step on
        const int64_t step = K_MAJOR ? static_cast<int64_t>(t) * KT : static_cast<int64_t>(t) * KT * o.ld;
        if constexpr (ASYNC) {
            const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(o.p + step), 0, left > 0 ? kInside : 0, 0x00027000);
            const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                uint32_t v = off[j];
                if (left < KT) {
                    int line, chunk;
                    place(j, line, chunk);
                    if ((K_MAJOR ? chunk * 8 : line) >= left) v = kOutside;
                }
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, OB_LDS(void, to + (j * THREADS + wave * 64) * 16), 16,
                                                         static_cast<int>(v), 0, 0, 0);
            }
        } else if (K_MAJOR ? left >= KT : left > KT && o.ld >= 8) {
            // Whole chunks.  By rows, one that reaches past the last row ends before the next k's does, which there is: it meets memory
            // of the operand's, and gives sums that nobody stores.
#pragma unroll
            for (int j = 0; j < kLoads; ++j) reg[j] = *reinterpret_cast<const u4u*>(at[j] + step);
        } else {   // the last step (all, of short lines): nothing behind the operand's end, zeros behind its last k
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                int line, chunk;
                place(j, line, chunk);
                const bool in = (K_MAJOR ? line : chunk * 8) < o.rows;
                const int along = K_MAJOR ? left - chunk * 8 : o.rows - (in ? chunk * 8 : 0);   // elements that there are from the chunk on
                const uint16_t* p = at[j] + step;
                u4v v{};
                if (K_MAJOR || line < left) {
                    if (along >= 8) {
                        v = *reinterpret_cast<const u4u*>(p);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (e < along) v[e >> 1] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
                    }
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
            return *reinterpret_cast<const s8v*>(at + (row0 + r) * (kLine * 16) + ((kk * 4 + g) ^ swizzle(r)) * 16);
        } else {
            // 16 lanes read four k of 16 rows, four rows each, and get four k of one row.  The compiler takes the first of these reads
            // for a possible reader of the loads into LDS that are on their way and waits for all of them (vmcnt(0)), which reads of
            // operands by K do not make it do: on tiles of 128 and 64 a step's loads, issued just before, then overlap with nothing; on
            // tiles of 256 the wait for the next step's alone is void.  1024^3 9.9 us by rows and 8.3 by K.
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
    static constexpr int kFm = WM / kMfma, kFn = WN / kMfma;
    static constexpr bool kTurns = kThreads == 512;   // see run_in_turns
    static constexpr int kStages = kTurns ? 4 : 2, kTileK = kTurns ? 32 : 64;
    static_assert(kTileK <= kTileStep && TM <= 256 && TN <= 256, "product_reach() is about such steps");
    using SL = Stage<TM, kTileK, kThreads, L_KMAJOR, ASYNC>;
    using SR = Stage<TN, kTileK, kThreads, R_KMAJOR, ASYNC>;
    static constexpr int kStage = SL::kBytes + SR::kBytes;
    static constexpr int kLds = kStages * kStage;
    static constexpr int kEach = SL::kLoads + SR::kLoads;   // loads of a step

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

    // The fragments of 32 k from 32 * half on, and their products.
    s8v l[kFm], r[kFn];
    __device__ __forceinline__ void fragments(const char* at, int half)
    {
#pragma unroll
        for (int j = 0; j < kFn; ++j) r[j] = SR::fragment(at + SL::kBytes, wave_n() + kMfma * j, half);
#pragma unroll
        for (int i = 0; i < kFm; ++i) l[i] = SL::fragment(at, wave_m() + kMfma * i, half);
    }
    __device__ __forceinline__ void multiply()
    {
#pragma unroll
        for (int i = 0; i < kFm; ++i)
#pragma unroll
            for (int j = 0; j < kFn; ++j) acc[i][j] = mfma<BF16>(r[j], l[i], acc[i][j]);
    }

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kFm; ++i)
#pragma unroll
            for (int j = 0; j < kFn; ++j) acc[i][j] = f4v{};
    }

    // The sums over all of K; every thread of the group, lds: kLds bytes.
    __device__ __forceinline__ void run(const Operand& lo, const Operand& ro, char* lds)
    {
        clear();
        if constexpr (kTurns)
            run_in_turns(lo, ro, lds);
        else
            run_in_step(lo, ro, lds);
    }

    // Bound by the power that the card may draw: 8192^3 fp16, both by K, 860 us (1278 TFLOP/s), 1.35e6 cycles at 1.58 GHz with the matrix cores
    // busy 77% of them; with all waves reading and multiplying together 1.70e6 cycles, 62%, at 1.96 GHz.  Operands of zeros: 1530 TFLOP/s.
    // By rows also by the wait that Stage::fragment() describes: busy 65% (B by rows), 58% in the Muon step.
    // Two waves share a SIMD, one of each half of the group.  While one multiplies, the other takes its next fragments from LDS and
    // starts loads, and a barrier changes their roles, so that the matrix cores have one wave's work at any time.  With the halves'
    // phases counted through, the first half takes step s in phase 2s and multiplies it in 2s + 1, the second takes it in 2s + 1:
    // step s's buffer is free from phase 2s + 2 on, where loads for step s + 4 go into it, and a step's loads have five phases.
    __device__ __forceinline__ void run_in_turns(const Operand& lo, const Operand& ro, char* lds)
    {
        SL sl;
        SR sr;
        const int steps = (lo.k + kTileK - 1) / kTileK;
        if (steps == 0) return;
        auto load = [&](int t) {   // beyond the last step: zeros that nobody reads
            char* to = lds + t % kStages * kStage;
            sl.load(lo, t, to);
            sr.load(ro, t, to + SL::kBytes);
        };
        sl.begin(lo);
        sr.begin(ro);
        load(0);
        load(1);
        load(2);
        wait_loads<2 * kEach>();
        barrier();
        const bool second = threadIdx.x >= kThreads / 2;
        if (second) barrier();
        for (int t = 0; t < steps; ++t) {
            fragments(lds + t % kStages * kStage, 0);
            load(t + 3);
            wait_loads<2 * kEach>();   // step t + 1 has arrived
            wait_reads();
            barrier();
            __builtin_amdgcn_s_setprio(1);
            multiply();
            __builtin_amdgcn_s_setprio(0);
            barrier();
        }
        if (!second) barrier();
        wait_loads<0>();
    }

    static __device__ __forceinline__ void barrier()
    {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
    // all reads of LDS have arrived; all loads into LDS but the last N have
    static __device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
    template <int N>
    static __device__ __forceinline__ void wait_loads()
    {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
    }

    // Every wave reads a step's fragments and multiplies them, while the operands of the next step are on their way.  (Three steps
    // ahead: 1024^3 on tiles of 64 8.1 us, 7.8 so; 2048^3 31.6 and 26.9, as fewer groups fit.)
    __device__ __forceinline__ void run_in_step(const Operand& lo, const Operand& ro, char* lds)
    {
        SL sl;
        SR sr;
        const int steps = (lo.k + kTileK - 1) / kTileK;
        if (steps == 0) return;
        sl.begin(lo);
        sr.begin(ro);
        sl.load(lo, 0, lds);
        sr.load(ro, 0, lds + SL::kBytes);
        sl.store(lds);
        sr.store(lds + SL::kBytes);
        if (ASYNC) wait_loads<0>();   // what other waves read behind the barrier has arrived
        __syncthreads();
        for (int t = 0; t < steps; ++t) {
            char* at = lds + (t & 1) * kStage;
            char* to = lds + (~t & 1) * kStage;
            if (t + 1 < steps) {
                sl.load(lo, t + 1, to);
                sr.load(ro, t + 1, to + SL::kBytes);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                fragments(at, half);
                multiply();
            }
            if (t + 1 < steps) {
                sl.store(to);
                sr.store(to + SL::kBytes);
            }
            if (ASYNC) wait_loads<0>();
            wait_reads();   // they have left the buffer that the next step's loads go into
            __syncthreads();
        }
    }

    // The sums as they lie in registers, to memory and added from there (of one turn of finish()).
    static constexpr int kFloats = TM * TN;
    __device__ __forceinline__ void put(float* to) const
    {
#pragma unroll
        for (int i = 0; i < kFm; ++i)
#pragma unroll
            for (int j = 0; j < kFn; ++j)
                *reinterpret_cast<f4v*>(to + ((i * kFn + j) * kThreads + static_cast<int>(threadIdx.x)) * 4) = acc[i][j];
    }
    __device__ __forceinline__ void add(const float* from, int only)
    {
#pragma unroll
        for (int i = 0; i < kFm; ++i) {
            if (i / 2 != only) continue;
#pragma unroll
            for (int j = 0; j < kFn; ++j)
                acc[i][j] += *reinterpret_cast<const f4v*>(from + ((i * kFn + j) * kThreads + static_cast<int>(threadIdx.x)) * 4);
        }
    }

    // The tile's sums by way of LDS (the buffers that run() has left), so that a wave meets whole lines of the result, in turns of
    // kRows of its rows.  Every thread of the group; only: the turn that is wanted (-1: all).
    //   x = f(row, column, four sums of the row from the column on, load(row, column))
    //   turned: g(row, column, four x of the column from the row on, load_turned(row, column))
    // A turn's loads are started before the turn before is finished: the results may lie where the loads read, so that the compiler
    // would keep each load behind the store before it, 32 waits in a row (4096 x 11008 x 4096 with a residual 1008 TFLOP/s, so 1104).
    static constexpr int kRows = 2 * kMfma, kTurnsOut = WM / kRows;
    static constexpr int kLdsOut = kRows * (WN + 4) * 4 * (kThreads / 64);
    template <class L, class F, class LT, class G>
    __device__ __forceinline__ void finish(char* lds, L&& load, F&& f, bool turned, LT&& load_turned, G&& g, int only = -1) const
    {
        constexpr int kLd = WN + 4;   // 4 floats more keep the rows of a write in different banks
        constexpr int kEachOut = kRows * WN / 256;   // times four elements of a lane in a turn
        static_assert(kLdsOut <= kLds, "every wave has its part of the buffers");
        const int lane = static_cast<int>(threadIdx.x) & 63, m = wave_m(), n = wave_n();
        float* mine = reinterpret_cast<float*>(lds) + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6) * (kRows * kLd);
        auto row = [&](int k) { return (lane + 64 * k) / (WN / 4); };
        auto col = [&](int k) { return (lane + 64 * k) % (WN / 4) * 4; };
        auto row_turned = [&](int k) { return (lane + 64 * k) % (kRows / 4) * 4; };
        auto col_turned = [&](int k) { return (lane + 64 * k) / (kRows / 4); };
        // two turns' loads if they take no more than 64 registers, else one's
        constexpr int kHeld = sizeof(load(0, 0)) * kEachOut * 2 <= 256 ? 2 : 1;
        decltype(load(0, 0)) held[kHeld][kEachOut];
        decltype(load_turned(0, 0)) held_turned[kEachOut];
        auto start = [&](int h) {
#pragma unroll
            for (int k = 0; k < kEachOut; ++k) held[h % kHeld][k] = load(m + kRows * h + row(k), n + col(k));
        };
        __syncthreads();   // the last fragments have left the buffers
        if (only < 0 && kHeld == 2) start(0);
#pragma unroll
        for (int h = 0; h < kTurnsOut; ++h) {
            if (only >= 0 && h != only) continue;
            if (only >= 0 || kHeld == 1) start(h);
            if (turned) {
#pragma unroll
                for (int k = 0; k < kEachOut; ++k) held_turned[k] = load_turned(m + kRows * h + row_turned(k), n + col_turned(k));
            }
            if (only < 0 && kHeld == 2 && h + 1 < kTurnsOut) start(h + 1);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < kFn; ++j)
                    *reinterpret_cast<f4v*>(mine + (kMfma * i + (lane & 15)) * kLd + kMfma * j + 4 * (lane >> 4)) = acc[2 * h + i][j];
#pragma unroll
            for (int k = 0; k < kEachOut; ++k) {
                f4v* at = reinterpret_cast<f4v*>(mine + row(k) * kLd + col(k));
                const f4v x = f(m + kRows * h + row(k), n + col(k), *at, held[h % kHeld][k]);
                if (turned) *at = x;
            }
            if (turned) {
#pragma unroll
                for (int k = 0; k < kEachOut; ++k) {
                    const float* at = mine + row_turned(k) * kLd + col_turned(k);
                    g(m + kRows * h + row_turned(k), n + col_turned(k), f4v{at[0], at[kLd], at[2 * kLd], at[3 * kLd]}, held_turned[k]);
                }
            }
        }
    }
};

}  // namespace
}  // namespace ob
