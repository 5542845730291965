// ob_product.h -- matrix products on the host, in plain C++17: the checks of a call's arguments and the choice of a
// kernel.  Used by the host side (ob_matmul_api.cpp) and checked on the CPU by tests/product_check.cpp.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "ob_adam.h"

namespace ob {

// Offsets stay below 2^60 elements, so that byte offsets and their sums fit 63 bits.
constexpr int64_t kProductReach = int64_t(1) << 60;
constexpr int64_t kProductMost = INT32_MAX - 256;   // an extent rounded up to a tile fits 31 bits

// extent steps of stride stay within reach
inline bool product_stride(int64_t extent, int64_t stride)
{
    return stride >= 0 && (extent <= 1 || stride <= kProductReach / (extent - 1));
}

inline bool product_aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline ob_status check_product(const ob_product* p)
{
    if (!p) return OB_ERR_ARG;
    for (int64_t x : {p->batch, p->m, p->n, p->k})
        if (x < 0 || x > kProductMost) return OB_ERR_ARG;
    if (p->in_type != OB_BF16 && p->in_type != OB_F16) return OB_ERR_DTYPE;
    if (p->out_type != OB_F32 && p->out_type != OB_BF16 && p->out_type != OB_F16) return OB_ERR_DTYPE;
    if (!std::isfinite(p->alpha) || !std::isfinite(p->beta)) return OB_ERR_ARG;
    if (p->symmetric != 0 && p->symmetric != 1) return OB_ERR_ARG;
    if (p->symmetric && p->m != p->n) return OB_ERR_ARG;
    if (p->reserved != 0) return OB_ERR_ARG;
    if (p->batch == 0 || p->m == 0 || p->n == 0) return OB_OK;
    if (!p->d || (p->beta != 0.0f && !p->c) || (p->k > 0 && (!p->a || !p->b))) return OB_ERR_ARG;
    const uintptr_t out = p->out_type == OB_F32 ? 4 : 2;
    if (p->k > 0) {
        if (p->a_row != 1 && p->a_col != 1) return OB_ERR_ARG;
        if (p->b_row != 1 && p->b_col != 1) return OB_ERR_ARG;
        if (!product_stride(p->m, p->a_row) || !product_stride(p->k, p->a_col) || !product_stride(p->batch, p->a_batch) ||
            !product_stride(p->k, p->b_row) || !product_stride(p->n, p->b_col) || !product_stride(p->batch, p->b_batch))
            return OB_ERR_ARG;
        if (!product_aligned(p->a, 2) || !product_aligned(p->b, 2)) return OB_ERR_ALIGN;
        if (p->d == p->a || p->d == p->b) return OB_ERR_ARG;   // work groups still read what others have written
    }
    if (!product_stride(p->m, p->d_row) || !product_stride(p->batch, p->d_batch)) return OB_ERR_ARG;
    // D's elements must not overlap
    if (p->m > 1 && p->d_row < p->n) return OB_ERR_ARG;
    if (p->batch > 1 && p->d_batch < (p->m - 1) * p->d_row + p->n) return OB_ERR_ARG;
    if (!product_aligned(p->d, out) || !product_aligned(p->workspace, 16)) return OB_ERR_ALIGN;
    if (p->beta != 0.0f) {
        if (!product_stride(p->m, p->c_row) || !product_stride(p->batch, p->c_batch)) return OB_ERR_ARG;
        if (!product_aligned(p->c, out)) return OB_ERR_ALIGN;
    }
    return OB_OK;
}

// An operand as the kernels see it: rows (of A, columns of B), by K or by rows.
struct ProductOperand {
    bool k_major;
    int64_t ld;
};

// Which of the two strides is the unit one; where both are 1, the one whose other extent is one or none.
inline ProductOperand product_operand(int64_t row_stride, int64_t k_stride, int64_t rows, int64_t k)
{
    const bool by_k = k_stride == 1 && (row_stride != 1 || rows <= 1 || k > 1);
    if (by_k) return {true, rows <= 1 ? std::max<int64_t>(k, 1) : row_stride};
    return {false, k <= 1 ? std::max<int64_t>(rows, 1) : k_stride};
}

// Whether an operand may be read 16 bytes at a time straight into LDS: no chunk of 8 elements is misaligned or reaches
// past the operand, and a tile's offsets fit 31 bits.
inline bool product_chunks(const ProductOperand& o, const void* p, int64_t batch, int64_t batch_stride, int64_t rows, int64_t k)
{
    const int64_t along = o.k_major ? k : rows, lines = o.k_major ? rows : k;
    return product_aligned(p, 16) && along % 8 == 0 && (lines <= 1 || o.ld % 8 == 0) && o.ld < (int64_t(1) << 21) &&
           (batch <= 1 || batch_stride % 8 == 0);
}

// k that a tile takes in a step at most; its loads have byte offsets of 32 bits from the step's first element, and one that ends
// behind 2^31 - 1 gives zeros.
constexpr int64_t kTileStep = 64;
// Whether the loads of `lines` lines (rows of an operand by K, k of one by rows), ld elements apart, stay within that; up to 256 elements
// of a line are taken.
inline bool product_reach(int64_t lines, int64_t ld) { return lines <= 1 || ld <= ((int64_t(1) << 30) - 1 - 256) / (lines - 1); }

// The tiles of a product: rows and columns of tiles, all of them or those with a part below the diagonal.
inline int64_t product_tiles(int64_t m, int64_t n, int64_t tile, bool symmetric)
{
    const int64_t a = (m + tile - 1) / tile, b = (n + tile - 1) / tile;
    return symmetric ? a * (a + 1) / 2 : a * b;
}

// How a launch's tiles are given to work groups: `full` of them to one each, and the `rest`, which would leave compute units
// idle, to `split` each, whose parts of K are added by another launch.
struct TileShares {
    int64_t full, rest;
    int32_t split;      // 1: rest is 0
};

// What the choice goes by.  kTileRate: operations a microsecond with one, two, ... work groups of a size on each of the 256
// compute units, of which a unit holds kTileHeld (by LDS).  kTilePower: what the whole card sustains, where its clock falls with the
// power that is drawn (a card half filled with tiles of 256 runs each a third faster).  kTileExtra: microseconds that a round takes
// besides its sums.  Measured on fp16 products of 256^3 to 4096^3, 64 x 64 x 65536, and symmetric ones of 528 to 2112 tiles, operands
// in 16-byte chunks: the estimates are within a fifth of those times.  Operands by way of registers are planned with the same rates and
// take longer (1531 x 1003 x 777: 9.0 us estimated, 15.6 to 16.1 measured).
constexpr int kTileSizes = 3;
constexpr int64_t kTileSize[kTileSizes] = {256, 128, 64};
constexpr int kTileHeld[kTileSizes] = {1, 2, 4};
constexpr double kTileRate[kTileSizes][4] = {{1784e6}, {640e6, 1000e6}, {290e6, 540e6, 640e6, 720e6}};
constexpr double kTilePower[kTileSizes] = {1200e6, 950e6, 700e6};
constexpr double kTileExtra[kTileSizes] = {8.0, 4.0, 3.0};
constexpr int64_t kUnits = 256;
// The launch that adds partial sums: microseconds, and bytes a microsecond (written, then read).
constexpr double kJoin = 5.0, kJoinBytes = 1.6e6;
constexpr int32_t kMostSplit = 16;
constexpr int64_t kLeastSteps = 8;                // of 32 k that a part has

// Microseconds for `tiles` tiles with sums over k.
inline double tile_round(int size, int64_t tiles, double k)
{
    const int held = kTileHeld[size];
    const int64_t slots = kUnits * held, rounds = tiles / slots, left = tiles % slots, n = (left + kUnits - 1) / kUnits;
    const double work = 2.0 * static_cast<double>(kTileSize[size] * kTileSize[size]) * k;
    double units = static_cast<double>(rounds * slots) / kTileRate[size][held - 1];
    if (left > 0) units += static_cast<double>(n * kUnits) / kTileRate[size][n - 1];
    const double power = static_cast<double>(tiles) / kTilePower[size];
    return work * std::max(units, power) + kTileExtra[size] * static_cast<double>(rounds + (left > 0));
}

// The best shares of `tiles` tiles, sums over k (the shortest, of those in a launch's last round) and their time.
inline TileShares tile_shares(int size, int64_t tiles, int64_t k, bool may_split, double& us)
{
    TileShares best{tiles, 0, 1};
    us = tile_round(size, tiles, static_cast<double>(k));
    const int64_t rest = tiles % (kUnits * kTileHeld[size]);
    if (!may_split || rest == 0) return best;
    const double before = tile_round(size, tiles - rest, static_cast<double>(k));
    for (int32_t s = 2; s <= kMostSplit && k / s >= 32 * kLeastSteps; ++s) {
        const double bytes = 8.0 * static_cast<double>(rest * s * kTileSize[size] * kTileSize[size]);
        const double t = before + tile_round(size, rest * s, static_cast<double>(k) / s) + kJoin + bytes / kJoinBytes;
        if (t < us) {
            us = t;
            best = {tiles - rest, rest, s};
        }
    }
    return best;
}

// The tile size and the shares that take the least time.  chunks: operands in 16-byte chunks; by way of registers there is no largest
// tile.
struct ProductPlan {
    int size;
    TileShares shares;
};
inline ProductPlan plan_product(const ob_product& p, bool chunks, bool may_split)
{
    ProductPlan best{};
    double least = -1.0;
    for (int size = chunks ? 0 : 1; size < kTileSizes; ++size) {
        const int64_t each = product_tiles(p.m, p.n, kTileSize[size], p.symmetric != 0);
        if (each > INT64_MAX / p.batch) continue;
        double us;
        const TileShares s = tile_shares(size, each * p.batch, std::max<int64_t>(p.k, 1), may_split, us);
        if (least < 0.0 || us < least) {
            least = us;
            best = {size, s};
        }
    }
    return best;
}

}  // namespace ob
