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
    }
    if (!product_stride(p->m, p->d_row) || !product_stride(p->batch, p->d_batch)) return OB_ERR_ARG;
    // D's elements must not overlap
    if (p->m > 1 && p->d_row < p->n) return OB_ERR_ARG;
    if (p->batch > 1 && p->d_batch < (p->m - 1) * p->d_row + p->n) return OB_ERR_ARG;
    if (!product_aligned(p->d, out)) return OB_ERR_ALIGN;
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

// The tiles of a product: rows and columns of tiles, all of them or those with a part below the diagonal.
inline int64_t product_tiles(int64_t m, int64_t n, int64_t tile, bool symmetric)
{
    const int64_t a = (m + tile - 1) / tile, b = (n + tile - 1) / tile;
    return symmetric ? a * (a + 1) / 2 : a * b;
}

}  // namespace ob
