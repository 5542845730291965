// ob_matmul.h -- shared between the host side (ob_matmul_api.cpp) and the kernels (ob_matmul.hip) of the products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ob_product.h"

namespace ob {

struct ProductArgs {
    const uint16_t* a;
    const uint16_t* b;
    const void* c;
    void* d;
    int64_t lda, ldb, ldc, ldd;
    int64_t batch_a, batch_b, batch_c, batch_d;
    int32_t m, n, k;
    int32_t out_type;
    float alpha, beta;
    int32_t symmetric;
    int32_t tiles_m, tiles_n;
    int64_t tiles;        // per matrix
    int64_t first;        // of the launch: its first tile, counted over the whole batch
    int64_t full;         // tiles of the launch that one work group takes each; then `split` work groups for each of the rest
    int32_t split;
    float* parts;         // the rest's partial sums: a tile's squared side of floats for each work group
};

// `count` work groups of the kernel for these layouts; size: place in kTileSize; chunks: both operands in 16-byte chunks.
template <bool BF16>
hipError_t launch_product(const ProductArgs& p, int size, bool a_kmajor, bool b_kmajor, bool chunks, int64_t count, hipStream_t s);
// The `rest` tiles behind the full ones from their partial sums.
hipError_t launch_product_join(const ProductArgs& p, int size, int64_t rest, hipStream_t s);

}  // namespace ob
