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
};

enum { TILE_256 = 0, TILE_128 = 1, TILE_64 = 2 };
constexpr int kTileSize[] = {256, 128, 64};

// Tiles [first, first + count) with the kernel for these layouts; chunks: both operands in 16-byte chunks.
template <bool BF16>
hipError_t launch_product(const ProductArgs& p, int tile, bool a_kmajor, bool b_kmajor, bool chunks, int64_t count, hipStream_t s);

}  // namespace ob
