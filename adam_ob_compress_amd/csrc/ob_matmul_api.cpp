// ob_matmul_api.cpp -- host side of the products (declarations and contracts in ob_adam.h).
#include "ob_adam.h"
#include "ob_matmul.h"
#include "ob_lists.h"

namespace {

// The largest tile whose count still fills the card: a tile of 256 uses every operand byte it brings into LDS 256 times,
// but 256 work groups are one for each compute unit.
int choose_tile(const ob_product& p, bool chunks)
{
    for (int t = chunks ? ob::TILE_256 : ob::TILE_128; t < ob::TILE_64; ++t)
        if (p.batch * ob::product_tiles(p.m, p.n, ob::kTileSize[t], p.symmetric) >= 192) return t;
    return ob::TILE_64;
}

}  // namespace

extern "C" {

ob_status ob_matmul(const ob_product* product, hipStream_t stream)
try {
    if (ob_status st = ob::check_product(product)) return st;
    const ob_product& p = *product;
    if (p.batch == 0 || p.m == 0 || p.n == 0) return OB_OK;
    const ob::ProductOperand a = ob::product_operand(p.a_row, p.a_col, p.m, p.k);
    const ob::ProductOperand b = ob::product_operand(p.b_col, p.b_row, p.n, p.k);
    const bool chunks = p.k == 0 || (ob::product_chunks(a, p.a, p.batch, p.a_batch, p.m, p.k) &&
                                     ob::product_chunks(b, p.b, p.batch, p.b_batch, p.n, p.k));
    const int tile = choose_tile(p, chunks);
    ob::ProductArgs args;
    args.a = static_cast<const uint16_t*>(p.a);
    args.b = static_cast<const uint16_t*>(p.b);
    args.c = p.c;
    args.d = p.d;
    args.lda = a.ld;
    args.ldb = b.ld;
    args.ldc = p.c_row;
    args.ldd = p.d_row;
    args.batch_a = p.a_batch;
    args.batch_b = p.b_batch;
    args.batch_c = p.c_batch;
    args.batch_d = p.d_batch;
    args.m = static_cast<int32_t>(p.m);
    args.n = static_cast<int32_t>(p.n);
    args.k = static_cast<int32_t>(p.k);
    args.out_type = p.out_type;
    args.alpha = p.alpha;
    args.beta = p.beta;
    args.symmetric = p.symmetric;
    const int size = ob::kTileSize[tile];
    args.tiles_m = static_cast<int32_t>((p.m + size - 1) / size);
    args.tiles_n = static_cast<int32_t>((p.n + size - 1) / size);
    args.tiles = ob::product_tiles(p.m, p.n, size, p.symmetric);
    if (args.tiles > INT64_MAX / p.batch) return OB_ERR_ARG;
    // a launch has fewer than 2^32 threads, of which a group has at most 512
    return ob::for_parts(args.tiles * p.batch, (int64_t(1) << 23) - 1, [&](int64_t first, int64_t count) {
        args.first = first;
        (void)hipGetLastError();  // clear a stale error so the check sees this launch only
        const hipError_t e = p.in_type == OB_BF16
                                 ? ob::launch_product<true>(args, tile, a.k_major, b.k_major, chunks, count, stream)
                                 : ob::launch_product<false>(args, tile, a.k_major, b.k_major, chunks, count, stream);
        return e == hipSuccess ? OB_OK : OB_ERR_HIP;
    });
} catch (...) {
    return OB_ERR_OOM;
}

}  // extern "C"
