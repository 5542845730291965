// ob_matmul_api.cpp -- host side of the products (declarations and contracts in ob_adam.h).
#include "ob_adam.h"
#include "ob_lists.h"
#include "ob_matmul.h"

namespace {

// How a product that is not refused and not empty is computed.
struct Ways {
    ob::ProductOperand a, b;
    bool chunks;
    ob::ProductPlan plan;
};

// A launch has fewer than 2^32 threads, of which a group has at most 512.
constexpr int64_t kMostTiles = (int64_t(1) << 23) - 1;

Ways ways_of(const ob_product& p, bool may_split)
{
    Ways w;
    w.a = ob::product_operand(p.a_row, p.a_col, p.m, p.k);
    w.b = ob::product_operand(p.b_col, p.b_row, p.n, p.k);
    w.chunks = p.k == 0 || (ob::product_chunks(w.a, p.a, p.batch, p.a_batch, p.m, p.k) &&
                            ob::product_chunks(w.b, p.b, p.batch, p.b_batch, p.n, p.k));
    w.plan = ob::plan_product(p, w.chunks, may_split);
    return w;
}

}  // namespace

extern "C" {

int64_t ob_matmul_workspace(const ob_product* product)
{
    if (ob::check_product(product) != OB_OK) return 0;
    const ob_product& p = *product;
    if (p.batch == 0 || p.m == 0 || p.n == 0) return 0;
    const ob::ProductPlan plan = ways_of(p, true).plan;
    const int64_t side = ob::kTileSize[plan.size];
    return plan.shares.rest * plan.shares.split * side * side * 4;
}

ob_status ob_matmul(const ob_product* product, hipStream_t stream)
try {
    if (ob_status st = ob::check_product(product)) return st;
    const ob_product& p = *product;
    if (p.batch == 0 || p.m == 0 || p.n == 0) return OB_OK;
    const Ways w = ways_of(p, p.workspace != nullptr);
    const ob::TileShares& shares = w.plan.shares;
    ob::ProductArgs args;
    args.a = static_cast<const uint16_t*>(p.a);
    args.b = static_cast<const uint16_t*>(p.b);
    args.c = p.c;
    args.d = p.d;
    args.lda = w.a.ld;
    args.ldb = w.b.ld;
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
    const int64_t size = ob::kTileSize[w.plan.size];
    args.tiles_m = static_cast<int32_t>((p.m + size - 1) / size);
    args.tiles_n = static_cast<int32_t>((p.n + size - 1) / size);
    args.tiles = ob::product_tiles(p.m, p.n, size, p.symmetric);
    args.parts = static_cast<float*>(p.workspace);
    if (args.tiles > INT64_MAX / p.batch) return OB_ERR_ARG;
    const int64_t total = args.tiles * p.batch;
    return ob::for_parts(total, kMostTiles, [&](int64_t first, int64_t count) {
        // the last launch has the tiles that are shared
        const bool last = first + count == total && shares.rest <= count;
        args.first = first;
        args.full = last ? count - shares.rest : count;
        args.split = last ? shares.split : 1;
        const int64_t rest = count - args.full, groups = args.full + rest * args.split;
        (void)hipGetLastError();  // clear a stale error so the check sees this launch only
        const hipError_t e = p.in_type == OB_BF16
                                 ? ob::launch_product<true>(args, w.plan.size, w.a.k_major, w.b.k_major, w.chunks, groups, stream)
                                 : ob::launch_product<false>(args, w.plan.size, w.a.k_major, w.b.k_major, w.chunks, groups, stream);
        if (e != hipSuccess) return OB_ERR_HIP;
        return rest == 0 || ob::launch_product_join(args, w.plan.size, rest, stream) == hipSuccess ? OB_OK : OB_ERR_HIP;
    });
} catch (...) {
    return OB_ERR_OOM;
}

}  // extern "C"
