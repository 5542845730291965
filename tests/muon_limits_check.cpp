// muon_limits_check.cpp -- CPU check of how far the tiles of a Muon plan's products reach: a tile's loads have byte offsets of 32
// bits from its first element, and a load that ends behind 2^31 - 1 bytes gives zeros.  Prints "ok <checks>".
#include <cstdio>
#include <cstdlib>

#include <vector>

#include "ob_muon.h"

static long checks = 0;
#define CHECK(x)                                              \
    do {                                                      \
        ++checks;                                             \
        if (!(x)) {                                           \
            std::printf("line %d: %s\n", __LINE__, #x);       \
            std::exit(1);                                     \
        }                                                     \
    } while (0)

constexpr int64_t kInside = (int64_t(1) << 31) - 1;   // bytes that a tile's loads may reach

// Where the last 16 bytes end that a tile of `size` loads in a step: of an operand by K (its rows are lines of `ld`, of which it takes
// `step` elements) and of one by rows (each k is a line, of which it takes the tile's rows).
static int64_t by_k(int64_t size, int64_t rows, int64_t ld, int64_t step)
{
    return 2 * ((std::min(size, rows) - 1) * ld + std::min(step, ld));
}
static int64_t by_rows(int64_t size, int64_t k, int64_t ld, int64_t step)
{
    return 2 * ((std::min(step, k) - 1) * ld + std::min(size, ld));
}

// The plan of E matrices of rows x cols: its status, and its reach if it is one.
static ob_status plan(int64_t E, int64_t rows, int64_t cols, int64_t* tile = nullptr)
{
    const int64_t size = E * rows * cols;
    const int32_t type = OB_BF16;
    ob::ListShape l;
    CHECK(ob::build_shape(1, &size, &type, &type, nullptr, nullptr, l) == OB_OK);
    ob::MuonShape s;
    const ob_status st = ob::build_muon(l, nullptr, nullptr, &rows, &cols, 200, s);
    if (st != OB_OK) return st;
    for (const ob::MuonGroup& g : s.groups) {
        for (int64_t q = 0; q < g.matrices.count; ++q) {
            const ob::MuonMatrix& m = s.matrices[g.matrices.first + q];
            for (int p = 0; p < 3; ++p) {
                const int64_t t = ob::kTileSize[g.tile[p]], step = t == 256 ? 32 : 64;
                if (tile) tile[p] = t;
                const int64_t reach = p == ob::MUON_GRAM   ? by_k(t, m.r, m.k, step)
                                      : p == ob::MUON_POLY ? by_k(t, m.r, m.r, step)
                                                           : std::max(by_k(t, m.r, m.r, step), by_rows(t, m.r, m.k, step));
                if (reach > kInside)
                    std::printf("%lld x %lld, product %d on tiles of %lld: %lld bytes\n", static_cast<long long>(rows),
                                static_cast<long long>(cols), p, static_cast<long long>(t), static_cast<long long>(reach));
                CHECK(reach <= kInside);
            }
        }
    }
    return OB_OK;
}

struct Mat {
    int64_t e, r, c;
};

// The tiles of a list's only group.
static void check_tiles(const std::vector<Mat>& mats, int64_t gram, int64_t poly, int64_t step)
{
    std::vector<int64_t> size, rows, cols;
    for (const Mat& m : mats) {
        size.push_back(m.e * m.r * m.c);
        rows.push_back(m.r);
        cols.push_back(m.c);
    }
    const std::vector<int32_t> type(mats.size(), OB_F32);
    ob::ListShape l;
    CHECK(ob::build_shape(static_cast<int64_t>(mats.size()), size.data(), type.data(), type.data(), nullptr, nullptr, l) == OB_OK);
    ob::MuonShape s;
    CHECK(ob::build_muon(l, nullptr, nullptr, rows.data(), cols.data(), 200, s) == OB_OK);
    CHECK(s.groups.size() == 1);
    const int64_t want[3] = {gram, poly, step};
    for (int p = 0; p < 3; ++p) CHECK(ob::kTileSize[s.groups[0].tile[p]] == want[p]);
}

int main()
{
    // the lists of tests/test_gpu_muon_large.py take every tile
    check_tiles({{2, 203, 300}, {1, 300, 203}, {1, 169, 178}, {1, 171, 169}}, 64, 64, 64);
    check_tiles({{7, 521, 777}, {6, 777, 520}}, 64, 64, 128);
    check_tiles({{100, 201, 203}, {103, 202, 197}}, 64, 64, 256);
    check_tiles({{4, 1100, 1301}, {4, 1303, 1101}}, 128, 128, 256);
    check_tiles({{32, 509, 1403}, {1, 1403, 510}, {31, 1402, 507}}, 256, 256, 256);
    // inside the limit for every tile; what fits only smaller tiles takes those; on both sides of the limit for the smallest
    int64_t tile[3];
    CHECK(plan(1, 4096, 11008) == OB_OK);
    CHECK(plan(1, 256, 4'000'000) == OB_OK);
    CHECK(plan(1, 256, 8'388'608, tile) == OB_OK && tile[0] == 64);
    CHECK(plan(1, 8'600'000, 128, tile) == OB_OK && tile[0] == 64);
    CHECK(plan(3, 128, 8'600'000) == OB_OK);
    CHECK(plan(1, 64, 17'000'000) == OB_OK);
    CHECK(plan(1, 64, 17'100'000) == OB_ERR_ARG);
    CHECK(plan(1, 17'100'000, 64) == OB_ERR_ARG);
    CHECK(plan(1, 1000, 17'100'000) == OB_ERR_ARG);
    CHECK(plan(1, 64, 1 << 25) == OB_ERR_ARG);
    CHECK(plan(1, 1 << 25, 40) == OB_ERR_ARG);
    CHECK(plan(1, 32, 34'000'000) == OB_OK);
    CHECK(plan(1, 32, 40'000'000) == OB_ERR_ARG);
    CHECK(plan(1, 1, 150'000'000) == OB_OK);
    CHECK(plan(1, 8, 160'000'000) == OB_ERR_ARG);
    CHECK(plan(1, 1, (int64_t(1) << 30) - 512) == OB_ERR_ARG);
    // around the limit, by steps of a line's 8 elements, in both orientations
    for (int64_t r : {8, 16, 24, 40, 56, 64, 72, 128, 192, 256, 320}) {
        const int64_t lines = std::min<int64_t>(r, 64) - 1, edge = (int64_t(1) << 30) / lines / 8 * 8;
        for (int64_t d = -64; d <= 64; d += 8) {
            const ob_status a = plan(1, r, edge + d), b = plan(1, edge + d, r);
            CHECK(a == b);
            if (d == -64) CHECK(a == OB_OK);
            if (d == 64) CHECK(a == OB_ERR_ARG);
        }
    }
    std::printf("ok %ld\n", checks);
    return 0;
}
