// ob_muon.h -- the Muon step on the host, in plain C++17: a plan's groups of matrices, their work and their places in the
// workspace, and the checks of a call's arguments.  Used by the host side (ob_muon_api.cpp) and the kernels (ob_muon.hip), and
// checked on the CPU by tests/muon_check.cpp.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "ob_lists.h"
#include "ob_product.h"

namespace ob {

// Matrices are taken with the smaller side first, r x k, both rounded up to 8 elements (16 bytes): what is added holds zeros.
struct MuonMatrix {
    int64_t elem;           // of the tensor: the matrix's first element
    int64_t state;          // its index in the flat states
    int64_t x[2], a, b;     // places in the workspace, in elements of 16 bits: X and the next X, A, b A + c A^2
    int32_t place;          // of its tensor in the list's order
    int32_t rows, cols;
    int32_t r, k;
    int32_t part0, parts;   // its partial sums of squares in the group's
    float lr_mult, wd_mult;
    int32_t reserved;
};

// Elements [start, start + len) of a matrix.
struct MuonItem {
    int64_t start;
    int32_t len;
    int32_t matrix;
};

// A tile of a matrix: rows from i * tile on, columns from j * tile on.
struct MuonTile {
    int32_t matrix, i, j;
};

constexpr int kMuonItem = 8192;       // elements of an item
constexpr int kMuonWriteTile = 64;    // side of the tiles that X is written by

// The three products of an iteration: A = X X^T (symmetric), b A + c A^2 (symmetric), X = a X + B X.
enum { MUON_GRAM = 0, MUON_POLY = 1, MUON_STEP = 2 };

struct MuonRange {
    int64_t first, count;
};

// Matrices that go through the iterations together, of one pair of types and at most kListPtrs tensors.
struct MuonGroup {
    int64_t place0, places;       // tensors in the list's order
    MuonRange matrices, items, write;
    MuonRange tiles[3];           // by product
    int32_t tile[3];              // place in kTileSize
};

// Matrices of one pair of types that fit a compute unit's LDS each: one launch does their whole step.
struct MuonSmall {
    int64_t place0, places;
    MuonRange matrices;
    int32_t lds;                  // place in kMuonSmallLds
};

// LDS that such a launch's work groups have: four, two or one of them on a compute unit.
constexpr int kMuonSmallSizes = 3;
constexpr int64_t kMuonSmallLds[kMuonSmallSizes] = {40 << 10, 80 << 10, 160 << 10};
constexpr int kMuonSmallBlocks = 10;   // blocks of 16 rows of the smaller side at most

// Layout of such a matrix in LDS, in elements of 16 bits: X with its rows up to a multiple of 32 (they are the sum's index in B X), its
// columns too, and 8 more elements to a line, so that lines start in different banks; A and B likewise.
struct MuonSmallLayout {
    int32_t rows, sums, cols;     // r up to 16 and to 32, k up to 32
    int32_t ldx, lda, a, b, scratch;
    int64_t bytes;
};
// One block of A alone, or three: the waves share their sums, by way of 8 KB.
constexpr int kMuonSmallScratch = 4096;
inline MuonSmallLayout muon_small_layout(int64_t r, int64_t k)
{
    MuonSmallLayout l{};
    const int64_t rows = (r + 15) / 16 * 16, sums = (r + 31) / 32 * 32, cols = (k + 31) / 32 * 32;
    const int64_t x = sums * (cols + 8), a = rows * (sums + 8), scratch = rows <= 32 ? kMuonSmallScratch : 0;
    l.bytes = 2 * (x + 2 * a + scratch) + 128;
    if (l.bytes > kMuonSmallLds[kMuonSmallSizes - 1]) return l;
    l.rows = static_cast<int32_t>(rows);
    l.sums = static_cast<int32_t>(sums);
    l.cols = static_cast<int32_t>(cols);
    l.ldx = l.cols + 8;
    l.lda = l.sums + 8;
    l.a = static_cast<int32_t>(x);
    l.b = static_cast<int32_t>(x + a);
    l.scratch = static_cast<int32_t>(x + 2 * a);
    return l;
}
inline bool muon_is_small(int64_t r, int64_t k)
{
    return r <= 16 * kMuonSmallBlocks && muon_small_layout(r, k).bytes <= kMuonSmallLds[kMuonSmallSizes - 1];
}

struct MuonShape {
    std::vector<MuonMatrix> matrices;
    std::vector<MuonItem> items;
    std::vector<MuonTile> write, tiles;
    std::vector<MuonGroup> groups;
    std::vector<MuonSmall> small;
    int64_t half_elems = 0;       // the largest group's 16-bit elements
    int64_t parts = 0, most = 0;  // its partial sums, its matrices
    int64_t workspace() const { return 2 * half_elems + 8 * parts + 4 * (most + most % 2); }
};

constexpr int64_t kMuonSide = int64_t(1) << 30;
// Workspace that a group of several matrices may take: room for enough tiles to fill the card many times over.
constexpr int64_t kMuonGroupBytes = int64_t(2) << 30;
inline int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

inline int64_t muon_tile_count(const MuonMatrix& m, int product, int64_t size)
{
    return product == MUON_STEP ? product_tiles(m.r, m.k, size, false) : product_tiles(m.r, m.r, size, true);
}

// Whether a tile of this side can load what the product has of the matrix (with a side of many millions it may not).
inline bool muon_reach(const MuonMatrix& m, int product, int64_t size)
{
    const int64_t lines = std::min<int64_t>(size, m.r);
    if (product == MUON_GRAM) return product_reach(lines, m.k);
    return product_reach(lines, m.r) && (product != MUON_STEP || product_reach(std::min<int64_t>(kTileStep, m.r), m.k));
}

// Tiles of all matrices [m0, m1) for `product`, ordered for a launch: work groups go around the eight XCDs, each of which
// gets one part of every matrix, in panels of eight rows of tiles (those below the diagonal row by row).
inline void muon_tiles(const std::vector<MuonMatrix>& mats, int64_t m0, int64_t m1, int product, int64_t size, std::vector<MuonTile>& out)
{
    std::vector<MuonTile> by[8], all;
    for (int64_t q = m0; q < m1; ++q) {
        const int64_t ti = (mats[q].r + size - 1) / size, tj = product == MUON_STEP ? (mats[q].k + size - 1) / size : ti;
        all.clear();
        const int32_t id = static_cast<int32_t>(q - m0);
        if (product == MUON_STEP) {
            for (int64_t p = 0; p < ti; p += 8)
                for (int64_t j = 0; j < tj; ++j)
                    for (int64_t i = p; i < std::min(ti, p + 8); ++i) all.push_back({id, static_cast<int32_t>(i), static_cast<int32_t>(j)});
        } else {
            for (int64_t i = 0; i < ti; ++i)
                for (int64_t j = 0; j <= i; ++j) all.push_back({id, static_cast<int32_t>(i), static_cast<int32_t>(j)});
        }
        // the parts start at another XCD for each matrix, so that small matrices spread
        const int64_t n = static_cast<int64_t>(all.size());
        for (int64_t x = 0; x < 8; ++x)
            for (int64_t t = n * x / 8; t < n * (x + 1) / 8; ++t) by[(x + q) % 8].push_back(all[t]);
    }
    int64_t total = 0;
    for (const auto& v : by) total += static_cast<int64_t>(v.size());
    // XCD x gets the places x, x + 8, ...; what some have too much goes to those that have too little
    std::vector<MuonTile> spare;
    int64_t want[8];
    for (int64_t x = 0; x < 8; ++x) {
        want[x] = total / 8 + (x < total % 8);
        while (static_cast<int64_t>(by[x].size()) > want[x]) {
            spare.push_back(by[x].back());
            by[x].pop_back();
        }
    }
    for (int64_t x = 0; x < 8; ++x)
        while (static_cast<int64_t>(by[x].size()) < want[x]) {
            by[x].push_back(spare.back());
            spare.pop_back();
        }
    for (int64_t t = 0; t < total; ++t) out.push_back(by[t % 8][static_cast<size_t>(t / 8)]);
}

// A group of the matrices from m0 on, all of whose tensors are in places [place0, place0 + places).
inline bool muon_close(MuonShape& s, int64_t m0, int64_t place0, int64_t places)
{
    const int64_t m1 = static_cast<int64_t>(s.matrices.size());
    MuonGroup g{};
    g.place0 = place0;
    g.places = places;
    g.matrices = {m0, m1 - m0};
    // the longest sums first, so that the last work groups are short ones
    std::stable_sort(s.matrices.begin() + m0, s.matrices.end(), [](const MuonMatrix& a, const MuonMatrix& b) { return a.k > b.k; });
    g.items.first = static_cast<int64_t>(s.items.size());
    g.write.first = static_cast<int64_t>(s.write.size());
    int64_t at = 0, parts = 0;
    auto room = [&](int64_t n) {   // n elements at a multiple of 256 bytes
        const int64_t x = at;
        at += (n + 127) / 128 * 128;
        return x;
    };
    for (int64_t q = m0; q < m1; ++q) {
        MuonMatrix& m = s.matrices[q];
        const int64_t n = static_cast<int64_t>(m.rows) * m.cols;
        m.part0 = static_cast<int32_t>(parts);
        for (int64_t i = 0; i < n; i += kMuonItem) {
            s.items.push_back({i, static_cast<int32_t>(std::min<int64_t>(kMuonItem, n - i)), static_cast<int32_t>(q - m0)});
            ++parts;
        }
        m.parts = static_cast<int32_t>(parts - m.part0);
        for (int32_t i = 0; i < (m.r + kMuonWriteTile - 1) / kMuonWriteTile; ++i)
            for (int32_t j = 0; j < (m.k + kMuonWriteTile - 1) / kMuonWriteTile; ++j) s.write.push_back({static_cast<int32_t>(q - m0), i, j});
        m.x[0] = room(static_cast<int64_t>(m.r) * m.k);
        m.x[1] = room(static_cast<int64_t>(m.r) * m.k);
        m.a = room(static_cast<int64_t>(m.r) * m.r);
        m.b = room(static_cast<int64_t>(m.r) * m.r);
        if (parts > INT32_MAX) return false;
    }
    g.items.count = static_cast<int64_t>(s.items.size()) - g.items.first;
    g.write.count = static_cast<int64_t>(s.write.size()) - g.write.first;
    for (int product = 0; product < 3; ++product) {
        double least = -1.0;
        int64_t count = 0;
        for (int t = 0; t < kTileSizes; ++t) {
            int64_t n = 0;
            double k_sum = 0.0;   // over the tiles
            bool reach = true;
            for (int64_t q = m0; q < m1; ++q) {
                const MuonMatrix& m = s.matrices[q];
                reach = reach && muon_reach(m, product, kTileSize[t]);
                const int64_t tiles = muon_tile_count(m, product, kTileSize[t]);
                n += tiles;
                k_sum += static_cast<double>(tiles) * (product == MUON_GRAM ? m.k : m.r);
            }
            const double us = tile_round(t, n, k_sum / static_cast<double>(n));
            if (!reach || n > INT32_MAX / 512 || (least >= 0.0 && us >= least)) continue;
            least = us;
            count = n;
            g.tile[product] = t;
        }
        if (least < 0.0) return false;
        g.tiles[product] = {static_cast<int64_t>(s.tiles.size()), count};
        muon_tiles(s.matrices, m0, m1, product, kTileSize[g.tile[product]], s.tiles);
    }
    s.half_elems = std::max(s.half_elems, at);
    s.parts = std::max(s.parts, parts);
    s.most = std::max(s.most, m1 - m0);
    s.groups.push_back(g);
    return true;
}

inline ob_status build_muon(const ListShape& l, const float* lr_mults, const float* wd_mults, const int64_t* rows, const int64_t* cols,
                            int64_t most_places, MuonShape& s)
{
    const size_t T = l.size.size();
    if (T > 0 && (!rows || !cols)) return OB_ERR_ARG;
    for (size_t t = 0; t < T; ++t) {
        if (rows[t] < 1 || cols[t] < 1 || rows[t] > kMuonSide || cols[t] > kMuonSide) return OB_ERR_ARG;
        if (l.size[t] % (rows[t] * cols[t]) != 0) return OB_ERR_ARG;
    }
    bool fits = true;
    const ob_status st = for_runs(l, most_places, true, [&](int64_t k, int64_t e) {
        // f(matrix, its place) for the run's matrices that are small, or are not
        auto each = [&](bool small, auto&& f) {
            for (int64_t j = k; j < e; ++j) {
                const int32_t t = l.order[j];
                const int64_t n = rows[t] * cols[t];
                const int64_t r = up8(std::min(rows[t], cols[t])), c = up8(std::max(rows[t], cols[t]));
                if (muon_is_small(r, c) != small) continue;
                for (int64_t x = 0; x < l.size[t]; x += n) {
                    MuonMatrix m{};
                    m.elem = x;
                    m.state = l.state_off[t] + x;
                    m.place = static_cast<int32_t>(j);
                    m.rows = static_cast<int32_t>(rows[t]);
                    m.cols = static_cast<int32_t>(cols[t]);
                    m.r = static_cast<int32_t>(r);
                    m.k = static_cast<int32_t>(c);
                    m.lr_mult = lr_mults ? lr_mults[j] : 1.0f;
                    m.wd_mult = wd_mults ? wd_mults[j] : 1.0f;
                    f(m, j);
                }
            }
        };
        const int64_t first = static_cast<int64_t>(s.matrices.size());
        int64_t most = 0;
        each(true, [&](const MuonMatrix& m, int64_t) {
            most = std::max(most, muon_small_layout(m.r, m.k).bytes);
            s.matrices.push_back(m);
        });
        int64_t m0 = static_cast<int64_t>(s.matrices.size());
        if (m0 > first) {
            // the longest first, so that the last work groups are short ones
            std::stable_sort(s.matrices.begin() + first, s.matrices.end(), [](const MuonMatrix& a, const MuonMatrix& b) {
                return static_cast<int64_t>(a.r) * a.k > static_cast<int64_t>(b.r) * b.k;
            });
            fits = fits && m0 - first <= INT32_MAX / 512;
            s.small.push_back({k, e - k, {first, m0 - first}, most <= kMuonSmallLds[0] ? 0 : most <= kMuonSmallLds[1] ? 1 : 2});
        }
        int64_t place0 = k, bytes = 0;
        each(false, [&](const MuonMatrix& m, int64_t j) {
            const int64_t takes = 4 * static_cast<int64_t>(m.r) * m.k + 4 * static_cast<int64_t>(m.r) * m.r;
            if (bytes > 0 && bytes + takes > kMuonGroupBytes) {
                fits = fits && muon_close(s, m0, place0, j - place0 + 1);
                m0 = static_cast<int64_t>(s.matrices.size());
                bytes = 0;
            }
            if (bytes == 0) place0 = j;
            bytes += takes;
            s.matrices.push_back(m);
        });
        if (static_cast<int64_t>(s.matrices.size()) > m0) fits = fits && muon_close(s, m0, place0, e - place0);
        return OB_OK;
    });
    if (st != OB_OK) return st;
    return fits ? OB_OK : OB_ERR_ARG;
}

inline ob_status check_muon(const ListShape& l, const void* const* g, void* const* p, const float* master, const float* m,
                            const void* workspace, int64_t workspace_bytes, const ob_muon_hparams* hp, const ob_control* control)
{
    if (!hp) return OB_ERR_ARG;
    if (!std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay)) return OB_ERR_ARG;
    if (!(hp->momentum >= 0.0f && hp->momentum < 1.0f)) return OB_ERR_ARG;
    if (!std::isfinite(hp->eps) || hp->eps < 1e-30f) return OB_ERR_ARG;
    if ((hp->nesterov != 0 && hp->nesterov != 1) || hp->iterations < 1 || hp->iterations > 16 || hp->reserved != 0) return OB_ERR_ARG;
    if (hp->scale != OB_MUON_PLAIN && hp->scale != OB_MUON_SHAPE && hp->scale != OB_MUON_MATCH_RMS) return OB_ERR_ARG;
    if (control && !is_aligned(control, 8)) return OB_ERR_ALIGN;
    if (l.n == 0) return OB_OK;
    if (!p || !m || (workspace_bytes > 0 && !workspace)) return OB_ERR_ARG;
    if (!is_aligned(m, 16) || !is_aligned(master, 16) || !is_aligned(workspace, 16)) return OB_ERR_ALIGN;
    return check_pointers(l, g, p);
}

}  // namespace ob
