// muon_check.cpp -- CPU checks of the Muon plan's host side (ob_muon.h): groups, places in the workspace, items and tiles, and
// the refusals.  Prints "ok <checks>".
#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include <tuple>

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

struct Mat {
    int64_t e, r, c;
};

static ob::ListShape list_of(const std::vector<Mat>& m, const std::vector<int32_t>& gd, const std::vector<int32_t>& pd)
{
    std::vector<int64_t> sizes;
    for (const Mat& x : m) sizes.push_back(x.e * x.r * x.c);
    ob::ListShape l;
    CHECK(ob::build_shape(static_cast<int64_t>(m.size()), sizes.data(), gd.data(), pd.data(), nullptr, nullptr, l) == OB_OK);
    return l;
}

// Everything that a plan promises.
static void check_plan(const std::vector<Mat>& mats, const std::vector<int32_t>& gd, const std::vector<int32_t>& pd, int64_t places)
{
    const ob::ListShape l = list_of(mats, gd, pd);
    std::vector<int64_t> rows, cols;
    std::vector<float> lr, wd;
    for (const Mat& m : mats) {
        rows.push_back(m.r);
        cols.push_back(m.c);
    }
    for (size_t k = 0; k < mats.size(); ++k) {
        lr.push_back(1.0f + static_cast<float>(k));
        wd.push_back(2.0f + static_cast<float>(k));
    }
    ob::MuonShape s;
    CHECK(ob::build_muon(l, lr.data(), wd.data(), rows.data(), cols.data(), places, s) == OB_OK);
    std::set<std::pair<int32_t, int64_t>> seen;   // (place, first element) of every matrix
    int64_t want = 0;
    for (const Mat& m : mats) want += m.e;
    CHECK(static_cast<int64_t>(s.matrices.size()) == want);
    // one matrix of a group or launch: in a tensor of it, with its description
    auto described = [&](const ob::MuonMatrix& m, int64_t place0, int64_t count) {
        CHECK(m.place >= place0 && m.place < place0 + count);
        const int32_t t = l.order[m.place], t0 = l.order[place0];
        CHECK(l.g_dtype[t] == l.g_dtype[t0] && l.p_dtype[t] == l.p_dtype[t0]);
        CHECK(m.rows == rows[t] && m.cols == cols[t] && m.state == l.state_off[t] + m.elem);
        CHECK(m.elem % (rows[t] * cols[t]) == 0 && m.elem < l.size[t]);
        CHECK(seen.insert({m.place, m.elem}).second);
        CHECK(m.r % 8 == 0 && m.k % 8 == 0 && m.r >= std::min(m.rows, m.cols) && m.k >= std::max(m.rows, m.cols) &&
              m.r < std::min(m.rows, m.cols) + 8 && m.k < std::max(m.rows, m.cols) + 8);
        CHECK(m.lr_mult == lr[m.place] && m.wd_mult == wd[m.place]);
    };
    for (const ob::MuonSmall& q : s.small) {
        CHECK(q.places >= 1 && q.places <= places && q.matrices.count >= 1 && q.lds >= 0 && q.lds < ob::kMuonSmallSizes);
        for (int64_t k = 0; k < q.matrices.count; ++k) {
            const ob::MuonMatrix& m = s.matrices[q.matrices.first + k];
            described(m, q.place0, q.places);
            CHECK(ob::muon_is_small(m.r, m.k));
            const ob::MuonSmallLayout y = ob::muon_small_layout(m.r, m.k);
            // as the kernel lays it out: X, A, B, the waves' shares of a sum, a number for each wave
            CHECK(y.rows % 16 == 0 && y.sums % 32 == 0 && y.cols % 32 == 0 && y.rows <= 16 * ob::kMuonSmallBlocks);
            CHECK(y.rows >= m.r && y.sums >= y.rows && y.cols >= m.k && y.ldx >= y.cols + 8 && y.lda >= y.sums + 8);
            CHECK(y.a == y.sums * y.ldx && y.b == y.a + y.rows * y.lda && y.scratch == y.b + y.rows * y.lda);
            CHECK(y.bytes >= 2 * (y.scratch + (y.rows <= 32 ? 8 * 64 * 8 : 0)) + 8 * 8 && y.bytes <= ob::kMuonSmallLds[q.lds]);
        }
    }
    for (const ob::MuonGroup& g : s.groups) {
        CHECK(g.places >= 1 && g.places <= places && g.matrices.count >= 1);
        int64_t bytes = 0;
        std::vector<std::pair<int64_t, int64_t>> room;
        std::vector<bool> part;
        for (int64_t q = 0; q < g.matrices.count; ++q) {
            const ob::MuonMatrix& m = s.matrices[g.matrices.first + q];
            described(m, g.place0, g.places);
            CHECK(!ob::muon_is_small(m.r, m.k));
            for (int64_t x : {m.x[0], m.x[1], m.a, m.b}) CHECK(x % 128 == 0);
            const int64_t rk = static_cast<int64_t>(m.r) * m.k, rr = static_cast<int64_t>(m.r) * m.r;
            room.push_back({m.x[0], rk});
            room.push_back({m.x[1], rk});
            room.push_back({m.a, rr});
            room.push_back({m.b, rr});
            bytes += 4 * rk + 4 * rr;
            CHECK(m.part0 + m.parts <= s.parts);
        }
        CHECK(bytes <= ob::kMuonGroupBytes || g.matrices.count == 1);
        CHECK(g.matrices.count <= s.most);
        std::sort(room.begin(), room.end());
        for (size_t k = 0; k < room.size(); ++k)
            CHECK(room[k].first + room[k].second <= (k + 1 < room.size() ? room[k + 1].first : s.half_elems));
        // items: every element of every matrix once, in order, each with a partial sum of its own
        std::vector<int64_t> next(g.matrices.count), parts(g.matrices.count);
        for (int64_t k = 0; k < g.items.count; ++k) {
            const ob::MuonItem& it = s.items[g.items.first + k];
            const ob::MuonMatrix& m = s.matrices[g.matrices.first + it.matrix];
            CHECK(it.start == next[it.matrix] && it.len > 0 && it.len <= ob::kMuonItem);
            CHECK(k == m.part0 + parts[it.matrix]);
            next[it.matrix] += it.len;
            ++parts[it.matrix];
        }
        for (int64_t q = 0; q < g.matrices.count; ++q) {
            const ob::MuonMatrix& m = s.matrices[g.matrices.first + q];
            CHECK(next[q] == static_cast<int64_t>(m.rows) * m.cols && parts[q] == m.parts);
        }
        // tiles: every tile of every matrix once (below the diagonal, of the symmetric products)
        auto cover = [&](const std::vector<ob::MuonTile>& tiles, ob::MuonRange range, int64_t size, bool symmetric) {
            std::set<std::tuple<int32_t, int32_t, int32_t>> have;
            for (int64_t k = 0; k < range.count; ++k) {
                const ob::MuonTile& t = tiles[range.first + k];
                const ob::MuonMatrix& m = s.matrices[g.matrices.first + t.matrix];
                CHECK(t.i >= 0 && t.j >= 0 && t.i * size < m.r && t.j * size < (symmetric ? m.r : m.k) && (!symmetric || t.j <= t.i));
                CHECK(have.insert(std::make_tuple(t.matrix, t.i, t.j)).second);
            }
            int64_t n = 0;
            for (int64_t q = 0; q < g.matrices.count; ++q) {
                const ob::MuonMatrix& m = s.matrices[g.matrices.first + q];
                const int64_t a = (m.r + size - 1) / size, b = (m.k + size - 1) / size;
                n += symmetric ? a * (a + 1) / 2 : a * b;
            }
            CHECK(n == range.count);
        };
        cover(s.write, g.write, ob::kMuonWriteTile, false);
        for (int p = 0; p < 3; ++p) cover(s.tiles, g.tiles[p], ob::kTileSize[g.tile[p]], p != ob::MUON_STEP);
    }
    CHECK(static_cast<int64_t>(seen.size()) == want);
    CHECK(s.workspace() % 8 == 0);
}

static ob_muon_hparams good()
{
    ob_muon_hparams hp{};
    hp.lr = 1e-3f;
    hp.momentum = 0.95f;
    hp.weight_decay = 0.1f;
    hp.eps = 1e-7f;
    hp.nesterov = 1;
    hp.iterations = 5;
    hp.scale = OB_MUON_MATCH_RMS;
    return hp;
}

int main()
{
    check_plan({{1, 64, 64}, {1, 100, 37}, {1, 5, 129}}, {0, 0, 0}, {0, 0, 0}, 200);
    check_plan({{32, 512, 1408}, {32, 1408, 512}, {1, 1, 1}}, {1, 1, 1}, {1, 1, 1}, 200);
    check_plan({{1, 4096, 4096}, {1, 11008, 4096}, {1, 4096, 11008}, {1, 7, 4096}}, {1, 1, 1, 1}, {1, 1, 1, 1}, 200);
    // mixed types, few places per launch, empty tensors, a tensor whose matrices fill more than one group
    check_plan({{1, 64, 64}, {0, 9, 9}, {3, 100, 37}, {1, 5, 129}, {2, 1, 70}, {1, 70, 1}, {1, 1, 1}}, {0, 1, 1, 2, 0, 1, 0}, {0, 1, 1, 0, 0, 0, 1}, 2);
    check_plan({{40, 4096, 4096}, {2, 300, 20}}, {0, 0}, {0, 0}, 200);
    check_plan({{1, 32000, 4096}, {1, 65536, 8192}, {1, 16, 16}}, {0, 0, 0}, {0, 0, 0}, 200);
    check_plan({}, {}, {}, 200);
    // around the limits of a compute unit's LDS, long thin ones, small ones between large ones
    check_plan({{1, 160, 160}, {1, 161, 160}, {1, 168, 168}, {3, 128, 256}, {1, 64, 1100}, {1, 16, 2300}, {1, 2400, 9}, {1, 700, 64}, {5, 33, 17}, {1, 4000, 4000}},
               {0, 0, 0, 0, 0, 0, 0, 0, 0, 0}, {0, 0, 0, 0, 0, 0, 0, 0, 0, 0}, 200);
    CHECK(ob::muon_is_small(160, 160) && !ob::muon_is_small(168, 168) && ob::muon_is_small(128, 256) && !ob::muon_is_small(128, 512));
    CHECK(ob::muon_is_small(16, 2048) && !ob::muon_is_small(8, 4096) && !ob::muon_is_small(INT64_C(1) << 30, INT64_C(1) << 30));

    // refusals of a plan
    const std::vector<Mat> one{{2, 8, 4}};
    const ob::ListShape l = list_of(one, {0}, {0});
    auto build = [&](int64_t r, int64_t c) {
        ob::MuonShape s;
        return ob::build_muon(l, nullptr, nullptr, &r, &c, 200, s);
    };
    CHECK(build(8, 4) == OB_OK && build(4, 8) == OB_OK && build(64, 1) == OB_OK);
    CHECK(build(0, 4) == OB_ERR_ARG && build(-8, -4) == OB_ERR_ARG && build(7, 4) == OB_ERR_ARG);
    CHECK(build(INT64_C(1) << 31, 4) == OB_ERR_ARG && build(INT64_C(1) << 30, INT64_C(1) << 30) == OB_ERR_ARG);
    ob::MuonShape none;
    CHECK(ob::build_muon(l, nullptr, nullptr, nullptr, nullptr, 200, none) == OB_ERR_ARG);

    // refusals of a step
    const void* g[1] = {reinterpret_cast<void*>(0x1000)};
    void* p[1] = {reinterpret_cast<void*>(0x2000)};
    const float* m = reinterpret_cast<float*>(0x3000);
    const void* w = reinterpret_cast<void*>(0x4000);
    const ob_muon_hparams hp = good();
    CHECK(ob::check_muon(l, g, p, nullptr, m, w, 64, &hp, nullptr) == OB_OK);
    CHECK(ob::check_muon(l, g, p, nullptr, m, w, 64, nullptr, nullptr) == OB_ERR_ARG);
    CHECK(ob::check_muon(l, nullptr, p, nullptr, m, w, 64, &hp, nullptr) == OB_ERR_ARG);
    CHECK(ob::check_muon(l, g, nullptr, nullptr, m, w, 64, &hp, nullptr) == OB_ERR_ARG);
    CHECK(ob::check_muon(l, g, p, nullptr, nullptr, w, 64, &hp, nullptr) == OB_ERR_ARG);
    CHECK(ob::check_muon(l, g, p, nullptr, m, nullptr, 64, &hp, nullptr) == OB_ERR_ARG);
    CHECK(ob::check_muon(l, g, p, nullptr, m + 1, w, 64, &hp, nullptr) == OB_ERR_ALIGN);
    CHECK(ob::check_muon(l, g, p, m + 1, m, w, 64, &hp, nullptr) == OB_ERR_ALIGN);
    CHECK(ob::check_muon(l, g, p, nullptr, m, reinterpret_cast<void*>(0x4008), 64, &hp, nullptr) == OB_ERR_ALIGN);
    CHECK(ob::check_muon(l, g, p, nullptr, m, w, 64, &hp, reinterpret_cast<ob_control*>(0x5004)) == OB_ERR_ALIGN);
    void* odd[1] = {reinterpret_cast<void*>(0x2002)};
    CHECK(ob::check_muon(l, g, odd, nullptr, m, w, 64, &hp, nullptr) == OB_ERR_ALIGN);
    CHECK(ob::check_muon(l, g, p, nullptr, m, nullptr, 0, &hp, nullptr) == OB_OK);   // a plan that needs none
    const void* no[1] = {nullptr};
    void* nop[1] = {nullptr};
    CHECK(ob::check_muon(l, no, nop, nullptr, m, w, 64, &hp, nullptr) == OB_OK);   // no gradient: nothing to do
    auto with = [&](auto&& change) {
        ob_muon_hparams h = good();
        change(h);
        return ob::check_muon(l, g, p, nullptr, m, w, 64, &h, nullptr);
    };
    using H = ob_muon_hparams;
    const float nan = std::nanf("");
    CHECK(with([&](H& h) { h.lr = nan; }) == OB_ERR_ARG);
    CHECK(with([](H& h) { h.weight_decay = INFINITY; }) == OB_ERR_ARG);
    CHECK(with([](H& h) { h.momentum = 1.0f; }) == OB_ERR_ARG);
    CHECK(with([](H& h) { h.momentum = -0.1f; }) == OB_ERR_ARG);
    CHECK(with([&](H& h) { h.momentum = nan; }) == OB_ERR_ARG);
    CHECK(with([](H& h) { h.momentum = 0.0f; }) == OB_OK);
    CHECK(with([](H& h) { h.eps = 0.0f; }) == OB_ERR_ARG);
    CHECK(with([&](H& h) { h.eps = nan; }) == OB_ERR_ARG);
    CHECK(with([](H& h) { h.nesterov = 2; }) == OB_ERR_ARG);
    CHECK(with([](H& h) { h.iterations = 0; }) == OB_ERR_ARG);
    CHECK(with([](H& h) { h.iterations = 17; }) == OB_ERR_ARG);
    CHECK(with([](H& h) { h.scale = 3; }) == OB_ERR_ARG);
    CHECK(with([](H& h) { h.reserved = 1; }) == OB_ERR_ARG);

    // norms and clipping
    const float* norms = reinterpret_cast<float*>(0x6000);
    CHECK(ob::check_tensor_norms(l, g, 1.0f, OB_NORM_2, norms, w) == OB_OK);
    CHECK(ob::check_tensor_norms(l, g, 0.0f, OB_NORM_2, norms, w) == OB_ERR_ARG);
    CHECK(ob::check_tensor_norms(l, g, nan, OB_NORM_2, norms, w) == OB_ERR_ARG);
    CHECK(ob::check_tensor_norms(l, g, 1.0f, 2, norms, w) == OB_ERR_ARG);
    CHECK(ob::check_tensor_norms(l, g, 1.0f, OB_NORM_MAX, nullptr, w) == OB_ERR_ARG);
    CHECK(ob::check_tensor_norms(l, g, 1.0f, OB_NORM_MAX, norms, nullptr) == OB_ERR_ARG);
    CHECK(ob::check_tensor_norms(l, g, 1.0f, OB_NORM_MAX, norms, reinterpret_cast<void*>(0x4004)) == OB_ERR_ALIGN);
    CHECK(ob::check_tensor_norms(l, nullptr, 1.0f, OB_NORM_2, norms, w) == OB_ERR_ARG);
    CHECK(ob::check_clip(l, g, nullptr, norms, 1.0f, 1.0f, 0) == OB_OK);
    CHECK(ob::check_clip(l, g, p, norms, 1.0f, 1.0f, 1) == OB_OK);
    CHECK(ob::check_clip(l, g, p, norms, 1.0f, 1.0f, 2) == OB_ERR_ARG);
    CHECK(ob::check_clip(l, g, p, norms, nan, 1.0f, 0) == OB_ERR_ARG);
    CHECK(ob::check_clip(l, g, p, norms, 1.0f, 0.0f, 0) == OB_ERR_ARG);
    CHECK(ob::check_clip(l, g, p, nullptr, 1.0f, 1.0f, 0) == OB_ERR_ARG);
    CHECK(ob::check_clip(l, g, nop, norms, 1.0f, 1.0f, 0) == OB_ERR_ARG);
    CHECK(ob::check_clip(l, g, odd, norms, 1.0f, 1.0f, 0) == OB_ERR_ALIGN);
    const ob::ListShape two = list_of({{1, 8, 4}, {1, 8, 4}}, {1, 1}, {0, 0});
    const void* gg[2] = {reinterpret_cast<void*>(0x1000), reinterpret_cast<void*>(0x1000)};
    CHECK(ob::check_clip(two, gg, nullptr, norms, 1.0f, 1.0f, 0) == OB_ERR_ARG);   // one gradient twice, in place
    gg[1] = reinterpret_cast<void*>(0x103e);
    CHECK(ob::check_clip(two, gg, nullptr, norms, 1.0f, 1.0f, 0) == OB_ERR_ARG);   // the last element of the first
    gg[1] = reinterpret_cast<void*>(0x1040);
    CHECK(ob::check_clip(two, gg, nullptr, norms, 1.0f, 1.0f, 0) == OB_OK);
    void* pp[2] = {reinterpret_cast<void*>(0x2000), reinterpret_cast<void*>(0x207c)};
    CHECK(ob::check_clip(two, gg, pp, norms, 1.0f, 1.0f, 0) == OB_ERR_ARG);
    pp[1] = reinterpret_cast<void*>(0x2080);
    CHECK(ob::check_clip(two, gg, pp, norms, 1.0f, 1.0f, 0) == OB_OK);
    std::printf("ok %ld\n", checks);
    return 0;
}
