// list_check.cpp -- CPU program: the host side of lists of tensors (ob_lists.h).  Layout, work blocks and
// launch runs of many random lists, each against what the kernels assume, and the refusals of every
// argument check.  Prints "ok <lists>" or the first failure.
#include <cstdio>
#include <cstdlib>
#include <limits>
#include <random>

#include "ob_lists.h"

#define CHECK(x)                                                                  \
    do {                                                                          \
        if (!(x)) {                                                               \
            std::printf("line %d: %s\n", __LINE__, #x);                           \
            return 1;                                                             \
        }                                                                         \
    } while (0)

static int check_list(std::mt19937_64& rng, int T)
{
    std::vector<int64_t> sizes;
    std::vector<int32_t> gd, pd;
    for (int t = 0; t < T; ++t) {
        const int kind = static_cast<int>(rng() % 5);
        sizes.push_back(kind == 0 ? 0 : kind == 1 ? static_cast<int64_t>(rng() % 7) : kind == 2 ? 255 + static_cast<int64_t>(rng() % 3)
                        : kind == 3 ? 4094 + static_cast<int64_t>(rng() % 5) : static_cast<int64_t>(rng() % 100000));
        gd.push_back(static_cast<int32_t>(rng() % 3));
        pd.push_back(static_cast<int32_t>(rng() % 3));
    }
    ob::ListShape l;
    CHECK(ob::build_shape(T, sizes.data(), gd.data(), pd.data(), nullptr, nullptr, l) == OB_OK);
    int64_t off = 0, n = 0;
    for (int t = 0; t < T; ++t) {
        CHECK(l.state_off[t] == off && off % OB_STATE_BLOCK == 0);
        off += (sizes[t] + 255) / 256 * 256;
        n += sizes[t];
    }
    CHECK(l.state_elems == off && l.n == n);
    std::vector<int> seen(T, 0);
    for (int32_t t : l.order) seen[t]++;
    for (int s : seen) CHECK(s == 1);
    for (int64_t elems : {1024, 4096, 16384}) {
        std::vector<ob::ListItem> items;
        std::vector<int64_t> first;
        CHECK(ob::build_items(l, elems, items, first));
        CHECK(first.size() == static_cast<size_t>(T) + 1 && first[T] == static_cast<int64_t>(items.size()));
        for (int k = 0; k < T; ++k) {
            int64_t at = 0;
            for (int64_t b = first[k]; b < first[k + 1]; ++b) {
                const ob::ListItem& it = items[b];
                CHECK(it.tensor == k && it.start == at && it.start % ob::kListTile == 0);
                CHECK(it.len >= 1 && it.len <= elems);
                at += it.len;
                CHECK(b + 1 == first[k + 1] || it.len == elems);
            }
            CHECK(at == sizes[l.order[k]]);
        }
    }
    for (int most : {1, 3, 224}) {
        for (bool par : {false, true}) {
            int64_t next = 0;
            int64_t last = -1;
            CHECK(ob::for_runs(l, most, par, [&](int64_t k, int64_t e) {
                      if (k != next || e <= k || e - k > most) return OB_ERR_ARG;
                      for (int64_t j = k; j < e; ++j) {
                          if (l.g_dtype[l.order[j]] != l.g_dtype[l.order[k]]) return OB_ERR_ARG;
                          if (par && l.p_dtype[l.order[j]] != l.p_dtype[l.order[k]]) return OB_ERR_ARG;
                      }
                      next = e;
                      last = k;
                      return OB_OK;
                  }) == OB_OK);
            CHECK(next == T && last < T);
        }
    }
    for (int64_t n : {int64_t(0), int64_t(1), int64_t(7), int64_t(8), int64_t(100)}) {
        int64_t next = 0;
        CHECK(ob::for_parts(n, 8, [&](int64_t i, int64_t c) {
                  if (i != next || c < 1 || c > 8) return OB_ERR_ARG;
                  next = i + c;
                  return OB_OK;
              }) == OB_OK);
        CHECK(next == n);
        CHECK(n == 0 || ob::for_parts(n, 8, [&](int64_t, int64_t) { return OB_ERR_HIP; }) == OB_ERR_HIP);
    }
    CHECK(ob::kMostGroups * ob::kListBlock < (int64_t(1) << 32));
    return 0;
}

static int check_refusals()
{
    const float nan = std::numeric_limits<float>::quiet_NaN(), inf = std::numeric_limits<float>::infinity();
    int64_t sizes[3] = {5, 0, 300};
    int32_t f32[3] = {OB_F32, OB_F32, OB_F32}, b16[3] = {OB_BF16, OB_BF16, OB_F16}, off[3] = {OB_F32, 3, OB_F32};
    float ones[3] = {1, 1, 1}, bad[3] = {1, nan, 1}, big[3] = {1, 1, inf};
    {
        ob::ListShape l;
        CHECK(ob::build_shape(-1, sizes, f32, f32, nullptr, nullptr, l) == OB_ERR_ARG);
        CHECK(ob::build_shape(3, nullptr, f32, f32, nullptr, nullptr, l) == OB_ERR_ARG);
        CHECK(ob::build_shape(3, sizes, nullptr, f32, nullptr, nullptr, l) == OB_ERR_ARG);
        CHECK(ob::build_shape(3, sizes, f32, nullptr, nullptr, nullptr, l) == OB_ERR_ARG);
        CHECK(ob::build_shape(3, sizes, off, f32, nullptr, nullptr, l) == OB_ERR_DTYPE);
    }
    {
        ob::ListShape l;
        CHECK(ob::build_shape(0, nullptr, nullptr, nullptr, nullptr, nullptr, l) == OB_OK && l.n == 0);
    }
    for (const auto& mults : {std::pair<float*, float*>{bad, ones}, {ones, big}}) {
        ob::ListShape l;
        CHECK(ob::build_shape(3, sizes, f32, f32, mults.first, mults.second, l) == OB_ERR_ARG);
    }
    {
        ob::ListShape l;
        int64_t neg[1] = {-1};
        CHECK(ob::build_shape(1, neg, f32, f32, nullptr, nullptr, l) == OB_ERR_ARG);
    }
    {
        ob::ListShape l;
        int64_t huge[2] = {ob::kListMost, 1};
        CHECK(ob::build_shape(2, huge, f32, f32, nullptr, nullptr, l) == OB_ERR_ARG);
    }
    {   // 2^43 elements: 2^31 blocks of 4096
        ob::ListShape l;
        int64_t huge[1] = {int64_t(1) << 43};
        std::vector<ob::ListItem> items;
        std::vector<int64_t> first;
        CHECK(ob::build_shape(1, huge, f32, f32, nullptr, nullptr, l) == OB_OK);
        CHECK(!ob::build_items(l, 4096, items, first) && items.empty());
    }
    ob::ListShape l;
    CHECK(ob::build_shape(3, sizes, b16, f32, ones, ones, l) == OB_OK);
    auto at = [](uintptr_t a) { return reinterpret_cast<void*>(a); };
    const void* g[3] = {at(0x1002), nullptr, at(0x2000)};
    void* p[3] = {at(0x10004), nullptr, at(0x20000)};
    ob_adamw_hparams hp = {1e-3f, 0.9f, 0.999f, 1e-8f, 0.01f, 1, 1, OB_ROUND_NEAREST, 0, 0};
    const ob_control* ctl = static_cast<const ob_control*>(at(0x30000));
    CHECK(ob::check_step(l, g, p, nullptr, false, &hp, nullptr) == OB_OK);
    CHECK(ob::check_step(l, g, p, nullptr, true, &hp, ctl) == OB_OK);
    CHECK(ob::check_step(l, g, p, nullptr, false, nullptr, nullptr) == OB_ERR_ARG);
    CHECK(ob::check_step(l, nullptr, p, nullptr, false, &hp, nullptr) == OB_ERR_ARG);
    CHECK(ob::check_step(l, g, nullptr, nullptr, false, &hp, nullptr) == OB_ERR_ARG);
    CHECK(ob::check_step(l, g, p, static_cast<float*>(at(0x1004)), false, &hp, nullptr) == OB_ERR_ALIGN);
    CHECK(ob::check_step(l, g, p, nullptr, false, &hp, static_cast<const ob_control*>(at(0x30004))) == OB_ERR_ALIGN);
    {
        const void* g2[3] = {at(0x1001), nullptr, at(0x2000)};
        CHECK(ob::check_step(l, g2, p, nullptr, false, &hp, nullptr) == OB_ERR_ALIGN);
        void* p2[3] = {at(0x10002), nullptr, at(0x20000)};
        CHECK(ob::check_step(l, g, p2, nullptr, false, &hp, nullptr) == OB_ERR_ALIGN);
        void* p3[3] = {at(0x10004), nullptr, nullptr};
        CHECK(ob::check_step(l, g, p3, nullptr, false, &hp, nullptr) == OB_ERR_ARG);
        const void* none[3] = {at(0x1002), nullptr, nullptr};   // no gradient: no parameter needed
        CHECK(ob::check_step(l, none, p3, nullptr, false, &hp, nullptr) == OB_OK);
        void* same[3] = {at(0x20000), nullptr, at(0x20000)};
        CHECK(ob::check_step(l, g, same, nullptr, false, &hp, nullptr) == OB_ERR_ARG);
        CHECK(ob::check_step(l, none, same, nullptr, false, &hp, nullptr) == OB_OK);
        void* into[3] = {at(0x20000 + 299 * 4), nullptr, at(0x20000)};   // descending, the last element shared
        CHECK(ob::check_step(l, g, into, nullptr, false, &hp, nullptr) == OB_ERR_ARG);
        void* next[3] = {at(0x20000 + 300 * 4), nullptr, at(0x20000)};
        CHECK(ob::check_step(l, g, next, nullptr, false, &hp, nullptr) == OB_OK);
    }
    auto refused = [&](auto&& change, bool eight = false, bool control = false) {
        ob_adamw_hparams h = hp;
        change(h);
        return ob::check_hparams(&h, eight, control) == OB_ERR_ARG;
    };
    for (float x : {1.0f, -0.1f, nan, inf}) {
        CHECK(refused([&](auto& h) { h.beta1 = x; }));
        CHECK(refused([&](auto& h) { h.beta2 = x; }));
    }
    for (float x : {nan, inf, -inf}) {
        CHECK(refused([&](auto& h) { h.lr = x; }));
        CHECK(refused([&](auto& h) { h.weight_decay = x; }));
        CHECK(refused([&](auto& h) { h.eps = x; }));
    }
    CHECK(refused([&](auto& h) { h.eps = -1e-8f; }));
    CHECK(!refused([&](auto& h) { h.eps = 0.0f; }) && refused([&](auto& h) { h.eps = 0.0f; }, true));
    CHECK(refused([&](auto& h) { h.eps = 1e-39f; }, true));
    CHECK(refused([&](auto& h) { h.rounding = 2; }));
    CHECK(refused([&](auto& h) { h.step = 0; }) && !refused([&](auto& h) { h.step = 0; }, false, true));
    CHECK(!refused([&](auto& h) { h.step = 0; h.bias_correction = 0; }));

    ob_control* c = static_cast<ob_control*>(at(0x30000));
    CHECK(ob::check_norm(l, g, 1.0f, 1.0f, nullptr, c) == OB_OK && ob::check_norm(l, g, -2.0f, inf, &hp, c) == OB_OK);
    CHECK(ob::check_norm(l, g, 1.0f, 1.0f, nullptr, nullptr) == OB_ERR_ARG);
    CHECK(ob::check_norm(l, nullptr, 1.0f, 1.0f, nullptr, c) == OB_ERR_ARG);
    for (float x : {0.0f, nan, inf}) CHECK(ob::check_norm(l, g, x, 1.0f, nullptr, c) == OB_ERR_ARG);
    CHECK(ob::check_norm(l, g, 1.0f, nan, nullptr, c) == OB_ERR_ARG);
    CHECK(ob::check_norm(l, g, 1.0f, 1.0f, nullptr, static_cast<ob_control*>(at(0x30004))) == OB_ERR_ALIGN);

    const float* f = static_cast<const float*>(at(0x1000));
    CHECK(ob::check_state8(-1, f, f, f, f, f, f) == OB_ERR_ARG);
    CHECK(ob::check_state8(ob::kListMost + 1, f, f, f, f, f, f) == OB_ERR_ARG);
    CHECK(ob::check_state8(0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr) == OB_OK);
    CHECK(ob::check_state8(9, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr) == OB_ERR_ARG);
    CHECK(ob::check_state8(9, f, nullptr, f, f, nullptr, nullptr) == OB_OK);
    CHECK(ob::check_state8(9, nullptr, f, nullptr, nullptr, f, f) == OB_OK);
    CHECK(ob::check_state8(9, f, nullptr, f, nullptr, nullptr, nullptr) == OB_ERR_ARG);
    CHECK(ob::check_state8(9, f, f, f, f, nullptr, f) == OB_ERR_ARG);
    CHECK(ob::check_state8(9, static_cast<const float*>(at(0x1004)), nullptr, f, f, nullptr, nullptr) == OB_ERR_ALIGN);
    CHECK(ob::check_state8(9, f, nullptr, at(0x1002), f, nullptr, nullptr) == OB_ERR_ALIGN);
    CHECK(ob::check_state8(9, f, nullptr, f, static_cast<const float*>(at(0x1002)), nullptr, nullptr) == OB_ERR_ALIGN);
    return 0;
}

int main()
{
    std::mt19937_64 rng(7);
    int lists = 0;
    for (int T : {0, 1, 2, 3, 10, 100, 500})
        for (int r = 0; r < 20; ++r, ++lists)
            if (check_list(rng, T)) return 1;
    if (check_refusals()) return 1;
    std::printf("ok %d\n", lists);
    return 0;
}
