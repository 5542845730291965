// ob_lists.h -- lists of tensors on the host, in plain C++17: their layout, work blocks and launches, and
// the checks of a call's arguments.  Used by the host side (ob_adamw_api.cpp) and checked on the CPU by
// tests/list_check.cpp.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <numeric>
#include <vector>

#include "ob_adam.h"

namespace ob {

// Work blocks of a list: 256 threads = four waves, a wave's tile being one state block of 256
// consecutive elements (four per lane), a block's tile four of them.
constexpr int kListBlock = 256;
constexpr int kListTile = 1024;
constexpr int kStepTiles = 4;   // tiles per item of the steps
constexpr int kStateBlock = OB_STATE_BLOCK;

// One work block: elements [start, start + len) of the tensor in place `tensor` of the list's order.
// start is a multiple of kListTile.
struct ListItem {
    int64_t start;
    int32_t len;
    int32_t tensor;
};

inline bool is_aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool list_dtype(int32_t d) { return d == OB_F32 || d == OB_BF16 || d == OB_F16; }
inline int64_t dtype_bytes(int32_t d) { return d == OB_F32 ? 4 : 2; }

// The list's tensors stand in an order of their own, by types, so that a launch meets one pair of types.
struct ListShape {
    int64_t n = 0, state_elems = 0;
    std::vector<int64_t> size, state_off;    // by tensor
    std::vector<int32_t> g_dtype, p_dtype;   // by tensor
    std::vector<int32_t> order;              // place -> tensor
};

// Most elements of a list: byte offsets into its fp32 states stay far below 2^63.
constexpr int64_t kListMost = int64_t(1) << 44;

inline ob_status build_shape(int64_t T, const int64_t* sizes, const int32_t* gd, const int32_t* pd, const float* lr,
                             const float* wd, ListShape& l)
{
    if (T < 0 || T > INT32_MAX) return OB_ERR_ARG;
    if (T > 0 && (!sizes || !gd || !pd)) return OB_ERR_ARG;
    for (int64_t t = 0; t < T; ++t) {
        if (!list_dtype(gd[t]) || !list_dtype(pd[t])) return OB_ERR_DTYPE;
        if (sizes[t] < 0 || sizes[t] > kListMost - l.state_elems) return OB_ERR_ARG;
        if ((lr && !std::isfinite(lr[t])) || (wd && !std::isfinite(wd[t]))) return OB_ERR_ARG;
        l.size.push_back(sizes[t]);
        l.g_dtype.push_back(gd[t]);
        l.p_dtype.push_back(pd[t]);
        l.state_off.push_back(l.state_elems);
        l.state_elems += (sizes[t] + kStateBlock - 1) / kStateBlock * kStateBlock;
        l.n += sizes[t];
    }
    l.order.resize(static_cast<size_t>(T));
    std::iota(l.order.begin(), l.order.end(), 0);
    std::stable_sort(l.order.begin(), l.order.end(), [&](int32_t a, int32_t b) {
        return gd[a] != gd[b] ? gd[a] < gd[b] : pd[a] < pd[b];
    });
    return OB_OK;
}

// The work blocks of `elems` elements (a multiple of kListTile), in the list's order; first[k]: index of
// the first block of the tensor in place k, first[T] the count.  False if the blocks would pass 2^31 - 1.
inline bool build_items(const ListShape& l, int64_t elems, std::vector<ListItem>& items, std::vector<int64_t>& first)
{
    int64_t total = 0;
    for (int64_t n : l.size) {
        total += n / elems + (n % elems != 0);
        if (total > INT32_MAX) return false;
    }
    items.reserve(static_cast<size_t>(total));
    for (size_t k = 0; k < l.order.size(); ++k) {
        first.push_back(static_cast<int64_t>(items.size()));
        const int64_t n = l.size[l.order[k]];
        for (int64_t s = 0; s < n; s += elems)
            items.push_back({s, static_cast<int32_t>(std::min(elems, n - s)), static_cast<int32_t>(k)});
    }
    first.push_back(static_cast<int64_t>(items.size()));
    return true;
}

// The launches of a call: f(k, e) for runs of places [k, e) of one gradient type (and one parameter type,
// with `parameters`), at most `most` tensors each, until f returns other than OB_OK.
template <class F>
ob_status for_runs(const ListShape& l, int64_t most, bool parameters, F&& f)
{
    const int64_t T = static_cast<int64_t>(l.order.size());
    for (int64_t k = 0; k < T;) {
        const int32_t a = l.order[k];
        int64_t e = k + 1;
        for (; e < T && e - k < most; ++e) {
            const int32_t b = l.order[e];
            if (l.g_dtype[b] != l.g_dtype[a] || (parameters && l.p_dtype[b] != l.p_dtype[a])) break;
        }
        if (ob_status st = f(k, e)) return st;
        k = e;
    }
    return OB_OK;
}

// A launch has at most 2^32 - 1 threads, so what needs more work groups of kListBlock is launched in parts:
// f(begin, count) over 0..n in parts of at most `most`, until f returns other than OB_OK.
constexpr int64_t kMostGroups = (int64_t(1) << 32) / kListBlock - 1;

template <class F>
ob_status for_parts(int64_t n, int64_t most, F&& f)
{
    for (int64_t i = 0; i < n; i += most)
        if (ob_status st = f(i, std::min(most, n - i))) return st;
    return OB_OK;
}

inline ob_status check_hparams(const ob_adamw_hparams* hp, bool eight, bool has_control)
{
    if (!hp) return OB_ERR_ARG;
    if (!(hp->beta1 >= 0.0f && hp->beta1 < 1.0f) || !(hp->beta2 >= 0.0f && hp->beta2 < 1.0f)) return OB_ERR_ARG;
    if (!std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay)) return OB_ERR_ARG;
    if (!std::isfinite(hp->eps) || hp->eps < 0.0f || (eight && hp->eps < 1e-30f)) return OB_ERR_ARG;
    if (hp->rounding != OB_ROUND_NEAREST && hp->rounding != OB_ROUND_STOCHASTIC) return OB_ERR_ARG;
    if (!has_control && hp->bias_correction && hp->step < 1) return OB_ERR_ARG;
    return OB_OK;
}

// Addresses of one call (p == NULL: gradients only): none missing, aligned to their elements, parameters
// apart from each other.
inline ob_status check_pointers(const ListShape& l, const void* const* g, void* const* p)
{
    if (l.n == 0) return OB_OK;
    if (!g) return OB_ERR_ARG;
    const size_t T = l.size.size();
    for (size_t t = 0; t < T; ++t) {
        if (l.size[t] == 0 || !g[t]) continue;
        if (!is_aligned(g[t], dtype_bytes(l.g_dtype[t]))) return OB_ERR_ALIGN;
        if (!p) continue;
        if (!p[t]) return OB_ERR_ARG;
        if (!is_aligned(p[t], dtype_bytes(l.p_dtype[t]))) return OB_ERR_ALIGN;
    }
    if (!p) return OB_OK;
    // ascending addresses, as of views into one buffer, need one look; others are sorted
    struct Range {
        uintptr_t a, b;
    };
    std::vector<Range> r;
    r.reserve(T);
    bool sorted = true;
    for (size_t t = 0; t < T; ++t) {
        if (l.size[t] == 0 || !g[t]) continue;
        const uintptr_t a = reinterpret_cast<uintptr_t>(p[t]);
        if (!r.empty() && a < r.back().a) sorted = false;
        r.push_back({a, a + static_cast<uintptr_t>(l.size[t] * dtype_bytes(l.p_dtype[t]))});
    }
    if (!sorted) std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.a < y.a; });
    for (size_t k = 1; k < r.size(); ++k)
        if (r[k].a < r[k - 1].b) return OB_ERR_ARG;
    return OB_OK;
}

// Arguments of a step but for its states.
inline ob_status check_step(const ListShape& l, const void* const* g, void* const* p, const float* master, bool eight,
                            const ob_adamw_hparams* hp, const ob_control* control)
{
    if (ob_status st = check_hparams(hp, eight, control != nullptr)) return st;
    if (control && !is_aligned(control, 8)) return OB_ERR_ALIGN;
    if (l.n == 0) return OB_OK;
    if (!p) return OB_ERR_ARG;
    if (!is_aligned(master, 16)) return OB_ERR_ALIGN;
    return check_pointers(l, g, p);
}

inline ob_status check_norm(const ListShape& l, const void* const* g, float g_mult, float max_norm,
                            const ob_adamw_hparams* hp, const ob_control* control)
{
    if (!control) return OB_ERR_ARG;
    if (!std::isfinite(g_mult) || g_mult == 0.0f || std::isnan(max_norm)) return OB_ERR_ARG;
    if (hp)
        if (ob_status st = check_hparams(hp, false, true)) return st;
    if (!is_aligned(control, 8)) return OB_ERR_ALIGN;
    return check_pointers(l, g, nullptr);
}

inline ob_status check_state8(int64_t n, const float* m, const float* v, const void* mc, const float* mq,
                              const void* vc, const float* vq)
{
    if (n < 0 || n > kListMost) return OB_ERR_ARG;
    if (n == 0) return OB_OK;
    const bool any_m = m || mc || mq, any_v = v || vc || vq;
    if ((any_m && !(m && mc && mq)) || (any_v && !(v && vc && vq)) || (!any_m && !any_v)) return OB_ERR_ARG;
    for (const void* x : {static_cast<const void*>(m), static_cast<const void*>(v)})
        if (!is_aligned(x, 16)) return OB_ERR_ALIGN;
    for (const void* x : {mc, vc, static_cast<const void*>(mq), static_cast<const void*>(vq)})
        if (!is_aligned(x, 4)) return OB_ERR_ALIGN;
    return OB_OK;
}

}  // namespace ob
