// ob_clip_api.cpp -- host side of norms and clipping over lists of tensors (declarations and contracts in ob_adam.h).
#include "ob_adam.h"
#include "ob_clip.h"
#include "ob_list_handle.h"

static_assert(OB_F32 == 0 && OB_BF16 == 1 && OB_F16 == 2, "kernels are chosen by these numbers");
static_assert(ob::kShortElems <= ob::kNormElems, "a tensor of a short list is one item");

extern "C" {

int64_t ob_tensor_norms_workspace(ob_tensors list)
{
    if (!list) return -1;
    return 8 * (list->norm.first.back() + static_cast<int64_t>(list->shape.size.size()));
}

ob_status ob_tensor_norms(ob_tensors list, const void* const* g, float g_mult, int32_t kind, float* norms, void* workspace,
                          hipStream_t stream)
try {
    if (!list) return OB_ERR_ARG;
    const ob_tensors_s& l = *list;
    if (ob_status st = ob::check_tensor_norms(l.shape, g, g_mult, kind, norms, workspace)) return st;
    ob::DeviceGuard guard(l.device);
    if (!guard.ok) return OB_ERR_HIP;
    int64_t left = 0;
    for (size_t t = 0; t < l.shape.size.size(); ++t) left += l.shape.size[t] * ob::dtype_bytes(l.shape.g_dtype[t]);
    const ob::NormTables tables{l.d_norm_first, l.d_order, static_cast<int64_t>(l.shape.size.size()), l.norm.first.back(),
                                static_cast<double*>(workspace)};
    ob::NormPtrs ptrs;
    bool brief = tables.tensors > 0 && tables.tensors <= ob::kShortTensors;
    int64_t total = 0;
    for (size_t t = 0; brief && t < l.shape.size.size(); ++t) {
        total += l.shape.size[t];
        brief = l.shape.size[t] <= ob::kShortElems && total <= ob::kShortTotal && l.shape.g_dtype[t] == l.shape.g_dtype[0];
    }
    if (brief) {
        for (int64_t k = 0; k < tables.tensors; ++k) {
            const int32_t t = l.shape.order[k];
            ptrs.g[k] = l.shape.size[t] > 0 ? g[t] : nullptr;
        }
        const ob::ListLaunch L{l.norm.d_items, l.d_tensors, tables.items, 0};
        (void)hipGetLastError();
        return ob::launch_short_norms(L, ptrs, l.shape.g_dtype[0], kind, tables, g_mult, norms, stream) == hipSuccess ? OB_OK : OB_ERR_HIP;
    }
    const ob_status st = ob::for_runs(l.shape, ob::kNormPtrs, false, [&](int64_t k, int64_t e) {
        const int gd = l.shape.g_dtype[l.shape.order[k]];
        const int64_t items = l.norm.first[e] - l.norm.first[k], bytes = ob::kNormElems * ob::dtype_bytes(gd);
        if (items > 0)
            for (int64_t j = k; j < e; ++j) ptrs.g[j - k] = g[l.shape.order[j]];
        return ob::for_parts(items, ob::kMostGroups, [&](int64_t i, int64_t n) {
            const int64_t at = l.norm.first[k] + i;
            const ob::ListLaunch L{l.norm.d_items + at, l.d_tensors, n, static_cast<int32_t>(k)};
            const int64_t nt = std::max<int64_t>(0, (left - ob::kKeepBytes) / bytes);   // items before the last kKeepBytes of the call
            left -= n * bytes;
            (void)hipGetLastError();  // clear a stale error so the check sees this launch only
            return ob::launch_item_norms(L, ptrs, gd, kind, nt, tables.partials + at, stream) == hipSuccess ? OB_OK : OB_ERR_HIP;
        });
    });
    if (st != OB_OK) return st;
    (void)hipGetLastError();
    return ob::launch_tensor_norms(tables, kind, g_mult, norms, stream) == hipSuccess ? OB_OK : OB_ERR_HIP;
} catch (...) {
    return OB_ERR_OOM;
}

ob_status ob_clip_grads(ob_tensors list, const void* const* g, void* const* out, const float* norms, float max_norm,
                        float g_mult, int32_t per_tensor, hipStream_t stream)
try {
    if (!list) return OB_ERR_ARG;
    const ob_tensors_s& l = *list;
    const ob::ListShape& sh = l.shape;
    if (ob_status st = ob::check_clip(sh, g, out, norms, max_norm, g_mult, per_tensor)) return st;
    if (sh.n == 0) return OB_OK;
    ob::DeviceGuard guard(l.device);
    if (!guard.ok) return OB_ERR_HIP;
    const ob::ClipParams cp{g_mult, max_norm, max_norm > 0.0f && !std::isinf(max_norm), norms, per_tensor ? l.d_order : nullptr,
                            static_cast<int64_t>(sh.size.size())};
    // the runs from the last one on, as their items
    struct Run {
        int64_t k, e;
    };
    std::vector<Run> runs;
    (void)ob::for_runs(sh, ob::kListPtrs, out != nullptr, [&](int64_t k, int64_t e) {
        runs.push_back({k, e});
        return OB_OK;
    });
    ob::ListPtrs ptrs;
    for (size_t r = runs.size(); r-- > 0;) {
        const int64_t k = runs[r].k, e = runs[r].e;
        for (int64_t j = k; j < e; ++j) {
            ptrs.g[j - k] = g[sh.order[j]];
            ptrs.p[j - k] = out ? out[sh.order[j]] : const_cast<void*>(g[sh.order[j]]);
        }
        const int gd = sh.g_dtype[sh.order[k]], od = out ? sh.p_dtype[sh.order[k]] : gd;
        const ob_status st = ob::for_parts(l.step.first[e] - l.step.first[k], ob::kMostGroups, [&](int64_t i, int64_t n) {
            const ob::ListLaunch L{l.step.d_items + l.step.first[k] + i, l.d_tensors, n, static_cast<int32_t>(k)};
            (void)hipGetLastError();
            return ob::launch_clip(L, ptrs, gd, od, cp, stream) == hipSuccess ? OB_OK : OB_ERR_HIP;
        });
        if (st != OB_OK) return st;
    }
    return OB_OK;
} catch (...) {
    return OB_ERR_OOM;
}

}  // extern "C"
