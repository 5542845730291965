// ob_clip.h -- shared between the host side (ob_clip_api.cpp) and the kernels (ob_clip.hip) of norms and clipping.
#pragma once

#include "ob_adamw.h"

namespace ob {

// The workspace: a partial result for each item of the list, in its order, then one for each tensor, by place.
struct NormTables {
    const int64_t* first;    // by place
    const int32_t* order;
    int64_t tensors, items;
    double* partials;        // [items], then [tensors]
};

// Partial results of the launch's items into partials[0 ...]; items below nt_items are read nontemporally.
hipError_t launch_item_norms(const ListLaunch& L, const NormPtrs& ptrs, int g_dtype, int kind, int64_t nt_items, double* partials,
                             hipStream_t s);
// The norms of a short list in one launch and one work group: at most kShortTensors tensors of one gradient type, of kShortElems
// elements each and kShortTotal together.  One launch against two, us (bf16): 12 x 1,024 3.7 and 5.9, 12 x 4,096 4.8 and 5.9,
// 32 x 1,024 5.8 and 6.6; beyond, one work group reads and walks too slowly: 32 x 4,096 8.2 and 6.6, 64 x 64 10.0 and 7.2,
// 64 x 8,192 22.7 and 7.8.  fp32 gives the same sides.
constexpr int64_t kShortTensors = 32, kShortElems = 4096, kShortTotal = 48 * 1024;
static_assert(kShortTensors <= kNormPtrs);
hipError_t launch_short_norms(const ListLaunch& L, const NormPtrs& ptrs, int g_dtype, int kind, const NormTables& t, double g_mult,
                              float* norms, hipStream_t s);
// norms from the partial results of all items.
hipError_t launch_tensor_norms(const NormTables& t, int kind, double g_mult, float* norms, hipStream_t s);

struct ClipParams {
    double g_mult, max_norm;
    int clip;               // to max_norm
    const float* norms;
    const int32_t* order;   // per tensor: norms[order[place]]; NULL: norms[total]
    int64_t total;
};
// g_dtype, out_dtype: of the launch's tensors.
hipError_t launch_clip(const ListLaunch& L, const ListPtrs& ptrs, int g_dtype, int out_dtype, const ClipParams& cp, hipStream_t s);

}  // namespace ob
