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
