// ob_adamw.h -- shared between the host side (ob_adamw_api.cpp) and the kernels (ob_adamw.hip,
// ob_state8.hip) of the steps over lists of tensors.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ob_lists.h"

namespace ob {

struct ListTensor {
    int64_t state_off;
    float lr_mult, wd_mult;
};

// A launch's tensor addresses travel in its arguments, so that no table is copied per call and a
// captured launch keeps its own.  224 pairs are 3.5 KB of the 4 KB that a launch's arguments may take.
constexpr int kListPtrs = 224;
struct ListPtrs {
    const void* g[kListPtrs];
    void* p[kListPtrs];
};
// The norm takes gradients only.
constexpr int kNormPtrs = 2 * kListPtrs;
struct NormPtrs {
    const void* g[kNormPtrs];
};

// How a tensor's parameters are held.
enum { PK_F32 = 0, PK_BF16 = 1, PK_F16 = 2, PK_MASTER_BF16 = 3, PK_MASTER_F16 = 4 };

struct ListLaunch {
    const ListItem* items;       // of this launch
    const ListTensor* tensors;   // of the whole list
    int64_t n_items;
    int32_t tensor0;             // place of the launch's first tensor: its addresses are ptrs.g[0], ptrs.p[0]
};

struct AdamWParams {
    double lr, beta1, one_m_beta1, beta2, one_m_beta2, eps, wd, bc1, bc2;
    float root_factor;           // bc1 / sqrt(bc2)
    int bias_correction;
    int stochastic;
    uint64_t seed, step;
    const ob_control* control;   // NULL: the corrections and the step above
};

struct State32 {
    float* master;
    float* m;
    float* v;
};
struct State8 {
    float* master;
    int8_t* mc;
    float* mq;
    uint8_t* vc;
    float* vq;
};

// One launcher per gradient type G (ob_dtype); pk: parameter kind.
template <int G>
hipError_t launch_adamw(const ListLaunch& L, const ListPtrs& ptrs, int pk, const State32& st, const AdamWParams& ap,
                        hipStream_t s);
template <int G>
hipError_t launch_adamw8(const ListLaunch& L, const ListPtrs& ptrs, int pk, const State8& st, const AdamWParams& ap,
                         hipStream_t s);

struct NormParams {
    double g_mult, max_norm, beta1, beta2;
    int clip, advance;   // clip to max_norm; count the step
    int first;           // the call's first launch: partial sums are written, else added to
    int ticket;          // this launch finishes the norm
};
// Sums of squares of the launch's gradients into the control block's partial sums [0, grid).  Items below
// nt_items are read nontemporally.
hipError_t launch_grad_sumsq(const ListLaunch& L, const NormPtrs& ptrs, int g_dtype, int grid, int64_t nt_items,
                             ob_control* ctl, const NormParams& np, hipStream_t s);
// The control block from them, after the last launch of a call.
hipError_t launch_grad_control(ob_control* ctl, int grid, const NormParams& np, hipStream_t s);

hipError_t launch_state8_encode(int64_t n, const float* m, const float* v, int8_t* mc, float* mq, uint8_t* vc,
                                float* vq, hipStream_t s);
hipError_t launch_state8_decode(int64_t n, const int8_t* mc, const float* mq, const uint8_t* vc, const float* vq,
                                float* m, float* v, hipStream_t s);

}  // namespace ob
