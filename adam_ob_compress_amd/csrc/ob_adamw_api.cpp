// ob_adamw_api.cpp -- host side of the calls over lists of tensors (declarations and contracts in
// ob_adam.h): checks of arguments, the list's work-block tables, and the launches.
#include "ob_adam.h"
#include "ob_adamw.h"

#include <algorithm>
#include <cstddef>
#include <vector>

static_assert(sizeof(ob_control) == 64 && offsetof(ob_control, bc1) == 24 && offsetof(ob_control, skip) == 44,
              "the control block's layout is part of the ABI");

namespace {

struct Table {
    std::vector<int64_t> first;      // [T + 1]: items of the tensor in place k are [first[k], first[k+1])
    const ob::ListItem* d_items = nullptr;
};

}  // namespace

struct ob_tensors_s {
    int device = 0;
    ob::ListShape shape;
    Table step, norm;
    const ob::ListTensor* d_tensors = nullptr;  // by place
    void* d_tables = nullptr;                   // one allocation: the items of both tables, the tensors
};

namespace {

// Elements per item of the steps and of the norm.
constexpr int64_t kStepElems = ob::kStepTiles * ob::kListTile;
constexpr int64_t kNormElems = 16 * ob::kListTile;
// Gradient bytes at a call's end that the norm reads with ordinary loads, which leave them in the last-level
// cache for the step that follows; what comes before is read nontemporally, which is faster.  Norm and step
// of 1.09e8 elements: bf16 278 us with ordinary loads and 293 nontemporal, fp32 (436 MB) 554 and 592; norm alone
// of 3.1 GB: 513 and 452.
constexpr int64_t kKeepBytes = int64_t(256) << 20;
// Up to this many blocks the last one finishes the norm, beyond it another launch does.  12 tensors of 20,000
// elements in all: 5.4 us and 6.2 (6.0 and 9.6 with the call); 200 of 1e7 (610 blocks): 19 us and 9, as each
// block's ticket makes its memory visible to the others.
constexpr int kTicketGrid = 128;
static_assert(kTicketGrid <= ob::kListBlock, "the last block reads one partial sum per thread");

// Elements of one launch of a conversion (4096 per work group).
constexpr int64_t kState8Part = ob::kMostGroups * 4096;

template <class T>
T* at(T* p, int64_t i)
{
    return p ? p + i : nullptr;
}

// The list's device is current for the duration of a call.
struct DeviceGuard {
    int back = -1;   // the device to return to; -1: none was left
    bool ok;
    explicit DeviceGuard(int dev)
    {
        int cur = -1;
        ok = hipGetDevice(&cur) == hipSuccess;
        if (ok && cur != dev) {
            ok = hipSetDevice(dev) == hipSuccess;
            back = cur;
        }
    }
    ~DeviceGuard()
    {
        if (back >= 0) (void)hipSetDevice(back);
    }
};

void free_list(ob_tensors l)
{
    if (!l) return;
    if (l->d_tables) (void)hipFree(l->d_tables);
    delete l;
}

ob_status list_create(int64_t T, const int64_t* sizes, const int32_t* gd, const int32_t* pd, const float* lr,
                      const float* wd, ob_tensors* out, ob_tensors& l)
{
    if (!out) return OB_ERR_ARG;
    *out = nullptr;
    l = new ob_tensors_s;
    if (ob_status st = ob::build_shape(T, sizes, gd, pd, lr, wd, l->shape)) return st;
    std::vector<ob::ListItem> step, norm;
    if (!ob::build_items(l->shape, kStepElems, step, l->step.first) ||
        !ob::build_items(l->shape, kNormElems, norm, l->norm.first))
        return OB_ERR_ARG;
    std::vector<ob::ListTensor> tensors;
    for (int32_t t : l->shape.order) tensors.push_back({l->shape.state_off[t], lr ? lr[t] : 1.0f, wd ? wd[t] : 1.0f});

    if (hipGetDevice(&l->device) != hipSuccess) return OB_ERR_HIP;
    const size_t a = step.size() * sizeof(ob::ListItem), b = norm.size() * sizeof(ob::ListItem);
    const size_t bytes = a + b + tensors.size() * sizeof(ob::ListTensor);
    if (bytes > 0) {
        std::vector<char> tables(bytes);
        std::copy_n(reinterpret_cast<const char*>(step.data()), a, tables.data());
        std::copy_n(reinterpret_cast<const char*>(norm.data()), b, tables.data() + a);
        std::copy_n(reinterpret_cast<const char*>(tensors.data()), bytes - a - b, tables.data() + a + b);
        hipError_t e = hipMalloc(&l->d_tables, bytes);
        if (e == hipSuccess) e = hipMemcpy(l->d_tables, tables.data(), bytes, hipMemcpyHostToDevice);
        // a first call may be on a stream that does not wait for the null stream
        if (e == hipSuccess) e = hipStreamSynchronize(nullptr);
        if (e != hipSuccess) return e == hipErrorOutOfMemory ? OB_ERR_OOM : OB_ERR_HIP;
        const char* d = static_cast<const char*>(l->d_tables);
        l->step.d_items = reinterpret_cast<const ob::ListItem*>(d);
        l->norm.d_items = reinterpret_cast<const ob::ListItem*>(d + a);
        l->d_tensors = reinterpret_cast<const ob::ListTensor*>(d + a + b);
    }
    *out = l;
    return OB_OK;
}

ob::AdamWParams adamw_params(const ob_adamw_hparams* hp, const ob_control* control)
{
    ob::AdamWParams ap;
    ap.lr = hp->lr;
    ap.beta1 = hp->beta1;
    ap.one_m_beta1 = 1.0 - static_cast<double>(hp->beta1);
    ap.beta2 = hp->beta2;
    ap.one_m_beta2 = 1.0 - static_cast<double>(hp->beta2);
    ap.eps = hp->eps;
    ap.wd = hp->weight_decay;
    ap.bias_correction = hp->bias_correction ? 1 : 0;
    ap.stochastic = hp->rounding == OB_ROUND_STOCHASTIC;
    ap.bc1 = ap.bc2 = 1.0;
    if (ap.bias_correction && !control) {
        ap.bc1 = 1.0 - std::pow(ap.beta1, static_cast<double>(hp->step));
        ap.bc2 = 1.0 - std::pow(ap.beta2, static_cast<double>(hp->step));
    }
    ap.root_factor = static_cast<float>(ap.bc1 / std::sqrt(ap.bc2));
    ap.seed = hp->sr_seed;
    ap.step = static_cast<uint64_t>(hp->step);
    ap.control = control;
    return ap;
}

// The launches of a step: f(gradient type, parameter kind, launch, addresses) for each.
template <class F>
ob_status launch_step(const ob_tensors_s& l, const void* const* g, void* const* p, bool master, F&& f)
{
    const ob::ListShape& sh = l.shape;
    ob::ListPtrs ptrs;
    return ob::for_runs(sh, ob::kListPtrs, true, [&](int64_t k, int64_t e) {
        for (int64_t j = k; j < e; ++j) {
            ptrs.g[j - k] = g[sh.order[j]];
            ptrs.p[j - k] = p[sh.order[j]];
        }
        const int gd = sh.g_dtype[sh.order[k]], pd = sh.p_dtype[sh.order[k]];
        const int pk = pd == OB_F32 ? ob::PK_F32 : pd + (master ? 2 : 0);
        return ob::for_parts(l.step.first[e] - l.step.first[k], ob::kMostGroups / ob::kStepTiles, [&](int64_t i, int64_t n) {
            const ob::ListLaunch L{l.step.d_items + l.step.first[k] + i, l.d_tensors, n, static_cast<int32_t>(k)};
            (void)hipGetLastError();  // clear a stale error so the check sees this launch only
            return f(gd, pk, L, ptrs) == hipSuccess ? OB_OK : OB_ERR_HIP;
        });
    });
}

}  // namespace

extern "C" {

ob_status ob_tensors_create(int64_t n_tensors, const int64_t* sizes, const int32_t* g_dtypes, const int32_t* p_dtypes,
                            const float* lr_mults, const float* wd_mults, ob_tensors* out)
{
    ob_tensors l = nullptr;
    ob_status st;
    try {
        st = list_create(n_tensors, sizes, g_dtypes, p_dtypes, lr_mults, wd_mults, out, l);
    } catch (...) {
        st = OB_ERR_OOM;  // host allocation failures are the only exceptions here
    }
    if (st != OB_OK) free_list(l);
    return st;
}

ob_status ob_tensors_destroy(ob_tensors list)
try {
    if (!list) return OB_ERR_ARG;
    DeviceGuard guard(list->device);
    free_list(list);
    return OB_OK;
} catch (...) {
    return OB_ERR_OOM;
}

int64_t ob_tensors_count(ob_tensors list) { return list ? static_cast<int64_t>(list->shape.size.size()) : -1; }
int64_t ob_tensors_num_elements(ob_tensors list) { return list ? list->shape.n : -1; }
int64_t ob_tensors_state_elems(ob_tensors list) { return list ? list->shape.state_elems : -1; }
int64_t ob_tensors_state_offset(ob_tensors list, int64_t t)
{
    return list && t >= 0 && t < static_cast<int64_t>(list->shape.size.size()) ? list->shape.state_off[static_cast<size_t>(t)] : -1;
}

ob_status ob_grad_norm(ob_tensors list, const void* const* g, float g_mult, float max_norm,
                       const ob_adamw_hparams* hp, ob_control* control, hipStream_t stream)
try {
    if (!list) return OB_ERR_ARG;
    const ob_tensors_s& l = *list;
    if (ob_status st = ob::check_norm(l.shape, g, g_mult, max_norm, hp, control)) return st;
    DeviceGuard guard(l.device);
    if (!guard.ok) return OB_ERR_HIP;

    // every launch has the same grid, so that the first one writes all partial sums and later ones add
    int grid = 0, launches = 0;
    int64_t left = 0;
    (void)ob::for_runs(l.shape, ob::kNormPtrs, false, [&](int64_t k, int64_t e) {
        const int64_t items = l.norm.first[e] - l.norm.first[k];
        grid = std::max(grid, static_cast<int>(std::min<int64_t>(items, OB_CONTROL_PARTIALS)));
        launches += items > 0;
        for (int64_t j = k; j < e; ++j) left += l.shape.size[l.shape.order[j]] * ob::dtype_bytes(l.shape.g_dtype[l.shape.order[j]]);
        return OB_OK;
    });
    ob::NormParams np;
    np.g_mult = g_mult;
    np.max_norm = max_norm;
    np.clip = max_norm > 0.0f && !std::isinf(max_norm);
    np.advance = hp != nullptr;
    np.beta1 = hp ? hp->beta1 : 0.0;
    np.beta2 = hp ? hp->beta2 : 0.0;
    np.first = 1;
    ob::NormPtrs ptrs;
    const ob_status st = ob::for_runs(l.shape, ob::kNormPtrs, false, [&](int64_t k, int64_t e) {
        const ob::ListLaunch L{l.norm.d_items + l.norm.first[k], l.d_tensors, l.norm.first[e] - l.norm.first[k],
                               static_cast<int32_t>(k)};
        if (L.n_items == 0) return OB_OK;
        const int gd = l.shape.g_dtype[l.shape.order[k]];
        for (int64_t j = k; j < e; ++j) ptrs.g[j - k] = g[l.shape.order[j]];
        // items before the last kKeepBytes of the call
        const int64_t nt = std::max<int64_t>(0, (left - kKeepBytes) / (kNormElems * ob::dtype_bytes(gd)));
        left -= L.n_items * kNormElems * ob::dtype_bytes(gd);
        np.ticket = --launches == 0 && grid <= kTicketGrid;
        (void)hipGetLastError();
        const hipError_t err = ob::launch_grad_sumsq(L, ptrs, gd, grid, nt, control, np, stream);
        np.first = 0;
        return err == hipSuccess ? OB_OK : OB_ERR_HIP;
    });
    if (st != OB_OK || (grid > 0 && grid <= kTicketGrid)) return st;
    (void)hipGetLastError();
    return ob::launch_grad_control(control, grid, np, stream) == hipSuccess ? OB_OK : OB_ERR_HIP;
} catch (...) {
    return OB_ERR_OOM;
}

ob_status ob_adamw_check(ob_tensors list, const void* const* g, void* const* p, const float* master, const float* m,
                         const float* v, const ob_adamw_hparams* hp, const ob_control* control)
try {
    if (!list) return OB_ERR_ARG;
    if (ob_status st = ob::check_step(list->shape, g, p, master, false, hp, control)) return st;
    if (list->shape.n == 0) return OB_OK;
    if (!m || !v) return OB_ERR_ARG;
    return ob::is_aligned(m, 16) && ob::is_aligned(v, 16) ? OB_OK : OB_ERR_ALIGN;
} catch (...) {
    return OB_ERR_OOM;
}

ob_status ob_adamw_step(ob_tensors list, const void* const* g, void* const* p, float* master, float* m, float* v,
                        const ob_adamw_hparams* hp, const ob_control* control, hipStream_t stream)
try {
    if (ob_status st = ob_adamw_check(list, g, p, master, m, v, hp, control)) return st;
    if (list->shape.n == 0) return OB_OK;
    const ob::AdamWParams ap = adamw_params(hp, control);
    const ob::State32 state{master, m, v};
    DeviceGuard guard(list->device);
    if (!guard.ok) return OB_ERR_HIP;
    return launch_step(*list, g, p, master != nullptr,
                       [&](int gd, int pk, const ob::ListLaunch& L, const ob::ListPtrs& ptrs) {
                           return gd == OB_BF16  ? ob::launch_adamw<OB_BF16>(L, ptrs, pk, state, ap, stream)
                                  : gd == OB_F16 ? ob::launch_adamw<OB_F16>(L, ptrs, pk, state, ap, stream)
                                                 : ob::launch_adamw<OB_F32>(L, ptrs, pk, state, ap, stream);
                       });
} catch (...) {
    return OB_ERR_OOM;
}

ob_status ob_adamw8_check(ob_tensors list, const void* const* g, void* const* p, const float* master,
                          const int8_t* m_codes, const float* m_scales, const uint8_t* v_codes, const float* v_scales,
                          const ob_adamw_hparams* hp, const ob_control* control)
try {
    if (!list) return OB_ERR_ARG;
    if (ob_status st = ob::check_step(list->shape, g, p, master, true, hp, control)) return st;
    if (list->shape.n == 0) return OB_OK;
    if (!m_codes || !m_scales || !v_codes || !v_scales) return OB_ERR_ARG;
    if (!ob::is_aligned(m_codes, 4) || !ob::is_aligned(v_codes, 4) || !ob::is_aligned(m_scales, 4) || !ob::is_aligned(v_scales, 4))
        return OB_ERR_ALIGN;
    return OB_OK;
} catch (...) {
    return OB_ERR_OOM;
}

ob_status ob_adamw8_step(ob_tensors list, const void* const* g, void* const* p, float* master, int8_t* m_codes,
                         float* m_scales, uint8_t* v_codes, float* v_scales, const ob_adamw_hparams* hp,
                         const ob_control* control, hipStream_t stream)
try {
    if (ob_status st = ob_adamw8_check(list, g, p, master, m_codes, m_scales, v_codes, v_scales, hp, control)) return st;
    if (list->shape.n == 0) return OB_OK;
    const ob::AdamWParams ap = adamw_params(hp, control);
    const ob::State8 state{master, m_codes, m_scales, v_codes, v_scales};
    DeviceGuard guard(list->device);
    if (!guard.ok) return OB_ERR_HIP;
    return launch_step(*list, g, p, master != nullptr,
                       [&](int gd, int pk, const ob::ListLaunch& L, const ob::ListPtrs& ptrs) {
                           return gd == OB_BF16  ? ob::launch_adamw8<OB_BF16>(L, ptrs, pk, state, ap, stream)
                                  : gd == OB_F16 ? ob::launch_adamw8<OB_F16>(L, ptrs, pk, state, ap, stream)
                                                 : ob::launch_adamw8<OB_F32>(L, ptrs, pk, state, ap, stream);
                       });
} catch (...) {
    return OB_ERR_OOM;
}

ob_status ob_state8_encode(int64_t n, const float* m, const float* v, int8_t* m_codes, float* m_scales,
                           uint8_t* v_codes, float* v_scales, hipStream_t stream)
{
    if (ob_status st = ob::check_state8(n, m, v, m_codes, m_scales, v_codes, v_scales)) return st;
    return ob::for_parts(n, kState8Part, [&](int64_t i, int64_t count) {
        (void)hipGetLastError();
        return ob::launch_state8_encode(count, at(m, i), at(v, i), at(m_codes, i), at(m_scales, i / OB_STATE_BLOCK),
                                        at(v_codes, i), at(v_scales, i / OB_STATE_BLOCK), stream) == hipSuccess
                   ? OB_OK
                   : OB_ERR_HIP;
    });
}

ob_status ob_state8_decode(int64_t n, const int8_t* m_codes, const float* m_scales, const uint8_t* v_codes,
                           const float* v_scales, float* m, float* v, hipStream_t stream)
{
    if (ob_status st = ob::check_state8(n, m, v, m_codes, m_scales, v_codes, v_scales)) return st;
    return ob::for_parts(n, kState8Part, [&](int64_t i, int64_t count) {
        (void)hipGetLastError();
        return ob::launch_state8_decode(count, at(m_codes, i), at(m_scales, i / OB_STATE_BLOCK), at(v_codes, i),
                                        at(v_scales, i / OB_STATE_BLOCK), at(m, i), at(v, i), stream) == hipSuccess
                   ? OB_OK
                   : OB_ERR_HIP;
    });
}

}  // extern "C"
