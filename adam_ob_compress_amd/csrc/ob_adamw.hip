// ob_adamw.hip -- AdamW steps over lists of tensors, with states in fp32 (k_adamw) and in 8 bits
// (k_adamw8); compiled once per gradient type (OB_AW_G: 0 fp32, 1 bf16, 2 fp16).
//
// Both are one pass over the data: every array is read once and written once.  HBM bounds them, but for
// 16-bit parameters with 8-bit states rounded by chance, where the vector ALU does (see k_adamw8).  A
// work group takes part of one tensor; a lane takes four consecutive elements of a 256-element state block
// per wave.  The tensors' addresses are launch arguments; parameters and gradients may start
// at any element (vector loads of element alignment), states are aligned by their layout.  Loads and stores are
// nontemporal: no byte is touched twice.
#include "ob_any.h"
#include "ob_state8.h"

#include <type_traits>

#ifndef OB_AW_G
#error "OB_AW_G selects the gradient type"
#endif

namespace ob {
namespace {

// Parameters by kind: i the element in the tensor, si the state index (of the master copy).
template <int PK>
struct Par {
    static constexpr bool kMaster = PK == PK_MASTER_BF16 || PK == PK_MASTER_F16;
    static constexpr int D = kMaster ? PK - 2 : PK;    // type behind p
    static constexpr bool kRound = !kMaster && D != 0; // the parameter itself is held in 16 bits

    static __device__ __forceinline__ f4 load4(const void* p, const float* master, int64_t i, int64_t si)
    {
        return kMaster ? ld4<true>(master, si) : load_any4<D>(p, i);
    }
    static __device__ __forceinline__ float load1(const void* p, const float* master, int64_t i, int64_t si)
    {
        return kMaster ? master[si] : load_any1<D>(p, i);
    }
    // x: new parameters in fp32; w: random words of the four elements (kRound with SR)
    template <bool SR>
    static __device__ __forceinline__ void store4(void* p, float* master, int64_t i, int64_t si, f4 x, const u4& w)
    {
        if (kMaster) st4<true>(master, si, x);
        store_any4<D, SR && kRound>(p, i, x, w);
    }
    template <bool SR>
    static __device__ __forceinline__ void store1(void* p, float* master, int64_t i, int64_t si, float x, uint32_t w)
    {
        if (kMaster) master[si] = x;
        store_any1<D, SR && kRound>(p, i, x, w);
    }
};

// What a block needs besides its item: from the arguments or the control block.
struct Step {
    float scale;
    double lr, wd, bc1, bc2;
    uint64_t t;
    bool skip;
};

__device__ __forceinline__ Step step_of(const AdamWParams& ap, const ListTensor& tn)
{
    Step s;
    s.scale = 1.0f;
    s.lr = ap.lr * static_cast<double>(tn.lr_mult);
    s.wd = ap.wd * static_cast<double>(tn.wd_mult);
    s.bc1 = ap.bc1;
    s.bc2 = ap.bc2;
    s.t = ap.step;
    s.skip = false;
    if (ap.control) {
        s.scale = ap.control->grad_scale;
        s.lr *= static_cast<double>(ap.control->lr_scale);
        if (ap.bias_correction) {
            s.bc1 = ap.control->bc1;
            s.bc2 = ap.control->bc2;
        }
        s.t = static_cast<uint64_t>(ap.control->step);
        s.skip = ap.control->skip != 0;
    }
    return s;
}

constexpr uint64_t kParStream = uint64_t(1) << 63;  // the counter's top bit: words for 16-bit parameters

// ------------------------------------------------------------------------------------------------
// fp32 states
// ------------------------------------------------------------------------------------------------

// One element; every line in double from fp32 operands, rounded once (a large update may nearly cancel
// p), in the order of the dense step, so that without decay and scale the bits are the dense step's.
__device__ __forceinline__ void adamw_elem(float g, float& mm, float& vv, float& pp, const Step& s, const AdamWParams& ap)
{
    const double gd = static_cast<double>(mul(g, s.scale));
    mm = static_cast<float>(ap.beta1 * static_cast<double>(mm) + ap.one_m_beta1 * gd);
    vv = static_cast<float>(ap.beta2 * static_cast<double>(vv) + ap.one_m_beta2 * (gd * gd));
    double mh = static_cast<double>(mm), vh = static_cast<double>(vv);
    if (ap.bias_correction) {
        mh = mh / s.bc1;
        vh = vh / s.bc2;
    }
    const double pd = static_cast<double>(pp);
    const double u = mh / (sqrt(vh) + ap.eps) + s.wd * pd;
    pp = static_cast<float>(pd - s.lr * u);
}

// m = b1 m + (1-b1) g;  v = b2 v + (1-b2) g^2;  p -= lr ((m/bc1) / (sqrt(v/bc2) + eps) + wd p).
// Bound by HBM: 22 to 28 bytes an element.  Measured (MI355X): 1.09e8 fp32 elements 500 us, 6.1 TB/s; 1.56e9 bf16
// parameters with a master 6.8 to 7.7 ms by the placement of the buffers, 5.7 to 6.4 TB/s; the double-precision
// lines hide (without the two divisions by bc1, bc2 the time is the same).
// One tile of an item per work group.  Two tiles, their loads ahead of the arithmetic, were 3 to 5 percent
// slower (1.56e9 bf16 parameters with a master 7.90 ms against 7.67, 1e9 without 3.93 against 3.79), consecutive
// tiles on one XCD 1 to 7 percent, ordinary loads or stores 7 to 14 percent.
template <int G, int PK, bool SR>
__global__ __launch_bounds__(kListBlock) void k_adamw(ListLaunch L, ListPtrs ptrs, State32 st, AdamWParams ap)
{
    using P = Par<PK>;
    const ListItem it = L.items[blockIdx.x / kStepTiles];
    const int at = static_cast<int>(blockIdx.x % kStepTiles) * kListTile + 4 * static_cast<int>(threadIdx.x);
    const void* g = ptrs.g[it.tensor - L.tensor0];
    const int cnt = it.len - at;
    if (g == nullptr || cnt <= 0) return;
    void* p = ptrs.p[it.tensor - L.tensor0];
    const ListTensor tn = L.tensors[it.tensor];
    const Step s = step_of(ap, tn);
    if (s.skip) return;
    const int64_t i = it.start + at, si = tn.state_off + i;
    u4 w{};
    if (SR) {   // by wave: a tensor's state starts at a multiple of 256 elements, which are a wave's 64 lanes
        const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
        const int64_t first = tn.state_off + it.start + static_cast<int>(blockIdx.x % kStepTiles) * kListTile + wave * kStateBlock;
        w = philox_lanes(ap.seed, s.t | kParStream, first >> 2, threadIdx.x & 63);
    }
    if (cnt >= 4) {
        const f4 gv = load_any4<G>(g, i);
        f4 mv = ld4<true>(st.m, si), vv = ld4<true>(st.v, si), pv = P::load4(p, st.master, i, si);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float mm = mv[k], vq = vv[k], pp = pv[k];
            adamw_elem(gv[k], mm, vq, pp, s, ap);
            mv[k] = mm;
            vv[k] = vq;
            pv[k] = pp;
        }
        st4<true>(st.m, si, mv);
        st4<true>(st.v, si, vv);
        P::template store4<SR>(p, st.master, i, si, pv, w);
        return;
    }
    for (int k = 0; k < cnt; ++k) {
        float mm = st.m[si + k], vq = st.v[si + k], pp = P::load1(p, st.master, i + k, si + k);
        adamw_elem(load_any1<G>(g, i + k), mm, vq, pp, s, ap);
        st.m[si + k] = mm;
        st.v[si + k] = vq;
        P::template store1<SR>(p, st.master, i + k, si + k, pp, k == 0 ? w.x[0] : k == 1 ? w.x[1] : w.x[2]);
    }
}

// ------------------------------------------------------------------------------------------------
// 8-bit states
// ------------------------------------------------------------------------------------------------

// Constants of the fp32 lines.
struct Step8 {
    float scale, b1, c1, b2, c2, root_factor, eps, lr, wd;   // root_factor, eps: times bc1, see adamw8_elem
};

__device__ __forceinline__ Step8 step8_of(const Step& s, const AdamWParams& ap)
{
    Step8 r;
    r.scale = s.scale;
    r.b1 = static_cast<float>(ap.beta1);
    r.c1 = static_cast<float>(ap.one_m_beta1);
    r.b2 = static_cast<float>(ap.beta2);
    r.c2 = static_cast<float>(ap.one_m_beta2);
    const bool own = ap.control && ap.bias_correction;
    r.root_factor = own ? ap.control->root_factor : ap.root_factor;
    r.eps = static_cast<float>(ap.eps * (own ? ap.control->bc1 : ap.bc1));
    r.lr = static_cast<float>(s.lr);
    r.wd = static_cast<float>(s.wd);
    return r;
}

// Moments and parameter of one element; root: about sqrt(v).  (m/bc1) / (sqrt(v/bc2) + eps) as
// m / (sqrt(v) * bc1/sqrt(bc2) + eps * bc1).
__device__ __forceinline__ void adamw8_elem(float g, float& mm, float& vv, float& pp, float& root, const Step8& s)
{
    g = mul(g, s.scale);
    mm = __builtin_fmaf(s.b1, mm, mul(s.c1, g));
    vv = __builtin_fmaf(s.b2, vv, mul(s.c2, mul(g, g)));
    root = __builtin_amdgcn_sqrtf(vv);
    const float den = fmaf(root, s.root_factor, s.eps);
    const float u = fmaf(mm, __builtin_amdgcn_rcpf(den), s.wd * pp);
    pp = fmaf(-s.lr, u, pp);
}

// A wave's span of S state blocks: elements from `at` on of the tensor, `left` of them there (FULL: all).
template <int G, int PK, bool SR, int S, bool FULL>
__device__ __forceinline__ void span8(const void* g, void* p, const State8& st, int64_t state_off, int64_t at, int left,
                                      const Step8& s, uint64_t seed, uint64_t t)
{
    using P = Par<PK>;
    const int lane4 = 4 * (static_cast<int>(threadIdx.x) & 63);
    const int64_t sb = (state_off + at) / kStateBlock;
    const int blocks = (left + kStateBlock - 1) / kStateBlock;
    float gv[S][4], pv[S][4], mv[S][4], vv[S][4], root[S][4];
    uint32_t mw[S], vw[S], tm[S], tv[S];
    const f4 qm = load_scales<S, FULL>(st.mq, sb, blocks), qv = load_scales<S, FULL>(st.vq, sb, blocks);
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const int64_t i = at + j * kStateBlock + lane4, si = state_off + i;
        const int cnt = FULL ? 4 : left - j * kStateBlock - lane4;
        mw[j] = load_codes<FULL, true>(st.mc, si, cnt);
        vw[j] = load_codes<FULL, true>(st.vc, si, cnt);
        f4 g4{}, p4{};
        if (FULL || cnt >= 4) {
            g4 = load_any4<G>(g, i);
            p4 = P::load4(p, st.master, i, si);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k >= cnt) continue;
                g4[k] = load_any1<G>(g, i + k);
                p4[k] = P::load1(p, st.master, i + k, si + k);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            gv[j][k] = g4[k];
            pv[j][k] = p4[k];
        }
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const int64_t i = at + j * kStateBlock + lane4, si = state_off + i;
        const int cnt = FULL ? 4 : left - j * kStateBlock - lane4;
        decode4<false>(mw[j], qm[j], mv[j]);
        decode4<true>(vw[j], qv[j], vv[j]);
        tm[j] = tv[j] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            adamw8_elem(gv[j][k], mv[j][k], vv[j][k], pv[j][k], root[j][k], s);
            if (FULL || k < cnt) {   // what is behind the tensor's end does not enter the scales
                tm[j] = max_u(tm[j], __float_as_uint(mv[j][k]) & 0x7fffffffu);
                tv[j] = max_u(tv[j], __float_as_uint(vv[j][k]));   // v >= 0, or a NaN of either sign
            }
        }
        u4 w{};
        if (SR && P::kRound) w = philox_lanes(seed, t | kParStream, (state_off + at + j * kStateBlock) >> 2, lane4 >> 2);
        if (FULL || cnt >= 4) {
            f4 p4;
#pragma unroll
            for (int k = 0; k < 4; ++k) p4[k] = pv[j][k];
            P::template store4<SR>(p, st.master, i, si, p4, w);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < cnt) P::template store1<SR>(p, st.master, i + k, si + k, pv[j][k], w.x[k]);
        }
    }
    const SpanScales q = span_scales<S>(tm, tv);
    store_scales<S, FULL>(st.mq, st.vq, sb, blocks, q);
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const int64_t si = state_off + at + j * kStateBlock + lane4;
        const int cnt = FULL ? 4 : left - j * kStateBlock - lane4;
        u4 w{};
        if (SR) w = philox_lanes(seed, t, (state_off + at + j * kStateBlock) >> 2, lane4 >> 2);
        store_codes<FULL>(st.mc, si, cnt, encode4<false, SR>(mv[j], nullptr, q.get(j, false), w));
        store_codes<FULL>(st.vc, si, cnt, encode4<true, SR>(vv[j], root[j], q.get(j, true), w));
    }
}

// The step with 8-bit states: decode, moments, parameter; then the scales of the new moments and their codes.
// Bytes: 10 to 16 an element and 16 per 256.  Operations: 49 of the vector ALU an element to nearest, 86
// by chance (random words 9, codes), 101 with 16-bit parameters rounded by chance too.  Measured (MI355X), 1e9
// elements: fp32 parameters 2.36 ms and bf16 with a master 2.68 ms, 5.9 to 6.0 TB/s, bf16 1.65 ms, 6.1 TB/s, all by
// HBM; bf16 by chance 2.51 to 2.55 ms, 4.0 TB/s, by the ALU (40e12 operations a second).
// S state blocks per wave.  A long list takes four: their loads are in flight together (one block per trip:
// 2.56 ms for fp32 parameters), and the scales' reductions and roots are paid once for four.  (The codes with ordinary
// loads: 2.47 ms, with ordinary stores 2.59.)  A short list, which
// leaves most of the card idle, takes one, so that more waves share the work.
template <int G, int PK, bool SR, int S>
__global__ __launch_bounds__(kListBlock) void k_adamw8(ListLaunch L, ListPtrs ptrs, State8 st, AdamWParams ap)
{
    constexpr int kParts = kSpan / S;   // work groups per item
    const ListItem it = L.items[blockIdx.x / kParts];
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int base = (static_cast<int>(blockIdx.x % kParts) * (kListBlock / 64) + wave) * S * kStateBlock;
    const void* g = ptrs.g[it.tensor - L.tensor0];
    const int left = it.len - base;   // uniform over a wave
    if (g == nullptr || left <= 0) return;
    void* p = ptrs.p[it.tensor - L.tensor0];
    const ListTensor tn = L.tensors[it.tensor];
    const Step sd = step_of(ap, tn);
    if (sd.skip) return;
    const Step8 s = step8_of(sd, ap);
    if (left >= S * kStateBlock)
        span8<G, PK, SR, S, true>(g, p, st, tn.state_off, it.start + base, left, s, ap.seed, sd.t);
    else
        span8<G, PK, SR, S, false>(g, p, st, tn.state_off, it.start + base, left, s, ap.seed, sd.t);
}

// ------------------------------------------------------------------------------------------------
// launches
// ------------------------------------------------------------------------------------------------

// Items (of up to 4096 elements) up to which a launch takes one state block per wave, against four.  fp32 parameters,
// to nearest: 26 items 3.8 us and 6.8, 313 5.2 and 8.0, 2021 20.8 and 21.7, 1.09e8 elements 265 and 250; bf16
// by chance: 26 4.2 and 8.4, 2021 25.5 and 25.6, 3973 46.5 and 43.5.
constexpr int64_t kShortItems = 2048;

// f(kind as a constant, rounding as a constant) for the run-time values
template <class F>
hipError_t by_kind(int pk, int sr, F&& f)
{
#define OB_KIND(K)                                                                                              \
    case K:                                                                                                     \
        return sr ? f(std::integral_constant<int, K>{}, std::true_type{})                                       \
                  : f(std::integral_constant<int, K>{}, std::false_type{});
    switch (pk) {
        OB_KIND(PK_F32)
        OB_KIND(PK_BF16)
        OB_KIND(PK_F16)
        OB_KIND(PK_MASTER_BF16)
        OB_KIND(PK_MASTER_F16)
    }
#undef OB_KIND
    return hipErrorInvalidValue;
}

}  // namespace

template <int G>
hipError_t launch_adamw(const ListLaunch& L, const ListPtrs& ptrs, int pk, const State32& st, const AdamWParams& ap,
                        hipStream_t s)
{
    // only 16-bit parameters are rounded by chance here
    const int sr = ap.stochastic && (pk == PK_BF16 || pk == PK_F16);
    return by_kind(pk, sr, [&](auto k, auto r) {
        constexpr int PK = decltype(k)::value;
        constexpr bool SR = decltype(r)::value && Par<PK>::kRound;
        hipLaunchKernelGGL((k_adamw<G, PK, SR>), dim3(static_cast<unsigned>(L.n_items * kStepTiles)), dim3(kListBlock), 0, s, L,
                           ptrs, st, ap);
        return hipGetLastError();
    });
}

template <int G>
hipError_t launch_adamw8(const ListLaunch& L, const ListPtrs& ptrs, int pk, const State8& st, const AdamWParams& ap,
                         hipStream_t s)
{
    return by_kind(pk, ap.stochastic, [&](auto k, auto r) {
        constexpr int PK = decltype(k)::value;
        constexpr bool SR = decltype(r)::value;
        if (L.n_items <= kShortItems)
            hipLaunchKernelGGL((k_adamw8<G, PK, SR, 1>), dim3(static_cast<unsigned>(L.n_items * kSpan)), dim3(kListBlock),
                               0, s, L, ptrs, st, ap);
        else
            hipLaunchKernelGGL((k_adamw8<G, PK, SR, kSpan>), dim3(static_cast<unsigned>(L.n_items)), dim3(kListBlock), 0,
                               s, L, ptrs, st, ap);
        return hipGetLastError();
    });
}

template hipError_t launch_adamw<OB_AW_G>(const ListLaunch&, const ListPtrs&, int, const State32&, const AdamWParams&,
                                          hipStream_t);
template hipError_t launch_adamw8<OB_AW_G>(const ListLaunch&, const ListPtrs&, int, const State8&, const AdamWParams&,
                                           hipStream_t);

}  // namespace ob
