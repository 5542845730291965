// ob_muon_api.cpp -- host side of the Muon step (declarations and contracts in ob_adam.h).
#include "ob_adam.h"
#include "ob_list_handle.h"
#include "ob_muon_kernels.h"

struct ob_muon_s {
    int device = 0;
    ob::ListShape list;
    ob::MuonShape shape;
    const ob::MuonMatrix* d_matrices = nullptr;
    const ob::MuonItem* d_items = nullptr;
    const ob::MuonTile* d_write = nullptr;
    const ob::MuonTile* d_tiles = nullptr;
    void* d_tables = nullptr;
};

namespace {

// Tensors of a group: their addresses are a launch's arguments, beside a call's own.
constexpr int kMuonPlaces = 200;
static_assert(kMuonPlaces <= ob::kListPtrs && sizeof(ob::ListPtrs) + sizeof(ob::MuonCall) + 16 <= 4096, "a launch's arguments fit 4 KB");

void free_plan(ob_muon p)
{
    if (!p) return;
    if (p->d_tables) (void)hipFree(p->d_tables);
    delete p;
}

ob_status plan_create(ob_tensors list, const int64_t* rows, const int64_t* cols, ob_muon* out, ob_muon& p)
{
    if (!out) return OB_ERR_ARG;
    *out = nullptr;
    if (!list) return OB_ERR_ARG;
    p = new ob_muon_s;
    p->device = list->device;
    p->list = list->shape;
    if (ob_status st = ob::build_muon(p->list, list->lr_mults.data(), list->wd_mults.data(), rows, cols, kMuonPlaces, p->shape)) return st;
    const ob::MuonShape& s = p->shape;
    std::vector<char> tables;
    auto put = [&](const auto& v) {   // v behind what is there, at a multiple of 16 bytes; its offset
        const size_t at = (tables.size() + 15) / 16 * 16, bytes = v.size() * sizeof(v[0]);
        tables.resize(at + bytes);
        std::copy_n(reinterpret_cast<const char*>(v.data()), bytes, tables.data() + at);
        return at;
    };
    const size_t a = put(s.matrices), b = put(s.items), c = put(s.write), d = put(s.tiles);
    if (!s.matrices.empty()) {
        ob::DeviceGuard guard(p->device);
        if (!guard.ok) return OB_ERR_HIP;
        hipError_t e = hipMalloc(&p->d_tables, tables.size());
        if (e == hipSuccess) e = hipMemcpy(p->d_tables, tables.data(), tables.size(), hipMemcpyHostToDevice);
        // a first call may be on a stream that does not wait for the null stream
        if (e == hipSuccess) e = hipStreamSynchronize(nullptr);
        if (e != hipSuccess) return e == hipErrorOutOfMemory ? OB_ERR_OOM : OB_ERR_HIP;
        const char* t = static_cast<const char*>(p->d_tables);
        p->d_matrices = reinterpret_cast<const ob::MuonMatrix*>(t + a);
        p->d_items = reinterpret_cast<const ob::MuonItem*>(t + b);
        p->d_write = reinterpret_cast<const ob::MuonTile*>(t + c);
        p->d_tiles = reinterpret_cast<const ob::MuonTile*>(t + d);
        // the host keeps the groups
        p->shape.matrices = {};
        p->shape.items = {};
        p->shape.write = {};
        p->shape.tiles = {};
    }
    *out = p;
    return OB_OK;
}

}  // namespace

extern "C" {

ob_status ob_muon_create(ob_tensors list, const int64_t* rows, const int64_t* cols, ob_muon* out)
{
    ob_muon p = nullptr;
    ob_status st;
    try {
        st = plan_create(list, rows, cols, out, p);
    } catch (...) {
        st = OB_ERR_OOM;  // host allocation failures are the only exceptions here
    }
    if (st != OB_OK) free_plan(p);
    return st;
}

ob_status ob_muon_destroy(ob_muon plan)
try {
    if (!plan) return OB_ERR_ARG;
    ob::DeviceGuard guard(plan->device);
    free_plan(plan);
    return OB_OK;
} catch (...) {
    return OB_ERR_OOM;
}

int64_t ob_muon_workspace(ob_muon plan) { return plan ? plan->shape.workspace() : -1; }

ob_status ob_muon_check(ob_muon plan, const void* const* g, void* const* p, const float* master, const float* m,
                        const void* workspace, const ob_muon_hparams* hp, const ob_control* control)
try {
    if (!plan) return OB_ERR_ARG;
    return ob::check_muon(plan->list, g, p, master, m, workspace, plan->shape.workspace(), hp, control);
} catch (...) {
    return OB_ERR_OOM;
}

ob_status ob_muon_step(ob_muon plan, const void* const* g, void* const* p, float* master, float* m, void* workspace,
                       const ob_muon_hparams* hp, const ob_control* control, hipStream_t stream)
try {
    if (ob_status st = ob_muon_check(plan, g, p, master, m, workspace, hp, control)) return st;
    const ob::ListShape& l = plan->list;
    const ob::MuonShape& s = plan->shape;
    if (l.n == 0) return OB_OK;
    ob::DeviceGuard guard(plan->device);
    if (!guard.ok) return OB_ERR_HIP;
    ob::MuonCall c;
    c.nesterov = hp->nesterov;
    c.scale = hp->scale;
    c.momentum = hp->momentum;
    c.lr = hp->lr;
    c.wd = hp->weight_decay;
    c.eps = hp->eps;
    c.m = m;
    c.master = master;
    c.half = static_cast<uint16_t*>(workspace);
    c.parts = reinterpret_cast<double*>(static_cast<char*>(workspace) + 2 * s.half_elems);
    c.factor = reinterpret_cast<float*>(c.parts + s.parts);
    c.control = control;
    ob::ListPtrs ptrs;
    (void)hipGetLastError();  // clear a stale error so the checks see these launches only
    int gd = 0, pk = 0;
    // the addresses of a group's tensors; whether any has a gradient
    auto take = [&](int64_t place0, int64_t places) {
        bool any = false;
        for (int64_t j = 0; j < places; ++j) {
            const int32_t t = l.order[place0 + j];
            ptrs.g[j] = l.size[t] > 0 ? g[t] : nullptr;
            ptrs.p[j] = l.size[t] > 0 ? p[t] : nullptr;
            any = any || ptrs.g[j];
        }
        const int32_t t0 = l.order[place0];
        gd = l.g_dtype[t0];
        pk = l.p_dtype[t0] == OB_F32 ? ob::PK_F32 : l.p_dtype[t0] + (master ? 2 : 0);
        c.place0 = static_cast<int32_t>(place0);
        return any;
    };
    for (const ob::MuonSmall& q : s.small) {
        if (!take(q.place0, q.places)) continue;
        c.matrices = plan->d_matrices + q.matrices.first;
        if (ob::launch_muon_small(c, ptrs, q.matrices.count, gd, pk, hp->iterations, q.lds, stream) != hipSuccess) return OB_ERR_HIP;
    }
    for (const ob::MuonGroup& q : s.groups) {
        if (!take(q.place0, q.places)) continue;
        c.matrices = plan->d_matrices + q.matrices.first;
        c.items = plan->d_items + q.items.first;
        c.write = plan->d_write + q.write.first;
        if (ob::launch_muon_momentum(c, ptrs, gd, q.items.count, stream) != hipSuccess) return OB_ERR_HIP;
        if (ob::launch_muon_factor(c, q.matrices.count, stream) != hipSuccess) return OB_ERR_HIP;
        if (ob::launch_muon_write(c, ptrs, gd, q.write.count, stream) != hipSuccess) return OB_ERR_HIP;
        for (int turn = 0; turn < hp->iterations; ++turn)
            for (int k = 0; k < 3; ++k) {
                const ob::MuonTile* tiles = plan->d_tiles + q.tiles[k].first;
                const hipError_t e = k == ob::MUON_STEP && turn == hp->iterations - 1
                                         ? ob::launch_muon_last(c, ptrs, tiles, q.tiles[k].count, q.tile[k], turn, pk, stream)
                                         : ob::launch_muon_product(c, k, tiles, q.tiles[k].count, q.tile[k], turn, stream);
                if (e != hipSuccess) return OB_ERR_HIP;
            }
    }
    return OB_OK;
} catch (...) {
    return OB_ERR_OOM;
}

}  // extern "C"
