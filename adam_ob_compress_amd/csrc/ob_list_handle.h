// ob_list_handle.h -- what an ob_tensors handle holds, for the host sides of the calls over lists of tensors.
#pragma once

#include "ob_adamw.h"

// The work blocks of a list on its device.
struct ob_list_table {
    std::vector<int64_t> first;      // [T + 1]: items of the tensor in place k are [first[k], first[k+1])
    const ob::ListItem* d_items = nullptr;
};

struct ob_tensors_s {
    int device = 0;
    ob::ListShape shape;
    std::vector<float> lr_mults, wd_mults;      // by place
    ob_list_table step, norm;
    const ob::ListTensor* d_tensors = nullptr;  // by place
    const int64_t* d_norm_first = nullptr;      // norm.first
    const int32_t* d_order = nullptr;           // shape.order
    void* d_tables = nullptr;                   // one allocation: the items of both tables, the tensors, the two above
};

namespace ob {

// Elements per item of the steps and of the norms.
constexpr int64_t kStepElems = kStepTiles * kListTile;
constexpr int64_t kNormElems = 16 * kListTile;

// Gradient bytes at a call's end that the norm reads with ordinary loads, which leave them in the last-level
// cache for the step that follows; what comes before is read nontemporally, which is faster.  Norm and step
// of 1.09e8 elements: bf16 278 us with ordinary loads and 293 nontemporal, fp32 (436 MB) 554 and 592; norm alone
// of 3.1 GB: 513 and 452.
constexpr int64_t kKeepBytes = int64_t(256) << 20;

// A device is current for the duration of a call.
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

}  // namespace ob
