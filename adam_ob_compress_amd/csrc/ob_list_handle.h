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
    ob_list_table step, norm;
    const ob::ListTensor* d_tensors = nullptr;  // by place
    void* d_tables = nullptr;                   // one allocation: the items of both tables, the tensors
};

namespace ob {

// Elements per item of the steps and of the norms.
constexpr int64_t kStepElems = kStepTiles * kListTile;
constexpr int64_t kNormElems = 16 * kListTile;

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
