// ob_muon_kernels.h -- shared between the host side (ob_muon_api.cpp) and the kernels (ob_muon.hip) of the Muon step.
#pragma once

#include "ob_adamw.h"
#include "ob_muon.h"

namespace ob {

// One group of a call.
struct MuonCall {
    const MuonMatrix* matrices;   // of the group
    const MuonItem* items;
    const MuonTile* write;
    int32_t place0;               // place of the launch's first tensor
    int32_t nesterov, scale;
    double momentum, lr, wd, eps;
    float* m;
    float* master;
    uint16_t* half;               // the workspace: 16-bit matrices, partial sums, factors of u
    double* parts;
    float* factor;
    const ob_control* control;
};

hipError_t launch_muon_momentum(const MuonCall& c, const ListPtrs& ptrs, int g_dtype, int64_t items, hipStream_t s);
hipError_t launch_muon_factor(const MuonCall& c, int64_t matrices, hipStream_t s);
hipError_t launch_muon_write(const MuonCall& c, const ListPtrs& ptrs, int g_dtype, int64_t tiles, hipStream_t s);
// One product of iteration `turn` (X is x[turn % 2]); tile: place in kTileSize.
hipError_t launch_muon_product(const MuonCall& c, int product, const MuonTile* tiles, int64_t count, int tile, int turn, hipStream_t s);
// The last MUON_STEP, whose result goes into the parameters of kind pk.
hipError_t launch_muon_last(const MuonCall& c, const ListPtrs& ptrs, const MuonTile* tiles, int64_t count, int tile, int turn, int pk,
                            hipStream_t s);

// The whole step for matrices that fit a compute unit's LDS: one work group for each; lds: place in kMuonSmallLds.
hipError_t launch_muon_small(const MuonCall& c, const ListPtrs& ptrs, int64_t matrices, int g_dtype, int pk, int iterations, int lds,
                             hipStream_t s);

}  // namespace ob
