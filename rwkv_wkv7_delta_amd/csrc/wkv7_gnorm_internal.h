// wkv7_gnorm_internal.h -- launcher interface of the group norm (contracts in
// include/wkv7.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace wkv7 {

// How a launch takes rows of G groups of W channels: `lanes` lanes and `each` pieces of
// `vec` channels per lane for a group, `groups` groups by `rows` rows side by side in a
// workgroup of `threads`, `blocks` of them over the groups and `parts` over the rows.
// each = 0: groups too wide for registers, read again for each of their sums.
struct GnPlan {
    int vec, lanes, each, groups, rows, threads;
    unsigned blocks, parts;
};

struct GnArgs {
    int64_t rows;
    int D, G, W;
    bool bf16, center, silu;
    int gate;                    // 0 none, 1 after the norm, 2 before
    float eps;
    const float *gamma, *beta;   // may be null
    const void *x, *z;           // z null without a gate
    void* y;
    // The backward:
    const void* dy;
    void *dx, *dz;
    float *dgamma, *dbeta;       // null without theirs
    float* part;                 // [parts][2][D]
    GnPlan plan;
};

hipError_t launch_gnorm_forward(const GnArgs& p, hipStream_t stream);
hipError_t launch_gnorm_backward(const GnArgs& p, hipStream_t stream);
// By token type, each in a translation unit of its own.
hipError_t launch_gnorm_backward_bf16(const GnArgs& p, hipStream_t stream);
hipError_t launch_gnorm_backward_f32(const GnArgs& p, hipStream_t stream);

}  // namespace wkv7
