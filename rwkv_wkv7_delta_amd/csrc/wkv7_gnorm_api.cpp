// wkv7_gnorm_api.cpp -- C ABI of the group norm: validation, launch plans, dispatch.
// Contracts in include/wkv7.h.

#include "wkv7.h"

#include <hip/hip_runtime.h>

#include "wkv7_gnorm_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool req(const void* p) { return p != nullptr && aligned(p, 16); }
bool opt(const void* p) { return p == nullptr || aligned(p, 16); }
bool both(const void* p, const void* with) { return with ? req(p) : p == nullptr; }

int from_hip(hipError_t e) { return e == hipSuccess ? WKV7_OK : WKV7_ERR_LAUNCH; }

int check(const wkv7_gnorm_desc* d) {
    if (!d) return WKV7_ERR_INVALID_ARG;
    if (d->rows < 0 || d->D < 0 || d->G < 1 || d->D % d->G != 0) return WKV7_ERR_INVALID_ARG;
    if ((d->center != 0 && d->center != 1) || (d->silu != 0 && d->silu != 1)) return WKV7_ERR_INVALID_ARG;
    if (d->gate < WKV7_GATE_NONE || d->gate > WKV7_GATE_BEFORE) return WKV7_ERR_INVALID_ARG;
    if (!(d->eps >= 0.f) || !(d->eps - d->eps == 0.f)) return WKV7_ERR_INVALID_ARG;
    if (d->dtype != WKV7_F32 && d->dtype != WKV7_BF16) return WKV7_ERR_UNSUPPORTED;
    if (d->D > (1 << 22) || (d->D > 0 && d->rows > ((int64_t)1 << 40) / d->D)) return WKV7_ERR_UNSUPPORTED;
    return WKV7_OK;
}

// Channels per access: 16 bytes where a group is made of them, for bf16 also pairs.
// Lanes: as few (4 to 64) as hold a group in one piece each, then 64 to 512 with two
// (four took more registers than there are in the backward).  As many groups side by side as 512 threads hold, of
// several rows if a row has fewer.  Forward about 8192 workgroups; backward 512, each going
// over as many rows as that leaves: each leaves a partial row of the sums for gamma and
// beta (2048, a partial row for each row side by side: 318 us where 512 take 100, (16384, 2048)
// in bf16).
wkv7::GnPlan plan(const wkv7_gnorm_desc* d, bool backward) {
    wkv7::GnPlan p;
    const int W = d->D / d->G, widest = d->dtype == WKV7_BF16 ? 8 : 4;
    p.vec = W % widest == 0 ? widest : d->dtype == WKV7_BF16 && W % 2 == 0 ? 2 : 1;
    const int pieces = (W + p.vec - 1) / p.vec;
    p.each = 1;
    p.lanes = pieces <= 4 ? 4 : pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : 64;
    if (pieces > 64) {
        p.each = pieces <= 1024 ? 2 : 0;
        p.lanes = pieces <= 128 ? 64 : pieces <= 256 ? 128 : pieces <= 512 || p.each == 0 ? 256 : 512;
    }
    const int64_t slots = p.each == 0 ? 1 : 512 / p.lanes;
    p.blocks = (unsigned)((d->G + slots - 1) / slots);
    p.groups = (int)((d->G + p.blocks - 1) / p.blocks);
    p.rows = (int)(slots / p.groups);
    if (p.rows < 1 || p.each == 0) p.rows = 1;
    // a few rows: no more side by side than there are
    if (p.rows > d->rows) p.rows = d->rows > 0 ? (int)d->rows : 1;
    p.threads = (p.groups * p.rows * p.lanes + 63) / 64 * 64;
    int64_t parts = ((backward ? 512 : 8192) + p.blocks - 1) / p.blocks;
    const int64_t most = (d->rows + p.rows - 1) / p.rows;
    if (parts > most) parts = most;
    p.parts = (unsigned)(parts < 1 ? 1 : parts);
    return p;
}

wkv7::GnArgs args(const wkv7_gnorm_desc* d, const float* gamma, const float* beta, const void* x, const void* z,
                  bool backward) {
    wkv7::GnArgs a{};
    a.rows = d->rows;
    a.D = d->D;
    a.G = d->G;
    a.W = d->D / d->G;
    a.bf16 = d->dtype == WKV7_BF16;
    a.center = d->center != 0;
    a.silu = d->silu != 0;
    a.gate = d->gate;
    a.eps = d->eps;
    a.gamma = gamma;
    a.beta = beta;
    a.x = x;
    a.z = z;
    a.plan = plan(d, backward);
    return a;
}

}  // namespace

extern "C" {

int wkv7_gnorm_forward(const wkv7_gnorm_desc* desc, const float* gamma, const float* beta, const void* x,
                       const void* z, void* y, void* stream) {
    const int st = check(desc);
    if (st != WKV7_OK) return st;
    if (desc->rows == 0 || desc->D == 0) return WKV7_OK;
    if (!req(x) || !req(y) || !opt(gamma) || !opt(beta) || (desc->gate != 0) != (z != nullptr) || !opt(z))
        return WKV7_ERR_INVALID_ARG;
    wkv7::GnArgs a = args(desc, gamma, beta, x, z, false);
    a.y = y;
    return from_hip(wkv7::launch_gnorm_forward(a, static_cast<hipStream_t>(stream)));
}

size_t wkv7_gnorm_backward_workspace_bytes(const wkv7_gnorm_desc* desc) {
    if (check(desc) != WKV7_OK || desc->rows == 0 || desc->D == 0) return 0;
    const wkv7::GnPlan p = plan(desc, true);
    return (size_t)p.parts * 2 * desc->D * sizeof(float);
}

int wkv7_gnorm_backward(const wkv7_gnorm_desc* desc, const float* gamma, const float* beta, const void* x,
                        const void* z, const void* dy, void* dx, void* dz, float* dgamma, float* dbeta,
                        void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check(desc);
    if (st != WKV7_OK) return st;
    if (desc->D == 0) return WKV7_OK;
    const bool some = desc->rows > 0;
    if ((some && !(req(x) && req(dy) && req(dx) && (desc->gate != 0) == (z != nullptr) && both(dz, z))) ||
        !(opt(x) && opt(z) && opt(dy) && opt(dx) && opt(dz) && opt(gamma) && opt(beta) && opt(workspace)) ||
        !both(dgamma, gamma) || !both(dbeta, beta))
        return WKV7_ERR_INVALID_ARG;
    const bool sums = gamma || beta;
    if (!some && !sums) return WKV7_OK;
    if (some && sums && (!workspace || workspace_bytes < wkv7_gnorm_backward_workspace_bytes(desc)))
        return WKV7_ERR_WORKSPACE;
    wkv7::GnArgs a = args(desc, gamma, beta, x, z, true);
    a.dy = dy;
    a.dx = dx;
    a.dz = dz;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    if (!some) {
        // Nothing to sum: the sums' launch writes zeros, whatever the workspace.
        a.part = dgamma ? dgamma : dbeta;
    }
    return from_hip(wkv7::launch_gnorm_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
