// The C ABI layers of linear attention, the group norm and the slots on descriptors up to the
// integer limits, with stub launchers that check what a launch would rely on.
#include <cstdio>
#include <vector>

#include "wkv7.h"
#include "wkv7_gnorm_internal.h"
#include "wkv7_linattn_internal.h"
#include "wkv7_slots_internal.h"

static long failed = 0, launches = 0;
static void check(bool ok, const char* what) {
    if (!ok) {
        ++failed;
        std::printf("failed: %s\n", what);
    }
}
constexpr int64_t kThreads = (int64_t)1 << 31;   // of a launch

namespace wkv7 {
static void segments(const LaArgs& p) {
    ++launches;
    const int64_t wgs = (int64_t)p.B * p.H * (p.P / la_value_block(p.P));
    check(p.nseg >= 1 && wgs * p.nseg * 512 <= kThreads, "segment threads");
    check(p.nseg == 1 || (p.seg_len % kLaChunk == 0 && p.seg_len > 0 && p.seg_state && p.seg_decay), "segments");
    check(p.nseg == 1 || ((int64_t)(p.nseg - 1) * p.seg_len < p.T && (int64_t)p.nseg * p.seg_len >= p.T), "segments cover T");
    check((int64_t)p.B * p.H * p.P * p.N / 4 <= kThreads, "join threads");
    for (const int64_t row : {(int64_t)p.H * p.P, (int64_t)p.G * p.N}) check(64 * row * 4 < (int64_t)1 << 31, "a tile's buffer");
}
hipError_t launch_la_forward(const LaArgs& p, hipStream_t) {
    segments(p);
    return hipSuccess;
}
hipError_t launch_la_adjoint(const LaBwdArgs& q, hipStream_t) {
    segments(q.f);
    return hipSuccess;
}
hipError_t launch_la_backward(const LaBwdArgs& q, hipStream_t) {
    segments(q.f);
    const LaArgs& p = q.f;
    const int64_t units = (int64_t)p.B * ((p.T + 63) / 64) * p.G * q.split;
    check(q.split >= 1 && q.split <= p.H / p.G && units < (int64_t)1 << 31, "units");
    const int per = (p.H / p.G + q.split - 1) / q.split;
    check((q.split - 1) * per < p.H / p.G && q.split * per >= p.H / p.G, "parts of the heads");
    if (q.split > 1) {
        const int64_t values = (p.packed ? p.tokens : (int64_t)p.B * p.T) * p.G * p.N;
        check(2 * (values / 4 + 256) <= kThreads && q.part_q && q.part_k > q.part_q, "threads of the parts' sums");
        check(q.part_k - q.part_q == q.split * values, "the parts' layout");
    }
    return hipSuccess;
}
hipError_t launch_la_step(const LaStepArgs& p, hipStream_t) {
    ++launches;
    check((int64_t)p.B * p.H * ((p.P * p.N + 4095) / 4096) * 256 <= kThreads, "step threads");
    return hipSuccess;
}
static hipError_t gnorm(const GnArgs& p) {
    ++launches;
    const GnPlan& g = p.plan;
    check(g.threads >= 64 && g.threads <= 512 && g.threads >= g.lanes * g.groups * g.rows, "norm threads");
    check((int64_t)g.blocks * g.groups >= p.G && g.rows >= 1 && g.parts >= 1, "groups covered");
    check(g.each == 0 || (int64_t)g.lanes * g.each * g.vec >= p.W, "a group's channels");
    check(p.W % g.vec == 0, "whole pieces");
    check((int64_t)g.blocks * g.parts * 512 <= kThreads, "norm grid");
    return hipSuccess;
}
hipError_t launch_gnorm_forward(const GnArgs& p, hipStream_t) { return gnorm(p); }
hipError_t launch_gnorm_backward(const GnArgs& p, hipStream_t) { return gnorm(p); }
static hipError_t slots(const SlotsArgs& p, int64_t rows) {
    ++launches;
    check(((p.bytes + 15) / 16 + 1023) / 1024 * p.planes * rows * 256 <= kThreads, "slots threads");
    return hipSuccess;
}
hipError_t launch_slots_copy(const SlotsArgs& p, hipStream_t) { return slots(p, p.n); }
hipError_t launch_slots_compact(const SlotsArgs& p, hipStream_t) { return slots(p, p.slots); }
}  // namespace wkv7

int main() {
    const std::vector<int32_t> sizes = {-1, 0, 1, 3, 63, 64, 65, 1000, 16384, 70000, 1 << 20, 1 << 23, 1 << 28,
                                        INT32_MAX - 64, INT32_MAX};
    void* const f = reinterpret_cast<void*>((uintptr_t)1 << 20);
    float* const ff = static_cast<float*>(f);
    const int32_t* const fi = static_cast<const int32_t*>(f);
    const size_t ws = SIZE_MAX;
    long refused = 0;
    auto tally = [&](int st, const char* what) {
        check(st == WKV7_OK || st == WKV7_ERR_INVALID_ARG || st == WKV7_ERR_UNSUPPORTED, what);
        refused += st != WKV7_OK;
    };
    for (int32_t B : sizes)
        for (int32_t T : sizes)
            for (int32_t H : {0, 1, 6, 32, 256, 1 << 15, 1 << 20, INT32_MAX})
                for (int32_t G : {1, 2, 256, INT32_MAX})
                    for (int32_t N : {32, 128})
                        for (int32_t P : {32, 64, 128, 1 << 30})
                            for (int32_t tokens : {-1, 0, 777, INT32_MAX - 64}) {
                                const wkv7_linattn_desc d = {B, T, H, G, N, P, P == 32 ? WKV7_F32 : WKV7_BF16, 0,
                                                             tokens >= 0, tokens < 0 ? 0 : tokens, 1.f};
                                wkv7_linattn_ckpt_bytes(&d);
                                wkv7_linattn_forward_workspace_bytes(&d);
                                wkv7_linattn_backward_workspace_bytes(&d);
                                tally(wkv7_linattn_forward(&d, fi, f, f, f, f, ff, f, ff, f, f, ws, nullptr), "forward");
                                tally(wkv7_linattn_backward(&d, fi, f, f, f, f, f, ff, f, f, f, f, f, ff, f, ws, nullptr),
                                      "backward");
                                tally(wkv7_linattn_step(&d, fi, 1 << 20, f, f, f, f, ff, f, nullptr), "step");
                            }
    for (int64_t rows : {(int64_t)-1, (int64_t)0, (int64_t)1, (int64_t)1000, (int64_t)1 << 30, (int64_t)1 << 40, INT64_MAX})
        for (int32_t D : {-1, 0, 1, 7, 64, 1001, 2560, 8192, 8200, 16390, 70000, 1 << 22, INT32_MAX})
            for (int32_t G : {0, 1, 7, 8, 40, 1 << 20})
                for (int32_t dtype : {WKV7_F32, WKV7_BF16}) {
                    const wkv7_gnorm_desc d = {rows, D, G, dtype, 1, 0, WKV7_GATE_NONE, 0.f};
                    wkv7_gnorm_backward_workspace_bytes(&d);
                    tally(wkv7_gnorm_forward(&d, ff, ff, f, nullptr, f, nullptr), "norm forward");
                    tally(wkv7_gnorm_backward(&d, ff, ff, f, nullptr, f, f, nullptr, ff, ff, f, ws, nullptr), "norm backward");
                }
    uint8_t* const keep = static_cast<uint8_t*>(f);
    int32_t* const out = static_cast<int32_t*>(f);
    for (int32_t planes : sizes)
        for (int32_t n : sizes)
            for (int64_t row : {(int64_t)-1, (int64_t)0, (int64_t)1, (int64_t)30, (int64_t)64, (int64_t)1 << 20,
                                ((int64_t)1 << 33) + 1, (int64_t)1 << 40, INT64_MAX}) {
                tally(wkv7_slots_copy(planes, 1 << 20, row, n, fi, fi, f, 1 << 20, f, nullptr), "copy");
                tally(wkv7_slots_compact(planes, n, row, keep, out, out, 1, f, f, ws, nullptr), "compact");
            }
    std::printf("%ld launches, %ld refused, %ld failed checks\n", launches, refused, failed);
    return failed != 0;
}
