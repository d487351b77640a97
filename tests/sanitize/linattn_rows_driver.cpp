// Launches of linear attention for packed rows whose longest length is overstated: stub launchers
// check that they are laid out for the tokens there are.
#include <cstdio>

#include "wkv7.h"
#include "wkv7_linattn_internal.h"

static long failed = 0, launches = 0;
static void check(bool ok, const char* what, int64_t a, int64_t b) {
    if (ok) return;
    ++failed;
    std::printf("failed: %s (%lld, %lld)\n", what, (long long)a, (long long)b);
}

namespace wkv7 {
static void rows(const LaArgs& p) {
    ++launches;
    check(p.T <= p.tokens, "laid out for tokens that are not there", p.T, p.tokens);
    check(p.nseg <= (p.tokens + kLaChunk - 1) / kLaChunk || p.nseg == 1, "segments without tokens", p.nseg, p.tokens);
}
hipError_t launch_la_forward(const LaArgs& p, hipStream_t) {
    rows(p);
    return hipSuccess;
}
hipError_t launch_la_adjoint(const LaBwdArgs& q, hipStream_t) {
    rows(q.f);
    return hipSuccess;
}
hipError_t launch_la_backward(const LaBwdArgs& q, hipStream_t) {
    rows(q.f);
    const LaArgs& p = q.f;
    // as the launch counts them, in 32 bits
    const int64_t units = (int64_t)p.B * ((p.T + 63) / 64) * p.G * q.split;
    check(units > 0 && units < (int64_t)1 << 32, "units of the gradients' launch", units, q.split);
    return hipSuccess;
}
hipError_t launch_la_step(const LaStepArgs&, hipStream_t) { return hipSuccess; }
}  // namespace wkv7

int main() {
    void* const f = reinterpret_cast<void*>((uintptr_t)1 << 20);
    float* const ff = static_cast<float*>(f);
    const int32_t* const fi = static_cast<const int32_t*>(f);
    for (int32_t T : {1, 64, 777, 1 << 17, 1 << 24, 1 << 29})
        for (int32_t tokens : {1, 63, 64, 777, 1 << 16, 1 << 20})
            for (int32_t H : {1, 12, 512, 32768}) {
                const wkv7_linattn_desc d = {1, T, H, 1, 64, 64, WKV7_BF16, 0, 1, tokens, 1.f};
                const size_t forward = wkv7_linattn_forward_workspace_bytes(&d), backward = wkv7_linattn_backward_workspace_bytes(&d);
                const int a = wkv7_linattn_forward(&d, fi, f, f, f, f, ff, f, ff, f, f, forward, nullptr);
                const int b = wkv7_linattn_backward(&d, fi, f, f, f, f, f, ff, f, f, f, f, f, ff, f, backward, nullptr);
                const int want = (int64_t)(tokens / 64 + 1) * H * 64 * 64 > (int64_t)1 << 40 ? WKV7_ERR_UNSUPPORTED : WKV7_OK;
                check(a == want && b == want, "statuses", a, b);
            }
    std::printf("%ld launches, %ld failed checks\n", launches, failed);
    return failed != 0;
}
