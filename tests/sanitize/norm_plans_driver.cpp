// How often a workgroup of the group norm goes over its rows: for each "rows D G dtype backward"
// of the command line, the number of passes, and whether the last one is not full.
#include <cstdio>
#include <cstdlib>

#include "wkv7.h"
#include "wkv7_gnorm_internal.h"

namespace wkv7 {
static hipError_t show(const GnArgs& p) {
    // a wide group's workgroup takes one row at a time
    const int64_t at_once = (int64_t)p.plan.parts * (p.plan.each == 0 ? 1 : p.plan.rows);
    std::printf("%lld %d\n", (long long)((p.rows + at_once - 1) / at_once), p.rows % at_once != 0);
    return hipSuccess;
}
hipError_t launch_gnorm_forward(const GnArgs& p, hipStream_t) { return show(p); }
hipError_t launch_gnorm_backward(const GnArgs& p, hipStream_t) { return show(p); }
}  // namespace wkv7

int main(int argc, char** argv) {
    void* const f = reinterpret_cast<void*>((uintptr_t)1 << 20);
    float* const ff = static_cast<float*>(f);
    for (int i = 1; i + 4 < argc; i += 5) {
        const wkv7_gnorm_desc d = {std::atoll(argv[i]), std::atoi(argv[i + 1]), std::atoi(argv[i + 2]), std::atoi(argv[i + 3]),
                                   1, 0, WKV7_GATE_NONE, 0.f};
        const int st = std::atoi(argv[i + 4]) ? wkv7_gnorm_backward(&d, ff, ff, f, nullptr, f, f, nullptr, ff, ff, f, SIZE_MAX, nullptr)
                                              : wkv7_gnorm_forward(&d, ff, ff, f, nullptr, f, nullptr);
        if (st != WKV7_OK) return 1;
    }
    return 0;
}
