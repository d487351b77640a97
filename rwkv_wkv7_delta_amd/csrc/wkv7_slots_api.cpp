// wkv7_slots_api.cpp -- C ABI of the copies between the slots of a cache: validation,
// dispatch.  Contracts in include/wkv7.h.

#include "wkv7.h"

#include <hip/hip_runtime.h>

#include "wkv7_slots_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool req(const void* p, uintptr_t a) { return p != nullptr && aligned(p, a); }

int from_hip(hipError_t e) { return e == hipSuccess ? WKV7_OK : WKV7_ERR_LAUNCH; }

int check(int32_t planes, int32_t slots, int64_t row_bytes) {
    if (planes < 0 || slots < 0 || row_bytes < 0) return WKV7_ERR_INVALID_ARG;
    if (slots > (1 << 22) || planes > (1 << 20) || row_bytes > ((int64_t)1 << 40)) return WKV7_ERR_UNSUPPORTED;
    return WKV7_OK;
}
// At most 2^23 workgroups (of rows, planes and 1024 pieces of 16 bytes of a row).
bool grid_fits(int64_t rows, int32_t planes, int64_t row_bytes) {
    const int64_t parts = (row_bytes + 16383) / 16384;
    if (rows == 0 || planes == 0 || parts == 0) return true;
    return rows * planes <= ((int64_t)1 << 23) / parts;
}

}  // namespace

extern "C" {

int wkv7_slots_copy(int32_t planes, int32_t slots, int64_t row_bytes, int32_t n, const int32_t* src,
                    const int32_t* dst, const void* from, int32_t from_slots, void* pool, void* stream) {
    const int st = check(planes, slots, row_bytes);
    if (st != WKV7_OK) return st;
    if (n < 0 || from_slots < 0) return WKV7_ERR_INVALID_ARG;
    // (every workgroup looks through the whole list: 65536 pairs in 2^22 slots take 2.5 ms)
    if (from_slots > (1 << 22) || n > 65536 || !grid_fits(n, planes, row_bytes)) return WKV7_ERR_UNSUPPORTED;
    if (n == 0 || planes == 0 || row_bytes == 0 || slots == 0) return WKV7_OK;
    if (!req(src, 4) || !req(dst, 4) || !req(pool, 16) || !aligned(from, 16) || (!from && from_slots > 0) ||
        (from == pool && from_slots != slots))
        return WKV7_ERR_INVALID_ARG;
    wkv7::SlotsArgs a{};
    a.planes = planes;
    a.slots = slots;
    a.from_slots = from_slots;
    a.n = n;
    a.bytes = row_bytes;
    a.src = src;
    a.dst = dst;
    a.from = from;
    a.pool = pool;
    return from_hip(wkv7::launch_slots_copy(a, static_cast<hipStream_t>(stream)));
}

size_t wkv7_slots_compact_workspace_bytes(int32_t slots) {
    return slots < 0 || slots > (1 << 22) ? 0 : ((size_t)slots * 2 + 1) * sizeof(int32_t);
}

int wkv7_slots_compact(int32_t planes, int32_t slots, int64_t row_bytes, const uint8_t* keep, int32_t* moved,
                       int32_t* count, int32_t clear, void* pool, void* workspace, size_t workspace_bytes,
                       void* stream) {
    const int st = check(planes, slots, row_bytes);
    if (st != WKV7_OK) return st;
    if (clear != 0 && clear != 1) return WKV7_ERR_INVALID_ARG;
    if (!grid_fits(slots, planes, row_bytes)) return WKV7_ERR_UNSUPPORTED;
    const bool some = slots > 0;
    if (!req(count, 4) || (some && !(keep && req(moved, 4))) || !aligned(pool, 16) ||
        (some && planes > 0 && row_bytes > 0 && !pool) || !aligned(workspace, 4))
        return WKV7_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < wkv7_slots_compact_workspace_bytes(slots)) return WKV7_ERR_WORKSPACE;
    wkv7::SlotsArgs a{};
    a.planes = some ? planes : 0;
    a.slots = a.from_slots = slots;
    a.bytes = row_bytes;
    a.keep = keep;
    a.moved = moved;
    a.count = count;
    a.clear = clear != 0;
    a.pairs = static_cast<int32_t*>(workspace);
    a.from = a.pool = pool;
    return from_hip(wkv7::launch_slots_compact(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
