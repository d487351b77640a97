// wkv7_slots_internal.h -- launcher interface of the slots of a cache (contracts in
// include/wkv7.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace wkv7 {

struct SlotsArgs {
    int planes, slots, from_slots, n;
    int64_t bytes;               // of a row
    const int32_t *src, *dst;    // a copy's pairs
    const void* from;            // the cache that is read
    void* pool;
    // A compaction:
    const uint8_t* keep;
    int32_t *moved, *count;
    bool clear;
    int32_t* pairs;              // scratch: [2 slots + 1] sources, targets, their number
};

hipError_t launch_slots_copy(const SlotsArgs& p, hipStream_t stream);
hipError_t launch_slots_compact(const SlotsArgs& p, hipStream_t stream);

}  // namespace wkv7
