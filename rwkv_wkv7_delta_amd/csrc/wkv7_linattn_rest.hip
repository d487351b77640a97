// wkv7_linattn_rest.hip -- zeros in the places of packed tokens that no row has.
//
// Rows lie one behind the other, so these are the tokens before the first start and those
// from the last one on; where they end is known on the device alone.  Two contiguous ranges
// of every tensor; where there are none (the usual call) a launch that writes nothing, 3.7 us.

#include "wkv7.h"

#include "wkv7_linattn_internal.h"

namespace wkv7 {

namespace {

constexpr int kThreads = 256, kGroups = 256;

struct RestArgs {
    int B;
    int64_t tokens;
    const int32_t* starts;
    char* wide[3];          // rows of whole 16-byte pieces; null: not wanted
    int64_t wide_bytes[3];  // of a row
    uint16_t* dg;           // rows of dg_halves 16-bit words
    int64_t dg_halves;
};

__global__ __launch_bounds__(kThreads) void la_rest_kernel(const RestArgs p) {
    typedef uint32_t Piece __attribute__((ext_vector_type(4)));
    const auto place = [&](int64_t x) { return x < 0 ? 0 : x > p.tokens ? p.tokens : x; };
    const int64_t head = place(p.starts[0]), last = place(p.starts[p.B]), tail = last < head ? head : last;
    const int64_t me = (int64_t)blockIdx.x * kThreads + threadIdx.x, all = (int64_t)kGroups * kThreads;
    for (int half = 0; half < 2; ++half) {
        const int64_t from = half ? tail : 0, n = half ? p.tokens - tail : head;
        for (int i = 0; i < 3; ++i) {
            if (!p.wide[i]) continue;
            Piece* const to = reinterpret_cast<Piece*>(p.wide[i] + from * p.wide_bytes[i]);
            for (int64_t c = me; c < n * (p.wide_bytes[i] / 16); c += all) to[c] = Piece{0, 0, 0, 0};
        }
        if (p.dg)
            for (int64_t c = me; c < n * p.dg_halves; c += all) p.dg[from * p.dg_halves + c] = 0;
    }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

}  // namespace wkv7

extern "C" int wkv7_linattn_clear_rest(const wkv7_linattn_desc* desc, const int32_t* starts, void* values, void* queries,
                                       void* keys, void* decays, void* stream) {
    using namespace wkv7;
    const int st = la_check(desc);
    if (st != WKV7_OK) return st;
    if (!desc->packed || !starts || !aligned(starts, 4)) return WKV7_ERR_INVALID_ARG;
    for (const void* x : {values, queries, keys, decays})
        if (!aligned(x, 16)) return WKV7_ERR_INVALID_ARG;
    if (desc->tokens == 0 || !(values || queries || keys || decays)) return WKV7_OK;
    const int64_t e = desc->dtype == WKV7_BF16 ? 2 : 4;
    RestArgs a{};
    a.B = desc->B;
    a.tokens = desc->tokens;
    a.starts = starts;
    a.wide[0] = static_cast<char*>(values);
    a.wide_bytes[0] = (int64_t)desc->H * desc->P * e;
    a.wide[1] = static_cast<char*>(queries);
    a.wide[2] = static_cast<char*>(keys);
    a.wide_bytes[1] = a.wide_bytes[2] = (int64_t)desc->G * desc->N * e;
    a.dg = static_cast<uint16_t*>(decays);
    a.dg_halves = desc->H * e / 2;
    la_rest_kernel<<<kGroups, kThreads, 0, static_cast<hipStream_t>(stream)>>>(a);
    return hipGetLastError() == hipSuccess ? WKV7_OK : WKV7_ERR_LAUNCH;
}
