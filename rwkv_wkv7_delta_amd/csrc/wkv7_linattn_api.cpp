// wkv7_linattn_api.cpp -- C ABI of linear attention with one decay per head:
// validation, segment plans, workspace layout, dispatch.  Contracts in include/wkv7.h.

#include "wkv7.h"

#include <hip/hip_runtime.h>

#include "wkv7_linattn_internal.h"

namespace {

using wkv7::kLaChunk;

constexpr int kUnits = 256;   // compute units of the device

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool req(const void* p) { return p != nullptr && aligned(p, 16); }
bool opt(const void* p) { return p == nullptr || aligned(p, 16); }

int from_hip(hipError_t e) { return e == hipSuccess ? WKV7_OK : WKV7_ERR_LAUNCH; }

// a b c d <= limit; every partial product is checked, so nothing wraps.
bool product_fits(int64_t a, int64_t b, int64_t c, int64_t d, int64_t limit) {
    if (a == 0 || b == 0 || c == 0 || d == 0) return true;
    return a <= limit / b && a * b <= limit / c && a * b * c <= limit / d;
}

bool size_ok(int32_t n) { return n == 32 || n == 64 || n == 128; }

int64_t blocks_of(int64_t T) { return (T + kLaChunk - 1) / kLaChunk; }
// Tiles of all rows, at most, and the rows of the checkpoint tensor.
int64_t tiles_of(const wkv7_linattn_desc* d) {
    return d->packed ? (int64_t)d->tokens / kLaChunk + d->B : (int64_t)d->B * blocks_of(d->T);
}
int64_t tokens_of(const wkv7_linattn_desc* d) { return d->packed ? d->tokens : (int64_t)d->B * d->T; }
// Tokens of a row that a launch is laid out for: no packed row has more than there are, and work
// laid out for a model's whole context would be units and segments without tokens.
int32_t longest(const wkv7_linattn_desc* d) { return d->packed && d->T > d->tokens ? d->tokens : d->T; }

int check(const wkv7_linattn_desc* d) { return wkv7::la_check(d); }

struct Plan {
    int nseg, seg_len;
};
// Time segments.  A launch without them has one workgroup per row, head and 64 value rows,
// which takes its tiles one after the other: where the workgroups are fewer than the compute
// units, as many segments as fill them, if that is worth a first sweep over the states and
// two more launches.  In tenths of a microsecond, measured where memory is not the limit: a
// tile takes 20 (fp32 45) read out, 17 (25) in the reverse sweep, which leaves its state (25
// and 43 at N = 128), and 12 (20) in a sweep over states alone, the launches 150.
// (1, 16384) tokens and 12 heads of 64 in bf16: 20 segments 57 us, 43 of them 67, 11 of them
// 82; (4, 1024) tokens, 12 heads: forward in 5 segments 24 us, without 34, and the gradients
// with their reverse sweep in 5 segments 42, without 48.
Plan plan(const wkv7_linattn_desc* d, bool read_out) {
    const int64_t wgs = (int64_t)d->B * d->H * (d->P / wkv7::la_value_block(d->P)), tiles = blocks_of(longest(d));
    const Plan none{1, (int)(tiles * kLaChunk)};
    if (wgs == 0 || tiles < 2) return none;
    int64_t n = kUnits / wgs;   // (one more, and some units have two: 37 us where 21 segments take 32)
    if (n > tiles) n = tiles;
    if (n < 2) return none;
    const int64_t each = (tiles + n - 1) / n;
    n = (tiles + each - 1) / each;
    const bool bf16 = d->dtype == WKV7_BF16, wide = d->N == 128;
    const int64_t sweep = bf16 ? 12 : 20, turn = read_out ? (bf16 ? 20 : 45) : bf16 ? (wide ? 25 : 17) : wide ? 43 : 25;
    if (n < 2 || each * (sweep + turn) + 150 >= tiles * turn) return none;
    return Plan{(int)n, (int)(each * kLaChunk)};
}

// Parts that a group's heads are taken in, so that the tiles alone need not fill the device.
int plan_split(const wkv7_linattn_desc* d) {
    const int64_t wgs = tiles_of(d) * d->G, shared = d->H / d->G;
    if (wgs == 0) return 1;
    int64_t n = 2 * kUnits / wgs;
    if (n > shared) n = shared;
    if (n < 2) return 1;
    const int64_t per = (shared + n - 1) / n;
    return (int)((shared + per - 1) / per);
}

size_t pad16(size_t bytes) { return (bytes + 15) / 16 * 16; }
size_t state_bytes(const wkv7_linattn_desc* d) { return (size_t)d->B * d->H * d->P * d->N * 4; }
size_t segment_bytes(const wkv7_linattn_desc* d, const Plan& s) {
    return (size_t)(s.nseg - 1) * (state_bytes(d) + pad16((size_t)d->B * d->H * 8));
}
size_t ckpt_bytes(const wkv7_linattn_desc* d) {
    if (tokens_of(d) == 0) return 0;
    return (size_t)tiles_of(d) * d->H * d->P * d->N * (d->dtype == WKV7_BF16 ? 2 : 4);
}
size_t both_bytes(const wkv7_linattn_desc* d) {
    if (d->fixed_decay || tokens_of(d) == 0) return 0;
    return (size_t)tiles_of(d) * d->H * (d->P / wkv7::la_value_block(d->P)) * 16;
}
size_t part_bytes(const wkv7_linattn_desc* d, int split) {
    return split > 1 ? (size_t)split * tokens_of(d) * d->G * d->N * 4 : 0;
}

wkv7::LaArgs args(const wkv7_linattn_desc* d, const int32_t* rows, const void* q, const void* k, const void* v,
                  const void* g, const float* s0, void* y, float* sT, void* ckpt, const Plan& s, void* seg) {
    char* const at = static_cast<char*>(seg);
    return wkv7::LaArgs{d->B, longest(d), d->H, d->G, d->N, d->P, d->dtype == WKV7_BF16, d->fixed_decay != 0,
                        d->packed != 0, d->scale, d->tokens, rows, q, k, v, g, s0, y, sT, ckpt, s.nseg, s.seg_len,
                        reinterpret_cast<float*>(at),
                        reinterpret_cast<double*>(at ? at + (size_t)(s.nseg - 1) * state_bytes(d) : nullptr)};
}

bool rows_ok(const wkv7_linattn_desc* d, const int32_t* rows) {
    return aligned(rows, 4) && (rows != nullptr || d->packed == 0);
}

}  // namespace

namespace wkv7 {
int la_check(const wkv7_linattn_desc* d) {
    if (!d) return WKV7_ERR_INVALID_ARG;
    if (d->B < 0 || d->T < 0 || d->H < 0 || d->G < 1 || d->H % d->G != 0 || d->tokens < 0)
        return WKV7_ERR_INVALID_ARG;
    if ((d->packed != 0 && d->packed != 1) || (d->fixed_decay != 0 && d->fixed_decay != 1))
        return WKV7_ERR_INVALID_ARG;
    if (!(d->scale - d->scale == 0.f)) return WKV7_ERR_INVALID_ARG;   // not finite
    if (!size_ok(d->N) || !size_ok(d->P)) return WKV7_ERR_UNSUPPORTED;
    if (d->dtype != WKV7_F32 && d->dtype != WKV7_BF16) return WKV7_ERR_UNSUPPORTED;
    // 64 token rows stay below 2^31 bytes, every grid at or below 2^31 threads.
    if (d->T > INT32_MAX - 64 || d->tokens > INT32_MAX - 64 || (int64_t)d->H * d->P > (1 << 22) ||
        (int64_t)d->G * d->N > (1 << 22))
        return WKV7_ERR_UNSUPPORTED;
    if (!product_fits(d->B, d->H, 4, 1, 1 << 23) || !product_fits(d->B, d->H, d->P, d->N, (int64_t)1 << 32) ||
        !product_fits(d->B, blocks_of(d->T), d->G, 1, 1 << 23) ||
        !product_fits(tiles_of(d), (int64_t)d->H * d->P, d->N, 1, (int64_t)1 << 40) ||
        !product_fits(tokens_of(d), (int64_t)d->H * d->P, 1, 1, (int64_t)1 << 40))
        return WKV7_ERR_UNSUPPORTED;
    return WKV7_OK;
}
}  // namespace wkv7

extern "C" {

size_t wkv7_linattn_ckpt_bytes(const wkv7_linattn_desc* desc) { return check(desc) == WKV7_OK ? ckpt_bytes(desc) : 0; }

size_t wkv7_linattn_forward_workspace_bytes(const wkv7_linattn_desc* desc) {
    if (check(desc) != WKV7_OK) return 0;
    return segment_bytes(desc, plan(desc, true));
}

size_t wkv7_linattn_backward_workspace_bytes(const wkv7_linattn_desc* desc) {
    if (check(desc) != WKV7_OK) return 0;
    return pad16(ckpt_bytes(desc)) + both_bytes(desc) + segment_bytes(desc, plan(desc, false)) +
           2 * part_bytes(desc, plan_split(desc));
}

int wkv7_linattn_forward(const wkv7_linattn_desc* desc, const int32_t* rows, const void* q, const void* k,
                         const void* v, const void* g, const float* s0, void* y, float* sT, void* ckpt,
                         void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check(desc);
    if (st != WKV7_OK) return st;
    if ((int64_t)desc->B * desc->H == 0) return WKV7_OK;
    const bool tokens = tokens_of(desc) > 0;
    if (!rows_ok(desc, rows) || (tokens && !(req(q) && req(k) && req(v) && req(g) && req(y))) ||
        !(opt(q) && opt(k) && opt(v) && opt(g) && opt(y) && opt(s0) && opt(sT) && opt(ckpt) && opt(workspace)))
        return WKV7_ERR_INVALID_ARG;
    const Plan s = plan(desc, true);
    const size_t need = segment_bytes(desc, s);
    if (need > 0 && (!workspace || workspace_bytes < need)) return WKV7_ERR_WORKSPACE;
    if (!tokens && !sT) return WKV7_OK;
    return from_hip(wkv7::launch_la_forward(args(desc, rows, q, k, v, g, s0, y, sT, ckpt, s, workspace),
                                            static_cast<hipStream_t>(stream)));
}

int wkv7_linattn_backward(const wkv7_linattn_desc* desc, const int32_t* rows, const void* q, const void* k,
                          const void* v, const void* g, const void* dy, const float* dsT, const void* ckpt, void* dq,
                          void* dk, void* dv, void* dg, float* ds0, void* workspace, size_t workspace_bytes,
                          void* stream) {
    const int st = check(desc);
    if (st != WKV7_OK) return st;
    if ((int64_t)desc->B * desc->H == 0) return WKV7_OK;
    const bool tokens = tokens_of(desc) > 0;
    if (!rows_ok(desc, rows) ||
        (tokens && !(req(q) && req(k) && req(v) && req(g) && req(dy) && req(ckpt) && req(dq) && req(dk) && req(dv) &&
                     (desc->fixed_decay ? dg == nullptr : req(dg)))) ||
        !(opt(q) && opt(k) && opt(v) && opt(g) && opt(dy) && opt(ckpt) && opt(dq) && opt(dk) && opt(dv) && opt(dg) &&
          opt(dsT) && opt(ds0) && opt(workspace)))
        return WKV7_ERR_INVALID_ARG;
    const Plan s = plan(desc, false);
    const int split = plan_split(desc);
    const size_t need = wkv7_linattn_backward_workspace_bytes(desc);
    if (need > 0 && (!workspace || workspace_bytes < need)) return WKV7_ERR_WORKSPACE;
    char* const adj = static_cast<char*>(workspace);
    char* const both = adj + pad16(ckpt_bytes(desc));
    char* const seg = both + both_bytes(desc);
    char* const part = seg + segment_bytes(desc, s);
    const wkv7::LaBwdArgs a{args(desc, rows, q, k, v, g, nullptr, nullptr, nullptr, const_cast<void*>(ckpt), s, seg),
                            dy, dsT, dq, dk, dv, dg, ds0, adj,
                            both_bytes(desc) ? reinterpret_cast<float*>(both) : nullptr, split, reinterpret_cast<float*>(part),
                            reinterpret_cast<float*>(part + part_bytes(desc, split))};
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    if (!tokens) return ds0 ? from_hip(wkv7::launch_la_adjoint(a, hs)) : WKV7_OK;
    return from_hip(wkv7::launch_la_backward(a, hs));
}

int wkv7_linattn_step(const wkv7_linattn_desc* desc, const int32_t* slots, int32_t nslots, const void* q,
                      const void* k, const void* v, const void* g, float* state, void* y, void* stream) {
    const int st = check(desc);
    if (st != WKV7_OK) return st;
    if (desc->packed || nslots < 0 || (!slots && nslots < desc->B)) return WKV7_ERR_INVALID_ARG;
    if (slots && desc->B > 65536) return WKV7_ERR_UNSUPPORTED;   // (a row looks through those before it)
    if ((int64_t)desc->B * desc->H == 0) return WKV7_OK;
    // (a cache without slots has no memory: no row's slot exists)
    if (!aligned(slots, 4) || !(req(q) && req(k) && req(v) && req(g) && req(y) && (nslots > 0 ? req(state) : opt(state))))
        return WKV7_ERR_INVALID_ARG;
    return from_hip(wkv7::launch_la_step(
        wkv7::LaStepArgs{desc->B, desc->H, desc->G, desc->N, desc->P, desc->dtype == WKV7_BF16,
                         desc->fixed_decay != 0, desc->scale, slots, nslots, q, k, v, g, state, y},
        static_cast<hipStream_t>(stream)));
}

}  // extern "C"
