// wkv7_ssm_api.cpp -- C ABI of the selective scan and the short causal
// convolution: validation, segment plans, workspace layout, dispatch.
// Contracts in include/wkv7.h.

#include "wkv7.h"

#include <hip/hip_runtime.h>

#include "wkv7_ssm_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool req(const void* p) { return p != nullptr && aligned(p, 16); }
bool opt(const void* p) { return p == nullptr || aligned(p, 16); }
// Given exactly when `with` is.
bool both(const void* p, const void* with) { return with ? req(p) : p == nullptr; }

int from_hip(hipError_t e) { return e == hipSuccess ? WKV7_OK : WKV7_ERR_LAUNCH; }

// Element counts that the size arithmetic and the launch grids hold: every
// partial product is checked, so nothing wraps.
bool product_fits(int64_t a, int64_t b, int64_t c, int64_t d, int64_t limit) {
    if (a == 0 || b == 0 || c == 0 || d == 0) return true;
    return a <= limit / b && a * b <= limit / c && a * b * c <= limit / d;
}

// ---- the convolution -----------------------------------------------------------

int check_conv(const wkv7_conv_desc* d) {
    if (!d) return WKV7_ERR_INVALID_ARG;
    if (d->B < 0 || d->T < 0 || d->D < 0) return WKV7_ERR_INVALID_ARG;
    if (d->silu != 0 && d->silu != 1) return WKV7_ERR_INVALID_ARG;
    if (d->W < 2 || d->W > 4) return WKV7_ERR_UNSUPPORTED;
    if (d->dtype != WKV7_F32 && d->dtype != WKV7_BF16) return WKV7_ERR_UNSUPPORTED;
    if (d->T > INT32_MAX - 1024 || d->D > (1 << 19)) return WKV7_ERR_UNSUPPORTED;   // 520 fp32 rows below 2^31 bytes
    // Below that no launch has more than 2^31 threads (a row of few channels takes a
    // wave all the same).
    if (!product_fits(d->B, (int64_t)d->T + 64, d->D < 64 ? 64 : d->D, 1, (int64_t)1 << 35) ||
        !product_fits(d->B, d->D, 4, 1, (int64_t)1 << 31))
        return WKV7_ERR_UNSUPPORTED;
    return WKV7_OK;
}

// Runs of the gradient: the sums over a run's tokens stay in registers and
// leave as one partial row, and a run steps W - 1 tokens past its end, so runs
// are as long as still leaves about kConvWaves waves of 64 column pieces; a
// multiple of 4 from 16 to 512 tokens.  A run is addressed with 32-bit byte
// offsets (D is limited for that).
constexpr int kConvWaves = 2048;
constexpr int kConvPiece = 4;   // channels of a gradient lane

struct ConvPlan {
    int run, parts;
};
ConvPlan plan_conv(const wkv7_conv_desc* d) {
    const int64_t piece = 64 * (d->D % kConvPiece == 0 ? kConvPiece : 1);
    const int64_t waves = ((int64_t)d->D + piece - 1) / piece * d->B;   // per run
    int64_t runs = waves > 0 ? kConvWaves / waves : 1;
    if (runs < 1) runs = 1;
    int64_t run = (((int64_t)d->T + runs - 1) / runs + 3) / 4 * 4;
    run = run < 16 ? 16 : run > 512 ? 512 : run;
    const int64_t all = ((int64_t)d->T + run - 1) / run * d->B;
    int64_t parts = (all + 3) / 4;
    if (parts < 1) parts = 1;
    return ConvPlan{(int)run, (int)parts};
}

wkv7::ConvArgs conv_args(const wkv7_conv_desc* d, const float* weight, const float* bias,
                         const int32_t* lengths, const void* x, const void* s0, void* y, void* sT) {
    return wkv7::ConvArgs{d->B, d->T, d->D, d->W, d->dtype == WKV7_BF16, d->silu != 0,
                          weight, bias, lengths, x, s0, y, sT};
}

// ---- the scan ------------------------------------------------------------------

int64_t channel_blocks(const wkv7_ssm_desc* d, bool backward) {
    const int ch = backward ? wkv7::ssm_bwd_channels(d->N) : wkv7::ssm_channels(d->N);
    return ((int64_t)d->D / d->G + ch - 1) / ch;
}

// Bytes by which a token moves the widest of the buffers that a segment's
// workgroup walks: fp32 tokens, fp32 checkpoints (every 16 tokens), partial sums.
int64_t token_bytes(const wkv7_ssm_desc* d) {
    const int64_t tok = (int64_t)d->D * (d->N / 4 > 4 ? d->N / 4 : 4), bc = (int64_t)d->G * d->N * 8;
    return tok > bc ? tok : bc;
}

// Time segments: a launch without them has one workgroup per batch row, group
// and channel block.  The first of the two launches repeats most of the
// exponentials, so a split only pays when it shortens the chain enough: three
// segments at least (two leave half the chain to each launch: an estimate, not
// measured; where one workgroup per unit is the aim, 86 to 128 of them leave units
// idle), of 64 tokens at least, as many as make one or two workgroups per compute unit.  Two at N = 16, and in the backward at N = 32, whose workgroups
// run two at a time (forward and backward at B = 4, T = 1024, D = 768, N = 16: one,
// two, four per unit 159, 104, 111 us; forward at B = 1, T = 16384, D = 768 95, 93,
// 98 us; backward at B = 2, T = 1024, D = 512, N = 32 53, 49, 52 us); one elsewhere,
// where more only add first launches' work (B = 3, T = 1024, D = 1024, N = 8: forward
// 25, 30, 30 us, backward 44, 50, 53; B = 1, T = 2048, D = 512, N = 64: 37, 42, 64 and
// 83, 87, 110; forward at N = 32 21.5, 24, 24).  At most 64: B = 1, T = 16384, D = 768
// with 32 at most took 116 us where 64 took 95.
struct SsmPlan {
    int nseg, seg_len;
};
constexpr int kMaxSegments = 64;
constexpr int kMinSegmentTokens = 64;

SsmPlan plan_ssm(const wkv7_ssm_desc* d, bool backward) {
    const SsmPlan none{1, d->T};
    const int64_t wgs = (int64_t)d->B * d->G * channel_blocks(d, backward);
    if (wgs == 0 || d->T == 0) return none;
    int64_t n = (d->N == 16 || (backward && d->N == 32) ? 2 : 1) * wkv7::kUnits / wgs;
    if (n > d->T / kMinSegmentTokens) n = d->T / kMinSegmentTokens;
    if (n > kMaxSegments) n = kMaxSegments;
    if (n < 3) n = 1;
    // No buffer of a segment, nor the eight tiles behind it, reaches 2^31 bytes.
    const int64_t most = ((int64_t)INT32_MAX / token_bytes(d) - 128) / 16 * 16;
    const int64_t least = most >= 16 ? (d->T + most - 1) / most : d->T;
    if (n < least) n = least;
    if (n < 2) return none;
    const int64_t len = (((int64_t)d->T + n - 1) / n + 15) / 16 * 16;
    n = ((int64_t)d->T + len - 1) / len;
    return SsmPlan{(int)n, (int)len};
}

int check_ssm(const wkv7_ssm_desc* d) {
    if (!d) return WKV7_ERR_INVALID_ARG;
    if (d->B < 0 || d->T < 0 || d->D < 0 || d->G < 1 || d->D % d->G != 0) return WKV7_ERR_INVALID_ARG;
    if (d->N != 8 && d->N != 16 && d->N != 32 && d->N != 64) return WKV7_ERR_UNSUPPORTED;
    if (d->dtype != WKV7_F32 && d->dtype != WKV7_BF16) return WKV7_ERR_UNSUPPORTED;
    if (d->ckpt_bits != 0 && d->ckpt_bits != 8 && d->ckpt_bits != 32) return WKV7_ERR_UNSUPPORTED;
    // A segment's rows are addressed with 32-bit byte offsets that move up to six
    // tiles past its end (token_bytes): no tile of 16 tokens has more than 2^28 bytes.
    if (d->T > INT32_MAX - 64 || d->D > (1 << 22) || (int64_t)d->D * d->N > (1 << 26) ||
        (int64_t)d->G * d->N > (1 << 21))
        return WKV7_ERR_UNSUPPORTED;
    const int64_t blocks = ((int64_t)d->T + 15) / 16, most = (int64_t)1 << 40;
    if (!product_fits(d->B, d->T, d->D, 1, most) || !product_fits(d->B, blocks, d->D, d->N, most) ||
        !product_fits(d->B, d->T, d->G, d->N, (int64_t)1 << 32) ||
        !product_fits(d->B, d->D, 64, 1, (int64_t)1 << 31))
        return WKV7_ERR_UNSUPPORTED;
    // A launch of 512 threads per workgroup stays at or below 2^31.
    for (const bool backward : {false, true})
        if (!product_fits(d->B, d->G, channel_blocks(d, backward), plan_ssm(d, backward).nseg, 1 << 22))
            return WKV7_ERR_UNSUPPORTED;
    return WKV7_OK;
}

size_t pad4(size_t floats) { return (floats + 3) / 4 * 4; }

// Floats of the segments' states and step sums.
size_t segment_floats(const wkv7_ssm_desc* d, const SsmPlan& s) {
    const size_t bd = (size_t)d->B * d->D;
    return (size_t)(s.nseg - 1) * bd * d->N + pad4((size_t)(s.nseg - 1) * bd);
}
// Floats of the backward's partial sums of dB and dC, dA, and the vectors.
size_t part_bc_floats(const wkv7_ssm_desc* d) {
    const int64_t blocks = channel_blocks(d, true);
    return blocks > 1 ? (size_t)blocks * d->B * d->T * d->G * 2 * d->N : 0;
}
size_t part_a_floats(const wkv7_ssm_desc* d, const SsmPlan& s) { return (size_t)s.nseg * d->B * d->D * d->N; }
size_t part_v_floats(const wkv7_ssm_desc* d, const SsmPlan& s) {
    return pad4((size_t)s.nseg * d->B * d->D * 2);
}
size_t backward_floats(const wkv7_ssm_desc* d, const SsmPlan& s) {
    return part_bc_floats(d) + part_a_floats(d, s) + part_v_floats(d, s) + segment_floats(d, s);
}

size_t ckpt_bytes(const wkv7_ssm_desc* d) {
    const size_t rows = (size_t)d->B * (((size_t)d->T + 15) / 16) * d->D, codes = rows * d->N;
    if (d->ckpt_bits == 0 || codes == 0) return 0;
    return d->ckpt_bits == 32 ? codes * 4 : (codes + 15) / 16 * 16 + rows * 4;
}

int check_params(const wkv7_ssm_params* p) {
    if (!p || !req(p->A) || !opt(p->dskip) || !opt(p->dt_bias) || !aligned(p->lengths, 4) ||
        (p->softplus != 0 && p->softplus != 1))
        return WKV7_ERR_INVALID_ARG;
    return WKV7_OK;
}

wkv7::SsmArgs ssm_args(const wkv7_ssm_desc* d, const wkv7_ssm_params* p, const void* x, const void* dt,
                       const void* Bm, const void* Cm, const void* z, const float* h0, void* y,
                       float* hT, void* ckpt, const SsmPlan& s, float* seg) {
    return wkv7::SsmArgs{d->B, d->T, d->D, d->N, d->G, d->dtype == WKV7_BF16, p->softplus != 0,
                         d->ckpt_bits, p->A, p->dskip, p->dt_bias, p->lengths, x, dt, Bm, Cm, z, h0, y,
                         hT, ckpt, s.nseg, s.seg_len, seg,
                         seg ? seg + (size_t)(s.nseg - 1) * d->B * d->D * d->N : nullptr};
}

}  // namespace

extern "C" {

int wkv7_conv_forward(const wkv7_conv_desc* desc, const float* weight, const float* bias,
                      const int32_t* lengths, const void* x, const void* s0, void* y, void* sT,
                      void* stream) {
    const int st = check_conv(desc);
    if (st != WKV7_OK) return st;
    if ((int64_t)desc->B * desc->D == 0) return WKV7_OK;
    const bool tokens = desc->T > 0;
    if (!req(weight) || !opt(bias) || !aligned(lengths, 4) || (tokens && !(req(x) && req(y))) ||
        !(opt(x) && opt(y) && opt(s0) && opt(sT)))
        return WKV7_ERR_INVALID_ARG;
    return from_hip(wkv7::launch_conv_forward(conv_args(desc, weight, bias, lengths, x, s0, y, sT),
                                              static_cast<hipStream_t>(stream)));
}

size_t wkv7_conv_backward_workspace_bytes(const wkv7_conv_desc* desc) {
    if (check_conv(desc) != WKV7_OK) return 0;
    return (size_t)plan_conv(desc).parts * desc->D * (desc->W + 1) * sizeof(float);
}

int wkv7_conv_backward(const wkv7_conv_desc* desc, const float* weight, const float* bias,
                       const int32_t* lengths, const void* x, const void* s0, const void* dy,
                       const void* dsT, void* dx, float* dweight, float* dbias, void* ds0,
                       void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_conv(desc);
    if (st != WKV7_OK) return st;
    if (desc->D == 0) return WKV7_OK;
    const bool tokens = (int64_t)desc->B * desc->T > 0;
    if (!req(weight) || !opt(bias) || !aligned(lengths, 4) || (tokens && !(req(x) && req(dy) && req(dx))) ||
        !(opt(x) && opt(dy) && opt(dx) && opt(s0) && opt(dsT) && opt(ds0) && opt(workspace)) ||
        !req(dweight) || !both(dbias, bias))
        return WKV7_ERR_INVALID_ARG;
    const ConvPlan plan = plan_conv(desc);
    if (!workspace || workspace_bytes < wkv7_conv_backward_workspace_bytes(desc)) return WKV7_ERR_WORKSPACE;
    const wkv7::ConvBwdArgs q{conv_args(desc, weight, bias, lengths, x, s0, nullptr, nullptr), dy, dsT, dx, ds0,
                              dweight, dbias, static_cast<float*>(workspace), plan.parts, plan.run};
    return from_hip(wkv7::launch_conv_backward(q, static_cast<hipStream_t>(stream)));
}

int wkv7_conv_step(const wkv7_conv_desc* desc, const float* weight, const float* bias, const void* x,
                   void* state, void* y, void* stream) {
    const int st = check_conv(desc);
    if (st != WKV7_OK) return st;
    if ((int64_t)desc->B * desc->D == 0) return WKV7_OK;
    if (!req(weight) || !opt(bias) || !req(x) || !req(state) || !req(y)) return WKV7_ERR_INVALID_ARG;
    return from_hip(wkv7::launch_conv_step(conv_args(desc, weight, bias, nullptr, x, nullptr, y, state),
                                           static_cast<hipStream_t>(stream)));
}

size_t wkv7_ssm_ckpt_bytes(const wkv7_ssm_desc* desc) {
    return check_ssm(desc) == WKV7_OK ? ckpt_bytes(desc) : 0;
}

size_t wkv7_ssm_forward_workspace_bytes(const wkv7_ssm_desc* desc) {
    if (check_ssm(desc) != WKV7_OK) return 0;
    const SsmPlan s = plan_ssm(desc, false);
    return s.nseg > 1 ? segment_floats(desc, s) * sizeof(float) : 0;
}

size_t wkv7_ssm_backward_workspace_bytes(const wkv7_ssm_desc* desc) {
    if (check_ssm(desc) != WKV7_OK) return 0;
    return backward_floats(desc, plan_ssm(desc, true)) * sizeof(float);
}

int wkv7_ssm_forward(const wkv7_ssm_desc* desc, const wkv7_ssm_params* params, const void* x,
                     const void* dt, const void* Bm, const void* Cm, const void* z, const float* h0,
                     void* y, float* hT, void* ckpt, void* workspace, size_t workspace_bytes,
                     void* stream) {
    int st = check_ssm(desc);
    if (st != WKV7_OK) return st;
    if ((int64_t)desc->B * desc->D == 0) return WKV7_OK;
    if ((st = check_params(params)) != WKV7_OK) return st;
    const bool tokens = desc->T > 0;
    if ((tokens && !(req(x) && req(dt) && req(Bm) && req(Cm) && req(y))) ||
        !(opt(x) && opt(dt) && opt(Bm) && opt(Cm) && opt(y) && opt(z) && opt(h0) && opt(hT) && opt(ckpt) &&
          opt(workspace)) ||
        (tokens && (ckpt != nullptr) != (desc->ckpt_bits != 0)))
        return WKV7_ERR_INVALID_ARG;
    const SsmPlan s = plan_ssm(desc, false);
    const size_t need = s.nseg > 1 ? segment_floats(desc, s) * sizeof(float) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return WKV7_ERR_WORKSPACE;
    if (!tokens && !hT) return WKV7_OK;
    return from_hip(wkv7::launch_ssm_forward(
        ssm_args(desc, params, x, dt, Bm, Cm, z, h0, y, hT, ckpt, s, static_cast<float*>(workspace)),
        static_cast<hipStream_t>(stream)));
}

int wkv7_ssm_backward(const wkv7_ssm_desc* desc, const wkv7_ssm_params* params, const void* x,
                      const void* dt, const void* Bm, const void* Cm, const void* z, const void* dy,
                      const float* dhT, const void* ckpt, const wkv7_ssm_grads* grads, void* workspace,
                      size_t workspace_bytes, void* stream) {
    int st = check_ssm(desc);
    if (st != WKV7_OK) return st;
    if (desc->ckpt_bits == 0) return WKV7_ERR_UNSUPPORTED;
    if (desc->D == 0) return WKV7_OK;
    if ((st = check_params(params)) != WKV7_OK) return st;
    if (!grads) return WKV7_ERR_INVALID_ARG;
    const bool tokens = (int64_t)desc->B * desc->T > 0;
    if ((tokens && !(req(x) && req(dt) && req(Bm) && req(Cm) && req(dy) && req(ckpt) && req(grads->dx) &&
                     req(grads->ddt) && req(grads->dBm) && req(grads->dCm) && both(grads->dz, z))) ||
        !(opt(z) && opt(dhT) && opt(grads->dh0) && opt(workspace)) || !req(grads->dA) ||
        !both(grads->ddskip, params->dskip) || !both(grads->ddt_bias, params->dt_bias))
        return WKV7_ERR_INVALID_ARG;
    const SsmPlan s = plan_ssm(desc, true);
    const size_t need = backward_floats(desc, s) * sizeof(float);
    if (need > 0 && (!workspace || workspace_bytes < need)) return WKV7_ERR_WORKSPACE;
    float* const bc = static_cast<float*>(workspace);
    float* const pa = bc + part_bc_floats(desc);
    float* const pv = pa + part_a_floats(desc, s);
    float* const seg = pv + part_v_floats(desc, s);
    const wkv7::SsmBwdArgs q{
        ssm_args(desc, params, x, dt, Bm, Cm, z, nullptr, nullptr, nullptr, const_cast<void*>(ckpt), s, seg),
        dy, dhT, grads->dx, grads->ddt, grads->dBm, grads->dCm, grads->dz, grads->dA, grads->ddskip,
        grads->ddt_bias, grads->dh0, part_bc_floats(desc) ? bc : nullptr, pa, pv};
    return from_hip(wkv7::launch_ssm_backward(q, static_cast<hipStream_t>(stream)));
}

int wkv7_ssm_step(const wkv7_ssm_desc* desc, const wkv7_ssm_params* params, const void* x, const void* dt,
                  const void* Bm, const void* Cm, const void* z, float* state, void* y, void* stream) {
    int st = check_ssm(desc);
    if (st != WKV7_OK) return st;
    if ((int64_t)desc->B * desc->D == 0) return WKV7_OK;
    if ((st = check_params(params)) != WKV7_OK) return st;
    if (params->lengths || !(req(x) && req(dt) && req(Bm) && req(Cm) && opt(z) && req(state) && req(y)))
        return WKV7_ERR_INVALID_ARG;
    return from_hip(wkv7::launch_ssm_step(
        ssm_args(desc, params, x, dt, Bm, Cm, z, nullptr, y, state, nullptr, SsmPlan{1, 1}, nullptr),
        static_cast<hipStream_t>(stream)));
}

}  // extern "C"
