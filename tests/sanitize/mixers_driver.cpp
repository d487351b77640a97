// The C ABI layer of the convolution and the scan on descriptors up to the
// integer limits, with stub launchers that check what a launch would rely on.
#include <cstdio>
#include <vector>

#include "wkv7.h"
#include "wkv7_ssm_internal.h"

static long failed = 0, launches = 0;
static void check(bool ok, const char* what) {
    if (!ok) {
        ++failed;
        std::printf("failed: %s\n", what);
    }
}

namespace wkv7 {
hipError_t launch_conv_forward(const ConvArgs& p, hipStream_t) {
    ++launches;
    const int64_t runs = ((int64_t)p.T + 15) / 16;
    check(runs * p.D * p.B <= (int64_t)1 << 31, "forward run threads");
    check((int64_t)p.B * (p.W - 1) * p.D <= (int64_t)1 << 31, "state threads");
    return hipSuccess;
}
hipError_t launch_conv_step(const ConvArgs& p, hipStream_t) {
    ++launches;
    check((int64_t)p.B * p.D <= (int64_t)1 << 31, "step threads");
    return hipSuccess;
}
hipError_t launch_conv_backward(const ConvBwdArgs& q, hipStream_t) {
    ++launches;
    const int64_t piece = 64 * (q.f.D % 4 == 0 ? 4 : 1), cblocks = (q.f.D + piece - 1) / piece;
    check(cblocks * q.parts * 256 <= (int64_t)1 << 31, "gradient threads");
    check(q.run >= 16 && q.run % 4 == 0, "run length");
    check((int64_t)q.parts * 4 * q.run >= (int64_t)q.f.B * q.f.T, "parts cover the tokens");
    check(((int64_t)q.run + 8) * q.f.D * 4 < (int64_t)1 << 31, "a run's buffer");
    return hipSuccess;
}
static void scan(const SsmArgs& p, int channels) {
    ++launches;
    const int64_t wgs = (int64_t)p.B * p.G * ((p.D / p.G + channels - 1) / channels);
    check(p.nseg >= 1 && wgs * p.nseg * 512 <= (int64_t)1 << 31, "scan threads");
    if (p.nseg > 1) {
        check(p.seg_len % 16 == 0 && p.seg_len > 0, "segment length");
        check((int64_t)(p.nseg - 1) * p.seg_len < p.T && (int64_t)p.nseg * p.seg_len >= p.T, "segments cover the tokens");
    }
    if (wgs == 0) return;
    // Offsets move up to six tiles behind the segment and have to stay below 2^32.
    const int64_t tiles = ((int64_t)p.seg_len + 15) / 16, e = p.bf16 ? 2 : 4;
    for (const int64_t tile : {16 * e * p.D, 16 * e * p.G * p.N, 16 * 8 * (int64_t)p.G * p.N,
                               p.ckpt_bits ? 4 * (int64_t)p.D * p.N : 0}) {
        check(tiles * tile < (int64_t)1 << 31, "a segment's buffer");
        check((tiles + 6) * tile < (int64_t)1 << 31, "offsets behind a segment");
    }
}
hipError_t launch_ssm_forward(const SsmArgs& p, hipStream_t) {
    scan(p, ssm_channels(p.N));
    return hipSuccess;
}
hipError_t launch_ssm_step(const SsmArgs& p, hipStream_t) {
    ++launches;
    const int64_t ch = 256 * 4 / p.N;
    check((p.D + ch - 1) / ch * p.B * 256 <= (int64_t)1 << 32, "step threads");
    return hipSuccess;
}
hipError_t launch_ssm_backward(const SsmBwdArgs& q, hipStream_t) {
    scan(q.f, ssm_bwd_channels(q.f.N));
    const int64_t sums = (int64_t)q.f.B * q.f.T * q.f.G * q.f.N / 2 + (int64_t)q.f.D * (q.f.N + 2) + 512;
    check(sums <= (int64_t)1 << 32, "threads of the sums");
    return hipSuccess;
}
}  // namespace wkv7

int main() {
    const std::vector<int32_t> sizes = {-1, 0, 1, 2, 15, 16, 17, 64, 1000, 4096, 70000, 1 << 19, 1 << 20, 1 << 22,
                                        1 << 24, 1 << 28, INT32_MAX - 2000, INT32_MAX - 64, INT32_MAX};
    void* const f = reinterpret_cast<void*>((uintptr_t)1 << 20);
    float* const ff = static_cast<float*>(f);
    const size_t ws = SIZE_MAX;
    const wkv7_ssm_params prm = {ff, nullptr, nullptr, nullptr, 1};
    const wkv7_ssm_grads g = {f, f, f, f, nullptr, ff, nullptr, nullptr, ff};
    long refused = 0;
    auto tally = [&](int st, const char* what) {
        check(st == WKV7_OK || st == WKV7_ERR_INVALID_ARG || st == WKV7_ERR_UNSUPPORTED, what);
        refused += st != WKV7_OK;
    };
    for (int32_t B : sizes)
        for (int32_t T : sizes)
            for (int32_t D : sizes) {
                for (int32_t W = 1; W <= 5; ++W)
                    for (int32_t dtype = 0; dtype <= 2; ++dtype) {
                        const wkv7_conv_desc d = {B, T, D, W, dtype, 1};
                        wkv7_conv_backward_workspace_bytes(&d);
                        tally(wkv7_conv_forward(&d, ff, nullptr, nullptr, f, f, f, f, nullptr), "conv forward");
                        tally(wkv7_conv_backward(&d, ff, nullptr, nullptr, f, f, f, f, f, ff, nullptr, f, f, ws,
                                                 nullptr), "conv backward");
                        tally(wkv7_conv_step(&d, ff, nullptr, f, f, f, nullptr), "conv step");
                    }
                for (int32_t N : {8, 16, 32, 64, 65, 1 << 30})
                    for (int32_t G : {0, 1, 2, 64, 1 << 20, INT32_MAX})
                        for (int32_t bits : {8, 32}) {
                            const wkv7_ssm_desc d = {B, T, D, N, G, WKV7_F32, bits};
                            const bool ok = wkv7_ssm_backward_workspace_bytes(&d) > 0;
                            wkv7_ssm_forward_workspace_bytes(&d);
                            check(ok || wkv7_ssm_ckpt_bytes(&d) == 0, "a size of a refused descriptor");
                            tally(wkv7_ssm_forward(&d, &prm, f, f, f, f, nullptr, ff, f, ff, f, f, ws, nullptr),
                                  "scan forward");
                            tally(wkv7_ssm_backward(&d, &prm, f, f, f, f, nullptr, f, ff, f, &g, f, ws, nullptr),
                                  "scan backward");
                            tally(wkv7_ssm_step(&d, &prm, f, f, f, f, nullptr, ff, f, nullptr), "scan step");
                        }
            }
    std::printf("%ld launches, %ld refused, %ld failed checks\n", launches, refused, failed);
    return failed != 0;
}
