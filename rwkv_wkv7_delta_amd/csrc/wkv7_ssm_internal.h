// wkv7_ssm_internal.h -- launcher interface of the selective scan and the short
// causal convolution (contracts in include/wkv7.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace wkv7 {

constexpr int kUnits = 256;        // compute units of the device
constexpr int kSsmChunk = 16;      // tokens per state checkpoint and per kernel tile
constexpr int kSsmThreads = 256;   // lanes that hold a scan workgroup's states
constexpr int kSsmStates = 4;      // states of a channel per lane (forward)

// Channels that one workgroup takes: of the forward (four states per lane) and of
// the backward (two, at N = 64 four).
inline int ssm_channels(int N) { return kSsmThreads * kSsmStates / N; }
inline int ssm_bwd_channels(int N) { return kSsmThreads * (N == 64 ? 4 : 2) / N; }

struct SsmArgs {
    int B, T, D, N, G;
    bool bf16, softplus;
    int ckpt_bits;              // 0, 8 or 32
    const float *A, *dskip, *dt_bias;   // dskip, dt_bias may be null
    const int32_t* lengths;     // may be null
    const void *x, *dt, *Bm, *Cm, *z;   // z may be null
    const float* h0;            // may be null
    void* y;
    float* hT;                  // may be null (the step: the state, in place)
    void* ckpt;                 // null when ckpt_bits = 0
    // Time segments (nseg = 1: none) of seg_len tokens, a multiple of 16; the
    // states that segments 0 .. nseg-2 leave from zero, [nseg-1][B][D][N], and
    // the sums of their steps, [nseg-1][B][D].
    int nseg, seg_len;
    float *seg_h, *seg_d;
};

struct SsmBwdArgs {
    SsmArgs f;                  // the forward's inputs; f.ckpt is read
    const void* dy;
    const float* dhT;           // may be null
    void *dx, *ddt, *dBm, *dCm, *dz;     // dz null without z
    float *dA, *ddskip, *ddt_bias, *dh0; // ddskip, ddt_bias null without theirs; dh0 may be null
    // Partial sums: dB and dC per channel block of a group, [blocks][B][T][G][2N]
    // (null with one block per group: written straight to dBm, dCm); dA and the
    // two vectors per (batch row, segment), [B * nseg][D][N] and [B * nseg][D][2].
    float *part_bc, *part_a, *part_v;
};

hipError_t launch_ssm_forward(const SsmArgs& p, hipStream_t stream);
hipError_t launch_ssm_backward(const SsmBwdArgs& p, hipStream_t stream);
hipError_t launch_ssm_step(const SsmArgs& p, hipStream_t stream);

struct ConvArgs {
    int B, T, D, W;
    bool bf16, silu;
    const float *weight, *bias;   // bias may be null
    const int32_t* lengths;       // may be null
    const void *x, *s0;           // s0 may be null
    void *y, *sT;                 // sT may be null (the step: the state, in place)
};

struct ConvBwdArgs {
    ConvArgs f;
    const void *dy, *dsT;         // dsT may be null
    void *dx, *ds0;               // ds0 may be null
    float *dweight, *dbias;       // dbias null without a bias
    float* part;                  // [parts][D][W + 1] partial sums
    int parts, run;               // runs of `run` tokens, parts of four runs
};

hipError_t launch_conv_forward(const ConvArgs& p, hipStream_t stream);
hipError_t launch_conv_backward(const ConvBwdArgs& p, hipStream_t stream);
hipError_t launch_conv_step(const ConvArgs& p, hipStream_t stream);

}  // namespace wkv7
