// wkv7_linattn_internal.h -- launcher interface of linear attention with one
// decay per head (contracts in include/wkv7.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "wkv7.h"

namespace wkv7 {

// The descriptor's status: WKV7_OK or why a call with it is refused.
int la_check(const wkv7_linattn_desc* d);

constexpr int kLaChunk = 64;   // tokens of a tile and of a checkpoint

// Value rows of the state that one workgroup takes.
inline int la_value_block(int P) { return P < 64 ? P : 64; }

struct LaArgs {
    int B, T, H, G, N, P;
    bool bf16, fixed, packed;
    float scale;
    int64_t tokens;             // packed: tokens of the tensors
    const int32_t* rows;        // lengths [B] (may be null), packed: starts [B + 1]
    const void *q, *k, *v, *g;
    const float* s0;            // may be null
    void* y;
    float* sT;                  // may be null
    void* ckpt;                 // may be null
    // Time segments (nseg = 1: none) of seg_len tokens, a multiple of 64; what
    // each but the last leaves from a zero state, [nseg - 1][B][H][P][N], then
    // the state behind it, and its summed decay (log2), [nseg - 1][B][H].
    int nseg, seg_len;
    float* seg_state;
    double* seg_decay;
};

struct LaBwdArgs {
    LaArgs f;                   // the forward's inputs; f.ckpt is read
    const void* dy;
    const float* dsT;           // may be null
    void *dq, *dk, *dv, *dg;    // dg null with constant decays
    float* ds0;                 // may be null
    void* adj;                  // gradient of the state behind every tile, laid out as the checkpoints (bf16: pack_adjoint)
    // Parts of <S, D> of every tile and head, fp32 [tiles][H][value blocks][4]; null without dg.
    float* both;
    // Heads of a group in `split` parts (1: none), each with its own partial sums
    // of dq and dk, fp32 [split][tokens][G][N] both.
    int split;
    float *part_q, *part_k;
};

struct LaStepArgs {
    int B, H, G, N, P;
    bool bf16, fixed;
    float scale;
    const int32_t* slots;       // may be null: state b of row b
    int nslots;
    const void *q, *k, *v, *g;
    float* state;
    void* y;
};

hipError_t launch_la_forward(const LaArgs& p, hipStream_t stream);
hipError_t launch_la_backward(const LaBwdArgs& p, hipStream_t stream);
hipError_t launch_la_step(const LaStepArgs& p, hipStream_t stream);
// The reverse sweep of the backward: dS behind every tile, and ds0.
hipError_t launch_la_adjoint(const LaBwdArgs& p, hipStream_t stream);

}  // namespace wkv7
