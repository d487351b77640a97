// wkv7_ssm_tile.h -- how the selective scan's kernels lay their work over a
// workgroup.
//
// A workgroup takes CH = 256 S / N channels of one group and one batch row and
// walks the tokens in tiles of 16.  Four step waves own the states: each of
// their sixteen 16-lane rows takes 16 channels (one per lane) and S of their N
// states, so a channel's states lie over P = N / S rows.  Four staging waves
// move everything else: they load the token rows two tiles ahead, form what
// depends on token and channel only, once, and leave it in LDS as fp32, read
// the partial sums that the step waves leave there, and store whole row pieces.
// One barrier per tile; both sides of every hand-over are double-buffered.
//
// With 16 channels on a row and 16 tokens in a tile, lane t of a row holds the
// row's S values of B and C for token t, and the products broadcast them by
// DPP (row_newbcast:t) as an operand: no LDS read per token for B and C, which
// otherwise (16 bytes per lane and token each) took more LDS time than the
// products themselves take on the vector ALU.
#pragma once

#include "wkv7_ssm_device.h"
#include "wkv7_ssm_internal.h"

namespace wkv7 {

constexpr int kTile = kSsmChunk;
constexpr int kStepThreads = 256;    // four step waves, then four staging waves

template <int N, int S>
struct Shape {
    static constexpr int P = N / S;                        // rows of 16 lanes per channel
    static constexpr int CH = kStepThreads * S / N;        // channels per workgroup
    static constexpr int EPT = CH / 16;                    // channels of a staging thread's piece
    static constexpr int BC = kTile * N / kStepThreads > 0 ? kTile * N / kStepThreads : 1;
    static constexpr int YS = CH + 16;                     // row stride of the partial sums
    static constexpr int HS = N + 4;                       // row stride of states in LDS
};

// Where a step lane stands: its channel in the workgroup, its first state, and
// the index of its group of states.
template <int N, int S>
struct StepLane {
    int cl, part, n0, t;   // t: the token whose B and C the lane holds
    __device__ __forceinline__ explicit StepLane(int tid) {
        const int row = tid / 16;
        t = tid % 16;
        cl = row / Shape<N, S>::P * 16 + t;
        part = row % Shape<N, S>::P;
        n0 = part * S;
    }
};

// The workgroup's place in the problem.  The device hands workgroups to its
// eight XCDs in turn; giving each XCD a run of consecutive places keeps
// neighbouring channel blocks, which share cache lines of the token rows and
// the rows of B and C, behind one L2.
struct Place {
    int j, g, b, seg;
    __device__ __forceinline__ Place(int blocks, int G, int B) {
        unsigned u = blockIdx.x;
        const unsigned n = gridDim.x, per = n / 8;
        if (u < per * 8) u = u % 8 * per + u / 8;
        j = u % blocks;
        u /= blocks;
        g = u % G;
        u /= G;
        b = u % B;
        seg = u / B;
    }
};

// The state h (S of a channel's) taken through `count` segments: h <- exp(A sum D) h
// + e each, e at e0 + k stride_e, sum D at d0 + k stride_d.  Eight segments' loads go
// out together: one by one their latencies add up.
template <int S>
__device__ __forceinline__ void through_segments(float (&h)[S], const float (&a2)[S], const float* e0, int64_t stride_e,
                                                 const float* d0, int64_t stride_d, int count) {
    for (int s = 0; s < count; s += 8) {
        float e[8][S], d[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int at = s + k < count ? s + k : count - 1;
            load_cols<S>(e0 + at * stride_e, e[k]);
            d[k] = d0[at * stride_d];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (s + k < count) {
#pragma unroll
                for (int n = 0; n < S; ++n) h[n] = fmaf(exp2_raw(d[k] * a2[n]), h[n], e[k][n]);
            }
        }
    }
}

// The value of lane `t` of the row in every lane of the row; folded into the
// multiply that uses it.
template <int t>
__device__ __forceinline__ float row_bcast(float x) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x150 + t, 0xF, 0xF, true));
}
// h <- a h + x on four states, and sum_n (c[n] broadcast from lane t) h[n]: the
// read-out's products take the broadcast as their DPP operand (the compiler
// would spend a move on each).  What the hardware leaves to the code here: an
// exponential's result may not be read by the very next vector instruction (the
// s_nop), and a DPP operand not have been written by the two vector instructions
// before (the two updates in front).  Updates and read-out alternate: a DPP sum
// that waits for the one before it takes 8 clocks instead of 4.
template <int t>
__device__ __forceinline__ float step_read(float (&h)[4], const float (&a)[4], const float (&x)[4],
                                           const float (&c)[4]) {
    float y;
    asm("s_nop 0\n\t"
        "v_fma_f32 %0, %5, %0, %9\n\t"
        "v_fma_f32 %1, %6, %1, %10\n\t"
        "v_mul_f32_dpp %4, %13, %0 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
        "v_fma_f32 %2, %7, %2, %11\n\t"
        "v_fmac_f32_dpp %4, %14, %1 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
        "v_fma_f32 %3, %8, %3, %12\n\t"
        "v_fmac_f32_dpp %4, %15, %2 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %4, %16, %3 row_newbcast:%17 row_mask:0xf bank_mask:0xf"
        : "+&v"(h[0]), "+&v"(h[1]), "+&v"(h[2]), "+&v"(h[3]), "=&v"(y)
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]),
          "v"(c[0]), "v"(c[1]), "v"(c[2]), "v"(c[3]), "n"(t));
    return y;
}

// f(integral_constant 0), ... f(15), or backwards: the token as a constant.
template <int t>
struct Tok {
    static constexpr int v = t;
};
template <typename F>
__device__ __forceinline__ void each_token(F&& f) {
    f(Tok<0>()); f(Tok<1>()); f(Tok<2>()); f(Tok<3>()); f(Tok<4>()); f(Tok<5>()); f(Tok<6>()); f(Tok<7>());
    f(Tok<8>()); f(Tok<9>()); f(Tok<10>()); f(Tok<11>()); f(Tok<12>()); f(Tok<13>()); f(Tok<14>()); f(Tok<15>());
}
template <typename F>
__device__ __forceinline__ void each_token_back(F&& f) {
    f(Tok<15>()); f(Tok<14>()); f(Tok<13>()); f(Tok<12>()); f(Tok<11>()); f(Tok<10>()); f(Tok<9>()); f(Tok<8>());
    f(Tok<7>()); f(Tok<6>()); f(Tok<5>()); f(Tok<4>()); f(Tok<3>()); f(Tok<2>()); f(Tok<1>()); f(Tok<0>());
}

}  // namespace wkv7
