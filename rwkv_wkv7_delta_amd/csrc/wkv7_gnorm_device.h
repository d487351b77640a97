// wkv7_gnorm_device.h -- rows, pieces and sums of the group norm kernels.
//
// Per row and group of W channels:
//   u = x, or x z sigmoid(z)
//   n = (u - mean u) / sqrt(mean (u - mean u)^2 + eps), or u / sqrt(mean u^2 + eps)
//   o = gamma n + beta,   y = o, or o sigmoid(o), and then perhaps times z sigmoid(z)
// Sums and moments are fp32, the deviations formed before they are squared.
//
// Bound by HBM: a group's values stay in registers between the sums and the result,
// so each tensor is read once.  P lanes take a group, K pieces of V channels each; a
// workgroup takes as many groups (of one or several rows) as make it full, always the
// same channels, so that gamma, beta and the sums of their gradients stay where they
// are over the rows.  32768 rows of 40 groups of 64 with a gate behind, bf16: 101 us,
// 5.0 TB/s (a copy of 1 GiB reaches 5.1).
#pragma once

#include "wkv7_gnorm_internal.h"
#include "wkv7_ssm_device.h"

namespace wkv7 {

// Sum over the P lanes that share a group: part of a wave, or (P > 64) several waves.
template <int P>
__device__ __forceinline__ float gn_sum(float x, float* lds) {
    if constexpr (P <= 16) {
        return group_sum<P>(x);
    } else if constexpr (P == 32) {
        x = row16_sum(x);
        return x + __shfl_xor(x, 16);
    } else {
        x = sum_rows4(row16_sum(x));
        if constexpr (P > 64) {
            __syncthreads();   // the sum before has been read
            if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
            __syncthreads();
            x = 0.f;
#pragma unroll
            for (int i = 0; i < P / 64; ++i) x += lds[threadIdx.x / P * (P / 64) + i];
        }
        return x;
    }
}

// V channels as loaded, or zeros.
template <typename T, int V>
struct GnPiece {
    static constexpr int kWords = (V * (int)sizeof(T) + 3) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p, bool in) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
        if (in) {
            if constexpr (sizeof(T) * V == 2) w[0] = *reinterpret_cast<const uint16_t*>(p);
            else if constexpr (sizeof(T) * V == 4) w[0] = *reinterpret_cast<const uint32_t*>(p);
            else {
                const uint4 u = *reinterpret_cast<const uint4*>(p);
                w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
            }
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return i % 2 == 0 ? bf16_lo(w[i / 2]) : bf16_hi(w[i / 2]);
    }
};

template <int V>
__device__ __forceinline__ void gn_vector(const float* p, bool in, float fill, float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = fill;
    if (p && in) {
        if constexpr (V % 4 == 0) load_cols<V>(p, x);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = p[i];
    }
}

__device__ __forceinline__ float silu(float z) { return z * sigmoid(z); }

// Where a thread stands: its group's lane, group and row among those side by side.
template <int P>
struct GnPlace {
    int lane, group, row, side;
    bool live;
    __device__ __forceinline__ GnPlace(const GnArgs& p) {
        const int slot = threadIdx.x / P;
        lane = threadIdx.x % P;
        row = slot / p.plan.groups;
        const int first = (int)(blockIdx.x % p.plan.blocks) * p.plan.groups;
        group = first + slot % p.plan.groups;
        side = (int)(blockIdx.x / p.plan.blocks) * p.plan.rows + row;
        live = row < p.plan.rows && group < p.G;
        group = group < p.G ? group : p.G - 1;
    }
};

}  // namespace wkv7
