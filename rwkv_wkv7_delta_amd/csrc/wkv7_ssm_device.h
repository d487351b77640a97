// wkv7_ssm_device.h -- device helpers of the selective scan and the short
// causal convolution.
#pragma once

#include "wkv7_device.h"

namespace wkv7 {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float exp_raw(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + exp_raw(-x));
}

// log(1 + exp(x)) = max(x, 0) + log(1 + e) with e = exp(-|x|) in (0, 1].  With
// u = fl(1 + e), log(1 + e) = log(u) + (e - (u - 1)) / u to second order in the
// rounding of u; u - 1 is exact, and the divisor is left out: the term is below
// 2^-24 where u is 1 or more, so that changes the sum by less than half a unit
// in its last place.  For e below 2^-24 the logarithm is 0 and the term is e.
__device__ __forceinline__ float softplus(float x) {
    const float e = exp_raw(-fabsf(x));
    const float u = 1.f + e;
    return fmaxf(x, 0.f) + fmaf(__builtin_amdgcn_logf(u), kLn2, e - (u - 1.f));
}

// ---- token rows ---------------------------------------------------------------
// Pieces of V consecutive elements, kept as loaded so that a prefetch does not
// wait for them.  kVec: whole pieces at their natural alignment; else element by
// element.
typedef uint32_t vu2 __attribute__((ext_vector_type(2)));
typedef uint32_t vu4 __attribute__((ext_vector_type(4)));

constexpr int kApart = 16;

template <typename T, int V, bool kVec>
struct Piece {
    static constexpr int kBytes = V * (int)sizeof(T);
    static constexpr int kWords = kVec ? (kBytes + 3) / 4 : V;
    uint32_t w[kWords];

    // From a row in memory (whole pieces only); c is a multiple of V.  Addresses at or
    // behind `lim` are clamped into the row.
    __device__ __forceinline__ void load(const T* row, int c, int lim) {
        static_assert(kVec, "element by element from buffers only");
        const T* p = row + (c < lim ? c : lim - V);
        if constexpr (kBytes == 2) {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (kBytes == 8) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            w[0] = u.x; w[1] = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
                w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
            }
        }
    }
    // At byte `at` of a buffer; what lies outside it reads as 0.  Without kVec the
    // elements are kApart elements apart: sixteen lanes' loads lie side by side.
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
        if constexpr (!kVec) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if constexpr (sizeof(T) == 4) w[i] = __builtin_amdgcn_raw_buffer_load_b32(r, at + 4 * kApart * i, 0, 0);
                else w[i] = __builtin_amdgcn_raw_buffer_load_b16(r, at + 2 * kApart * i, 0, 0);
            }
        } else if constexpr (kBytes == 2) {
            w[0] = __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
        } else if constexpr (kBytes == 4) {
            w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
        } else if constexpr (kBytes == 8) {
            const vu2 u = __builtin_bit_cast(vu2, __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0));
            w[0] = u.x; w[1] = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const vu4 u = __builtin_bit_cast(vu4, __builtin_amdgcn_raw_buffer_load_b128(r, at + 4 * i, 0, 0));
                w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else if constexpr (!kVec) return bf16_lo(w[i]);
        else return i % 2 == 0 ? bf16_lo(w[i / 2]) : bf16_hi(w[i / 2]);
    }
};

// Stored in a row unless c lies at or behind `lim`.
template <int V>
__device__ __forceinline__ void store_piece(float* row, int c, int lim, const float (&x)[V]) {
    if (c >= lim) return;
    if constexpr (V == 1) {
        row[c] = x[0];
    } else if constexpr (V == 2) {
        *reinterpret_cast<float2*>(row + c) = make_float2(x[0], x[1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4*>(row + c + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    }
}
template <int V>
__device__ __forceinline__ void store_piece(bf16_t* row, int c, int lim, const float (&x)[V]) {
    if (c >= lim) return;
    if constexpr (V == 1)
        row[c] = f2bf(x[0]);
    else if constexpr (V == 2)
        *reinterpret_cast<uint32_t*>(row + c) = pack_bf16x2(x[0], x[1]);
    else if constexpr (V == 4)
        *reinterpret_cast<uint2*>(row + c) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    else
        *reinterpret_cast<uint4*>(row + c) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                        pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// The same into a buffer, of the first `valid` elements (kVec: all or none);
// what lies outside the buffer is dropped.
constexpr uint32_t kNowhere = 0x7ffffff0u;   // behind the end of every buffer here

template <typename T, bool kVec, int V>
__device__ __forceinline__ void store_piece(__amdgpu_buffer_rsrc_t r, uint32_t at, int valid, const float (&x)[V]) {
    if constexpr (!kVec) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t o = i < valid ? at + i * kApart * (uint32_t)sizeof(T) : kNowhere;
            if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[i]), r, o, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b16(f2bf(x[i]), r, o, 0, 0);
        }
    } else {
        const uint32_t o = valid > 0 ? at : kNowhere;
        constexpr int kWords = V * (int)sizeof(T) / 4;
        if constexpr (kWords == 0) {
            __builtin_amdgcn_raw_buffer_store_b16(f2bf(x[0]), r, o, 0, 0);
        } else {
            uint32_t w[kWords];
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x[i]);
                else w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            }
            if constexpr (kWords == 1) {
                __builtin_amdgcn_raw_buffer_store_b32(w[0], r, o, 0, 0);
            } else if constexpr (kWords == 2) {
                const vu2 u = {w[0], w[1]};
                __builtin_amdgcn_raw_buffer_store_b64(u, r, o, 0, 0);
            } else {
#pragma unroll
                for (int i = 0; i < kWords; i += 4) {
                    const vu4 u = {w[i], w[i + 1], w[i + 2], w[i + 3]};
                    __builtin_amdgcn_raw_buffer_store_b128(u, r, o + 4 * i, 0, 0);
                }
            }
        }
    }
}

// `bytes` at p as a buffer (0: every access lies outside, nothing is touched).
// Both are the same in every lane; said so, or the compiler may keep them per
// lane and loop over the lanes at each access.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int bytes) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint64_t v = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(u >> 32)) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)u);
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(v), (short)0,
                                             __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

// Sum and maximum over each aligned group of P = 2, 4, 8 or 16 lanes, in every lane.
template <int P>
__device__ __forceinline__ float group_sum(float x) {
    if constexpr (P == 2) return x + __builtin_amdgcn_update_dpp(0.0f, x, 0xB1, 0xF, 0xF, false);
    else return lanes_sum<P>(x);
}
template <int P>
__device__ __forceinline__ float group_max(float x) {
    x = fmaxf(x, __builtin_amdgcn_update_dpp(0.0f, x, 0xB1, 0xF, 0xF, false));
    if (P >= 4) x = fmaxf(x, __builtin_amdgcn_update_dpp(0.0f, x, 0x4E, 0xF, 0xF, false));
    if (P >= 8) x = fmaxf(x, __builtin_amdgcn_update_dpp(0.0f, x, 0x141, 0xF, 0xF, false));
    if (P >= 16) x = fmaxf(x, __builtin_amdgcn_update_dpp(0.0f, x, 0x140, 0xF, 0xF, false));
    return x;
}

// Valid tokens of batch row b: lengths[b] clamped to [0, T], or T.
__device__ __forceinline__ int row_length(const int32_t* lengths, int b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : n > T ? T : n;
}

// ---- state checkpoints --------------------------------------------------------
// 32 bits: fp32 [B][blocks][D][N].  8 bits: int8 codes of the same shape, then,
// from a 16-byte boundary, fp32 scales [B][blocks][D]: one scale for the N
// states of a channel, its largest magnitude over 127, so a code is off by at
// most half a scale.  A row whose largest magnitude is below 1e-35 is stored as
// zeros; one that holds an infinity or a NaN gets a NaN scale, so what is read
// back is NaN and never plausible.
__device__ __forceinline__ size_t ckpt_scale_offset(size_t codes) { return (codes + 15) / 16 * 16; }

// Four states of a channel whose N states lie over P lanes: the codes packed
// into a word, and the scale.
template <int P>
__device__ __forceinline__ uint32_t encode8(const float (&h)[4], float& scale) {
    float m = 0.f, bad = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m = fmaxf(m, fabsf(h[i]));
        bad = fmaf(h[i], 0.f, bad);   // NaN if any of them is not finite
    }
    m = group_max<P>(m);
    bad = group_sum<P>(bad);
    const bool some = m >= 1e-35f && bad == 0.f;
    const float inv = some ? 127.f / m : 0.f;
    scale = bad == 0.f ? (some ? m / 127.f : 0.f) : bad;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int q = some ? (int)rintf(h[i] * inv) : 0;
        w |= (uint32_t)(q & 0xff) << (8 * i);
    }
    return w;
}

}  // namespace wkv7
