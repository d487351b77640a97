// wkv7_linattn_device.h -- tiles, operands and decays of the linear attention
// kernels.
//
// A tile is 64 tokens of one head; a workgroup is eight waves, two per SIMD, so that
// one computes while the other waits for its operands (twelve where there are
// gradients).  Products go through the matrix cores in 16 x 16 results, 32 deep: for bf16 tokens one
// 16x16x32 instruction, for fp32 tokens eight 16x16x4 ones.  Which 32 values of
// the contraction a lane's eight operand elements stand for is the same for
// both operands of every product here, one of
//   rows     8 g + j                (read along a row of memory)
//   columns  4 g + j, 16 + 4 g + j - 4  (j < 4, j >= 4; read down a column)
// with g = lane / 16: the second is also how the lanes hold two result tiles
// (row 4 g + q in register q), so a result feeds the next product in place.
#pragma once

#include "wkv7_linattn_internal.h"
#include "wkv7_mfma.h"
#include "wkv7_ssm_device.h"

namespace wkv7 {

constexpr int kLaThreads = 512;

template <typename T> struct LaMat;

template <> struct LaMat<bf16_t> {
    typedef bf16x8 Frag;
    typedef bf16x4 Half;
    static constexpr int kParts = 3;   // bf16 terms that carry a 32-bit operand
    static constexpr int kTerms = 2;   // and those of a weight, or of a state that is read out
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) { return mfma32(a, b, c); }
    static __device__ __forceinline__ Frag cat(Half a, Half b) { return cat8(a, b); }
    static __device__ __forceinline__ Half half(f32x4 x) { return cvt4(x); }
    static __device__ __forceinline__ f32x4 wide(Half x) { return unpack4(x); }
    static __device__ __forceinline__ Frag rows(const bf16_t* p) {
        return __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(p));
    }
    static __device__ __forceinline__ Half column(const bf16_t* tile, int stride, int g, int l16) {
        return ld4_tr(tr_addr(tile, stride, g, l16));
    }
    static __device__ __forceinline__ Half four(const bf16_t* p) {
        return __builtin_bit_cast(bf16x4, *reinterpret_cast<const uint2*>(p));
    }
    static __device__ __forceinline__ void put(bf16_t* p, f32x4 x) { put(p, cvt4(x)); }
    static __device__ __forceinline__ void put(bf16_t* p, Half x) { *reinterpret_cast<uint2*>(p) = __builtin_bit_cast(uint2, x); }
};

template <> struct LaMat<float> {
    struct Frag {
        float v[8];
    };
    typedef f32x4 Half;
    static constexpr int kParts = 1, kTerms = 1;
    static __device__ __forceinline__ f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag cat(Half a, Half b) {
        Frag f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f.v[j] = a[j];
            f.v[4 + j] = b[j];
        }
        return f;
    }
    static __device__ __forceinline__ Half half(f32x4 x) { return x; }
    static __device__ __forceinline__ f32x4 wide(Half x) { return x; }
    static __device__ __forceinline__ Frag rows(const float* p) {
        return cat(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4));
    }
    static __device__ __forceinline__ Half column(const float* tile, int stride, int g, int l16) {
        Half h;
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = tile[(4 * g + q) * stride + l16];
        return h;
    }
    static __device__ __forceinline__ Half four(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
    static __device__ __forceinline__ void put(float* p, f32x4 x) { *reinterpret_cast<f32x4*>(p) = x; }
};

// Two column halves, rows r0 and r0 + 16 of a tile in LDS.
template <typename T>
__device__ __forceinline__ typename LaMat<T>::Frag columns(const T* tile, int stride, int g, int l16) {
    typedef LaMat<T> M;
    return M::cat(M::column(tile, stride, g, l16), M::column(tile + 16 * stride, stride, g, l16));
}

// A 32-bit operand as kParts operands in the tokens' type that sum to it: three
// bf16 terms hold 24 bits, so that states (fp32) lose nothing to the matrix
// cores' input type.  The first two are cut off, not rounded: the cut value is its
// own fp32 image, so that the rest is one subtraction away.  Finite values only.
template <typename T>
__device__ __forceinline__ void split_parts(const f32x4& lo, const f32x4& hi, typename LaMat<T>::Frag (&f)[LaMat<T>::kParts]) {
    typedef LaMat<T> M;
    if constexpr (M::kParts == 1) {
        f[0] = M::cat(lo, hi);
    } else {
        f32x4 x[2] = {lo, hi};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            vu4 w;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t a = __float_as_uint(x[h][2 * j]), b = __float_as_uint(x[h][2 * j + 1]);
                    w[2 * h + j] = __builtin_amdgcn_perm(b, a, 0x07060302u);   // the upper halves
                    x[h][2 * j] -= __uint_as_float(a & 0xffff0000u);
                    x[h][2 * j + 1] -= __uint_as_float(b & 0xffff0000u);
                }
            f[i] = __builtin_bit_cast(typename M::Frag, w);
        }
        f[2] = M::cat(M::half(x[0]), M::half(x[1]));
    }
}

// A weight within a tile, or a read-out's state, as kTerms halves that sum to it: with bf16
// tokens what is cut off after 8 bits and the rest, rounded, so that 2^-17 of it is lost, a
// 256th of the output's own rounding.  (Rounded to one bf16, they made outputs 1.4 times as
// wrong as their rounding.)  An infinity becomes a NaN.
template <typename T>
__device__ __forceinline__ void split_terms(const f32x4& x, typename LaMat<T>::Half (&h)[LaMat<T>::kTerms]) {
    typedef LaMat<T> M;
    if constexpr (M::kTerms == 1) {
        h[0] = x;
    } else {
        vu2 w;
        f32x4 rest;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t a = __float_as_uint(x[2 * j]), b = __float_as_uint(x[2 * j + 1]);
            w[j] = __builtin_amdgcn_perm(b, a, 0x07060302u);   // the upper halves
            rest[2 * j] = x[2 * j] - __uint_as_float(a & 0xffff0000u);
            rest[2 * j + 1] = x[2 * j + 1] - __uint_as_float(b & 0xffff0000u);
        }
        h[0] = __builtin_bit_cast(typename M::Half, w);
        h[1] = M::half(rest);
    }
}

// State columns [n][p] of 16 value rows, moved on over a tile: decayed by `all`, and each
// token's value, times its factor and `scale`, with its key.
template <typename T, int NT>
__device__ __forceinline__ void move_state(f32x4 (&st)[NT], const T* k, int kstride, const T* v, int vstride,
                                           const float* factor, float scale, float all, bool odd, int g, int l16) {
    typedef LaMat<T> M;
#pragma unroll
    for (int n = 0; n < NT; ++n) st[n] *= all;
    if (!odd) {
#pragma unroll
        for (int t = 0; t < kLaChunk; t += 32) {
            f32x4 x[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                x[u] = M::wide(M::column(v + (t + 16 * u) * vstride, vstride, g, l16));
                x[u] *= *reinterpret_cast<const f32x4*>(factor + t + 16 * u + 4 * g) * scale;
            }
            typename M::Frag f[M::kParts];
            split_parts<T>(x[0], x[1], f);
#pragma unroll
            for (int i = M::kParts - 1; i >= 0; --i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    st[n] = M::mma(columns<T>(k + t * kstride + 16 * n, kstride, g, l16), f[i], st[n]);
        }
    } else {
        // Infinities and NaN: without the parts, which would meet them as zeros.
        for (int t = 0; t < kLaChunk; ++t) {
            const float x = Elem<T>::load1(v + t * vstride + l16) * (factor[t] * scale);
#pragma unroll
            for (int n = 0; n < NT; ++n) st[n] += M::wide(M::four(k + t * kstride + 16 * n + 4 * g)) * x;
        }
    }
}

// ---- where a row's tokens are ---------------------------------------------------
struct LaRow {
    int64_t first;   // its first token among all
    int64_t ckpt;    // its first checkpoint
    int len;         // its tokens
    int stored;      // token places whose outputs are written
};
__device__ __forceinline__ LaRow la_row(const int32_t* rows, bool packed, int64_t tokens, int T, int b) {
    LaRow r;
    if (packed) {
        int64_t a = rows[b], e = rows[b + 1];
        a = a < 0 ? 0 : a > tokens ? tokens : a;
        e = e < a ? a : e > tokens ? tokens : e;
        r.first = a;
        r.len = r.stored = (int)(e - a);
        r.ckpt = a / kLaChunk + b;
    } else {
        r.first = (int64_t)b * T;
        r.len = row_length(rows, b, T);
        r.stored = T;
        r.ckpt = (int64_t)b * ((T + kLaChunk - 1) / kLaChunk);
    }
    r.len = __builtin_amdgcn_readfirstlane(r.len);
    r.stored = __builtin_amdgcn_readfirstlane(r.stored);
    return r;
}

// `n` rows of `width` elements, `stride` elements apart, as a buffer: what lies
// behind the last of them reads as 0 and is not written.  The offsets of 64 rows
// stay below 2^31 bytes (sizes are limited for that).
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const T* p, int n, int64_t stride, int width) {
    return buffer_of(p, n > 0 ? ((n - 1) * (int)stride + width) * (int)sizeof(T) : 0);
}

// A tile of up to 64 rows on its way from memory to LDS: 16 bytes per lane and load.
template <typename T, int W, int kThreads = kLaThreads, int kFirst = 0>   // threads kFirst ..
struct LaStage {
    static constexpr int kPieces = W * (int)sizeof(T) / 16;          // per row
    static constexpr int kRowsPer = kThreads / kPieces;            // rows of one load of the workgroup
    static constexpr int kLoads = kLaChunk > kRowsPer ? kLaChunk / kRowsPer : 1;
    static constexpr int kStride = W + 16 / (int)sizeof(T);          // elements of an LDS row: 16 bytes apart in the banks
    vu4 w[kLoads];

    // (With more threads than pieces several take the same one: no branch around the store.)
    __device__ __forceinline__ static uint32_t piece() { return (threadIdx.x - kFirst) % (kLaChunk * kPieces); }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row_bytes) {
        const uint32_t me = piece(), at = me / kPieces * row_bytes + me % kPieces * 16;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            w[i] = __builtin_bit_cast(vu4, __builtin_amdgcn_raw_buffer_load_b128(r, at + i * kRowsPer * row_bytes, 0, 0));
    }
    __device__ __forceinline__ void store(T* lds) const {
        const uint32_t me = piece();
        T* const p = lds + me / kPieces * kStride + me % kPieces * (16 / (int)sizeof(T));
#pragma unroll
        for (int i = 0; i < kLoads; ++i) *reinterpret_cast<vu4*>(p + i * kRowsPer * kStride) = w[i];
    }
    // Whether any of the lane's values is infinite or NaN.
    __device__ __forceinline__ bool odd() const {
        if constexpr (sizeof(T) == 2) {
            typedef unsigned short us2 __attribute__((ext_vector_type(2)));
            us2 m = {0, 0};
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    m = __builtin_elementwise_max(m, __builtin_bit_cast(us2, w[i][j] & 0x7fff7fffu));
            return m[0] >= 0x7f80 || m[1] >= 0x7f80;
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t u = w[i][j] & 0x7fffffffu;
                    m = m > u ? m : u;
                }
            return m >= 0x7f800000u;
        }
    }
};

// ---- decays ---------------------------------------------------------------------
// Running sums of a tile's log decays, in units of log 2.  Summed in 64 bits and
// kept as two floats: a difference of two of them is then as exact as a float
// is, however far the sums have run.
struct LaDecay {
    float hi[kLaChunk], lo[kLaChunk];
    float up[kLaChunk];     // 2^(G_t): from the tile's start to behind token t
    float down[kLaChunk];   // 2^(G_end - G_t): from behind token t to the tile's end
    float all;              // 2^(G_end)
    int odd[8];             // waves that found values that are not finite
    double sum;             // G_end
};

template <int kCtrl, int kRowMask>
__device__ __forceinline__ double dpp_double(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, kCtrl, kRowMask, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), kCtrl, kRowMask, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum over this lane and those before it in the wave: row_shr 1, 2, 4, 8, then
// each row's last lane to the row behind (rows 1 and 3) and lane 31 to the upper half.
__device__ __forceinline__ double wave_running_sum(double x) {
    x += dpp_double<0x111, 0xF>(x);
    x += dpp_double<0x112, 0xF>(x);
    x += dpp_double<0x114, 0xF>(x);
    x += dpp_double<0x118, 0xF>(x);
    x += dpp_double<0x142, 0xA>(x);
    x += dpp_double<0x143, 0xC>(x);
    return x;
}

template <int kWaves = 8>
__device__ __forceinline__ bool any_odd(const int (&odd)[8]) {
    int x = odd[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) x |= odd[i];
    return __builtin_amdgcn_readfirstlane(x) != 0;
}

// What lane t of a wave reads of token t's log decay; 0 behind the tile's n tokens.
template <typename T>
struct LaLog {
    uint32_t w;
    bool fixed;
    __device__ __forceinline__ void load(const LaArgs& p, int64_t token, int h, int n) {
        const uint32_t t = threadIdx.x % 64;
        fixed = p.fixed;
        if (p.fixed) {
            const auto r = buffer_of(static_cast<const float*>(p.g) + h, n > 0 ? 4 : 0);
            w = __builtin_amdgcn_raw_buffer_load_b32(r, (int)t < n ? 0 : kNowhere, 0, 0);
        } else {
            const auto r = rows_of(static_cast<const T*>(p.g) + token * p.H + h, n, p.H, 1);
            const uint32_t at = t * (uint32_t)(p.H * (int)sizeof(T));
            if constexpr (sizeof(T) == 2) w = __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
            else w = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
        }
    }
    __device__ __forceinline__ float get() const {
        return sizeof(T) == 4 || fixed ? __uint_as_float(w) : bf16_lo(w);
    }
};

// ---- a wave's 16 rows between memory and operands ---------------------------------
// Sixteen rows of W elements pass through LDS that only this wave touches, so that
// memory sees whole rows, 16 bytes a lane.
template <typename T, int W>
struct LaRows16 {
    static constexpr int kPieces = W * (int)sizeof(T) / 16, kEach = 16 * kPieces / 64;
    static constexpr int kStride = W + 16 / (int)sizeof(T);
    static constexpr int kSize = 16 * kStride;   // elements of LDS
    vu4 w[kEach];

    // What the wave's lanes wrote is there for its lanes to read, and the reverse.
    static __device__ __forceinline__ void settle() {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row_bytes, int row0) {
        const int lane = threadIdx.x % 64;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = i * 64 + lane;
            w[i] = __builtin_bit_cast(vu4, __builtin_amdgcn_raw_buffer_load_b128(
                r, (row0 + at / kPieces) * row_bytes + at % kPieces * 16, 0, 0));
        }
    }
    __device__ __forceinline__ void put(T* lds) const {
        const int lane = threadIdx.x % 64;
        settle();
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = i * 64 + lane;
            *reinterpret_cast<vu4*>(lds + at / kPieces * kStride + at % kPieces * (16 / (int)sizeof(T))) = w[i];
        }
        settle();
    }
    // Results [w][row] (row l16, columns 16 i + 4 g ..) of the rows row0 .. to memory; of 32 bits
    // (rounded) or as halves.
    template <typename X>
    static __device__ __forceinline__ void store(T* lds, const X (&x)[W / 16], __amdgpu_buffer_rsrc_t r,
                                                 uint32_t row_bytes, int row0) {
        const int lane = threadIdx.x % 64, g = lane / 16, l16 = lane % 16;
        settle();
#pragma unroll
        for (int i = 0; i < W / 16; ++i) LaMat<T>::put(lds + l16 * kStride + 16 * i + 4 * g, x[i]);
        settle();
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = i * 64 + lane;
            const vu4 v = *reinterpret_cast<const vu4*>(lds + at / kPieces * kStride + at % kPieces * (16 / (int)sizeof(T)));
            __builtin_amdgcn_raw_buffer_store_b128(v, r, (row0 + at / kPieces) * row_bytes + at % kPieces * 16, 0, 0);
        }
    }
};

// The 16 value rows that a wave holds of a state, as halves, columns n0 .. of N, to a
// checkpoint of PB rows (a buffer of them, or of nothing).
template <typename T, int N, int NT>
__device__ __forceinline__ void store_mark(T* lds, const typename LaMat<T>::Half (&st)[NT], __amdgpu_buffer_rsrc_t r,
                                           int ptile, int n0) {
    if constexpr (16 * NT == N && sizeof(T) == 2) {
        LaRows16<T, N>::store(lds, st, r, N * sizeof(T), ptile);
    } else {
        const int lane = threadIdx.x % 64, g = lane / 16, l16 = lane % 16;
        const uint32_t at = ((ptile + l16) * N + n0 + 4 * g) * (uint32_t)sizeof(T);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if constexpr (sizeof(T) == 2)
                __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(vu2, st[n]), r, at + 32 * n, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(vu4, st[n]), r, at + 64 * n, 0, 0);
        }
    }
}

// ---- adjoint states between the backward's kernels ------------------------------------
// With bf16 tokens a workspace of the checkpoints' size holds the gradients of the states, 16
// bits a value, and one bf16 would leave dk and dv 1.4 times as wrong as their own rounding.
// Eight neighbours along a row share an exponent instead: each is a half (relative to the
// largest, which becomes 2^14 up to 2^15) whose last bit gives place to one bit of the 8 of
// that exponent.  Ten significant bits down to 2^-28 of the largest of the eight, 2^-38 of
// that below.  Where one of the eight is not finite (exponent 255) each is a bf16 instead; where
// all are below 2^-112 they are read as such; below 2^-126 (exponent 0) they are zeros.
constexpr int kAdjointBias = 127 + 14;
constexpr uint32_t kAdjointBits = 0x00010001u;   // in the word of two

// As the lanes hold state rows: eight are four of lane row g and four of lane row g + 1 (g even).
template <int NT>
__device__ __forceinline__ void pack_adjoint(const f32x4 (&x)[NT], int g, bf16x4 (&to)[NT]) {
    uint32_t e[NT];
    vu2 w[NT];
    bool odd = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        // (the maximum that keeps a NaN)
        const float m = __builtin_elementwise_maximum(
            __builtin_elementwise_maximum(__builtin_elementwise_maximum(fabsf(x[n][0]), fabsf(x[n][1])), fabsf(x[n][2])),
            fabsf(x[n][3]));
        const auto both = __builtin_amdgcn_permlane16_swap(__float_as_uint(m), __float_as_uint(m), false, false);
        e[n] = (both[0] > both[1] ? both[0] : both[1]) >> 23;
        odd |= e[n] == 255;
        const int by = e[n] == 0 ? -300 : kAdjointBias - (int)e[n];
        // Cut off to eleven bits; with one added, the ten above the last are the nearest.
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[n][i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(
                          __builtin_ldexpf(x[n][2 * i], by), __builtin_ldexpf(x[n][2 * i + 1], by))) + kAdjointBits;
    }
    if (__builtin_amdgcn_ballot_w64(odd) != 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) w[n][i] = e[n] == 255 ? cvt2(x[n][2 * i], x[n][2 * i + 1]) : w[n][i];
    }
    // Bit j of the exponent to element j: bits 0 and 16 of each word.
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const uint32_t spread = (e[n] | e[n] << 15) >> 4 * (g & 1);
        w[n][0] = (spread & kAdjointBits) | (w[n][0] & ~kAdjointBits);
        w[n][1] = (spread >> 2 & kAdjointBits) | (w[n][1] & ~kAdjointBits);
        to[n] = __builtin_bit_cast(bf16x4, w[n]);
    }
}

// Eight packed values as two terms in the matrix cores' type, which hold their ten bits: the
// first eight of them, and the rest.
__device__ __forceinline__ void unpack_adjoint(const vu4& d, vu4 (&term)[2]) {
    const uint32_t s = (d[0] & kAdjointBits) | (d[1] & kAdjointBits) << 2 | (d[2] & kAdjointBits) << 4 |
                       (d[3] & kAdjointBits) << 6;
    const int e = (int)((s | s >> 15) & 255u);
    const float scale = __uint_as_float((uint32_t)(e - (kAdjointBias - 127)) << 23);
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const h2 all = __builtin_bit_cast(h2, d[i] & 0xfffefffeu), top = __builtin_bit_cast(h2, d[i] & 0xfff8fff8u);
        const float a = fmaf((float)top[0], scale, 0.f), b = fmaf((float)top[1], scale, 0.f);
        term[0][i] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);   // the upper halves
        term[1][i] = cvt2(fmaf((float)all[0], scale, -a), fmaf((float)all[1], scale, -b));
    }
    // bf16 values, and a scale that is no float (without values there is nothing to scale).
    const bool tiny = (uint32_t)(e - 1) < kAdjointBias - 127;
    if (__builtin_amdgcn_ballot_w64(e == 255 || tiny) != 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const h2 all = __builtin_bit_cast(h2, d[i] & 0xfffefffeu);
            const float a = __builtin_ldexpf((float)all[0], e - kAdjointBias), b = __builtin_ldexpf((float)all[1], e - kAdjointBias);
            const uint32_t one = cvt2(a, b);
            term[0][i] = e == 255 ? d[i] & 0xfffefffeu : tiny ? one : term[0][i];
            term[1][i] = e == 255 || tiny ? 0u : term[1][i];
        }
    }
}

// By one whole wave.  A log decay of -infinity forgets everything: 2^-144270 is 0,
// and sums that hold it stay exact to 2^-30.
// A decay that is not a number, or infinite (a logarithm above 1e5), counts as 1 in the sums,
// so that the pairs of tokens behind it keep their weights; what crosses it becomes NaN through
// `up`, `down` and `all`: every token from it on reads the state before the tile, every one
// before it meets the state's gradient behind it, and both are scaled by these.
__device__ __forceinline__ void put_decays(LaDecay& d, float log_decay) {
    const int t = threadIdx.x % 64;
    const bool bad = !(log_decay <= 1e5f);
    const uint64_t odd = __builtin_amdgcn_ballot_w64(bad);
    const float nan = __builtin_nanf("");
    const double g = bad ? 0.0 : (double)fmaxf(log_decay, -1e5f) * 1.4426950408889634;
    const double c = wave_running_sum(g);
    const uint64_t u = __builtin_bit_cast(uint64_t, c);
    const uint32_t l0 = __builtin_amdgcn_readlane((uint32_t)u, 63), l1 = __builtin_amdgcn_readlane((uint32_t)(u >> 32), 63);
    const double end = __builtin_bit_cast(double, (uint64_t)l1 << 32 | l0);
    const float hi = (float)c;
    d.hi[t] = hi;
    d.lo[t] = (float)(c - (double)hi);
    d.up[t] = odd << (63 - t) != 0 ? nan : exp2_raw((float)c);
    d.down[t] = odd >> t >> 1 != 0 ? nan : exp2_raw((float)(end - c));
    // (64 lanes alike: no branch)
    d.all = odd != 0 ? nan : exp2_raw((float)end);
    d.sum = odd != 0 ? (double)nan : end;
}

}  // namespace wkv7
