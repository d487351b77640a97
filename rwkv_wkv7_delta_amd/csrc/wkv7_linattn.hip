// wkv7_linattn.hip -- linear attention with one decay per head: prompts and
// single tokens.
//
// Per head, S (P x N, fp32) over the tokens:
//   S_t = exp(g_t) S_{t-1} + v_t k_t^T,   y_t = scale S_t q_t.
// Over a tile of 64 tokens, with G_t the sum of the log decays up to and with t
// and S the state before the tile,
//   y_t = scale (e^{G_t} S q_t + sum_{s <= t} e^{G_t - G_s} (q_t . k_s) v_s)
//   S  <- e^{G_end} S + sum_s (e^{G_end - G_s} v_s) k_s^T
// which are plain matrix products: a scalar decay only scales their rows.

#include "wkv7_linattn_device.h"

namespace wkv7 {

namespace {

// The head that a workgroup takes: neighbouring workgroups take heads of different
// groups, so that the heads that read the same keys come G apart (on one XCD where
// G is a multiple of 8).
__device__ __forceinline__ int head_of(int i, int H, int G) { return i % G * (H / G) + i / G; }

struct LaBlock {
    int b, h, p0, r;   // batch row, head, first value row, segment in the order of the sweep
};
template <int PB>
__device__ __forceinline__ LaBlock la_block(const LaArgs& p) {
    const unsigned bh = (unsigned)p.B * p.H, i = blockIdx.x;
    LaBlock w;
    const unsigned j = i % bh, rest = i / bh;
    w.b = (int)(j / p.H);
    w.h = head_of((int)(j % p.H), p.H, p.G);
    const unsigned blocks = (unsigned)p.P / PB;
    w.p0 = (int)(rest % blocks) * PB;
    w.r = (int)(rest / blocks);
    return w;
}

// State rows p0 + 16 wave .. of [B][H][P][N], as 16 x 16 results [n][p].
template <int N>
__device__ __forceinline__ float* state_at(float* base, const LaArgs& p, int b, int h, int row) {
    return base + (((size_t)b * p.H + h) * p.P + row) * N;
}

// ---- the sweep over states alone ------------------------------------------------
// Forward (kReverse = false): S from k and v; reverse: its gradient D, from q and
// dy: D <- e^{G_end} D + scale sum_t (e^{G_t} dy_t) q_t^T.
// kSegment: what a segment leaves from zero, and its summed decay.  Else (the
// reverse only) D behind every tile is written, and the gradient of the first state.
template <typename T, int N, int PB, bool kReverse, bool kSegment>
__global__ __launch_bounds__(kLaThreads) void la_sweep_kernel(const LaArgs p, const T* kk, const T* vv,
                                                              const float* first, float* last, T* marks) {
    typedef LaMat<T> M;
    typedef LaStage<T, N> SK;
    typedef LaStage<T, PB> SV;
    constexpr int NT = N / 16;
    __shared__ __attribute__((aligned(16))) T s_k[kLaChunk * SK::kStride];
    __shared__ __attribute__((aligned(16))) T s_v[kLaChunk * SV::kStride];
    __shared__ LaDecay s_d;
    const LaBlock w = la_block<PB>(p);
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, l16 = lane % 16;
    const LaRow row = la_row(p.rows, p.packed, p.tokens, p.T, w.b);
    const int seg = kReverse ? p.nseg - 1 - w.r : w.r;
    const int64_t begin = (int64_t)seg * p.seg_len;
    const int64_t stop = seg == p.nseg - 1 ? row.len : begin + p.seg_len;
    const int end = (int)(stop < row.len ? stop : row.len);
    const bool mine = wave < PB / 16;
    const int prow = w.p0 + 16 * wave + l16;
    f32x4 st[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) st[n] = zero4();
    const size_t states = (size_t)p.B * p.H * p.P * N;
    if (mine && !kSegment) {
        const float* from = w.r > 0 ? p.seg_state + (w.r - 1) * states : first;
        if (from) {
            from = state_at<N>(const_cast<float*>(from), p, w.b, w.h, prow);
#pragma unroll
            for (int n = 0; n < NT; ++n) st[n] = *reinterpret_cast<const f32x4*>(from + 16 * n + 4 * g);
        }
    }
    const int kh = w.h / (p.H / p.G);
    const int64_t krow = (int64_t)p.G * N, vrow = (int64_t)p.H * p.P;
    const int tiles = end > begin ? (int)((end - begin + kLaChunk - 1) / kLaChunk) : 0;
    SK rk;
    SV rv;
    LaLog<T> lg;
    auto load = [&](int c) {
        const int64_t t0 = begin + (int64_t)c * kLaChunk;
        const int n = (int)(end - t0 < kLaChunk ? end - t0 : kLaChunk);
        const int64_t at = row.first + t0;
        rk.load(rows_of(kk + at * krow + kh * N, n, krow, N), (uint32_t)(krow * sizeof(T)));
        rv.load(rows_of(vv + at * vrow + (int64_t)w.h * p.P + w.p0, n, vrow, PB), (uint32_t)(vrow * sizeof(T)));
        if (wave == 0) lg.load(p, at + lane, w.h, lane < n);
    };
    const auto tile_of = [&](int i) { return kReverse ? tiles - 1 - i : i; };
    double total = 0;
    if (tiles > 0) load(tile_of(0));
    for (int i = 0; i < tiles; ++i) {
        __syncthreads();
        rk.store(s_k);
        rv.store(s_v);
        if (wave == 0) put_decays(s_d, lg.x);
        __syncthreads();
        if (i + 1 < tiles) load(tile_of(i + 1));
        if (mine) {
            if (!kSegment) {
                T* const m = marks + (((row.ckpt + begin / kLaChunk + tile_of(i)) * p.H + w.h) * p.P + prow) * N;
#pragma unroll
                for (int n = 0; n < NT; ++n) M::put(m + 16 * n + 4 * g, st[n]);
            }
            if (kSegment) total += s_d.sum;
            const float all = s_d.all;
#pragma unroll
            for (int n = 0; n < NT; ++n) st[n] *= all;
#pragma unroll
            for (int t = 0; t < kLaChunk; t += 32) {
                f32x4 x[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t1 = t + 16 * u;
                    x[u] = M::wide(M::column(s_v + t1 * SV::kStride + 16 * wave, SV::kStride, g, l16));
                    const f32x4 e = *reinterpret_cast<const f32x4*>((kReverse ? s_d.up : s_d.down) + t1 + 4 * g);
                    x[u] *= kReverse ? e * p.scale : e;
                }
                typename M::Frag f[M::kParts];
                split_parts<T>(x[0], x[1], f);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const typename M::Frag a = columns<T>(s_k + t * SK::kStride + 16 * n, SK::kStride, g, l16);
#pragma unroll
                    for (int i2 = M::kParts - 1; i2 >= 0; --i2) st[n] = M::mma(a, f[i2], st[n]);
                }
            }
        }
    }
    if (mine && last && (kSegment || w.r == p.nseg - 1)) {
        float* const to = state_at<N>(last + (kSegment ? w.r * states : 0), p, w.b, w.h, prow);
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(to + 16 * n + 4 * g) = st[n];
    }
    if (kSegment && threadIdx.x == 0 && w.p0 == 0) p.seg_decay[((size_t)w.r * p.B + w.b) * p.H + w.h] = total;
}

// The states behind the segments: each from the one before, decayed, and its own.
__global__ __launch_bounds__(256) void la_join_kernel(const LaArgs p, const float* first) {
    const size_t states = (size_t)p.B * p.H * p.P * p.N;
    const size_t e = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (e >= states) return;
    const size_t head = e / ((size_t)p.P * p.N), heads = (size_t)p.B * p.H;
    f32x4 s = zero4();
    if (first) s = *reinterpret_cast<const f32x4*>(first + e);
    for (int r = 0; r + 1 < p.nseg; ++r) {
        float* const at = p.seg_state + r * states + e;
        const float d = exp2_raw((float)p.seg_decay[r * heads + head]);
        s = s * d + *reinterpret_cast<const f32x4*>(at);
        *reinterpret_cast<f32x4*>(at) = s;
    }
}

// ---- prompts --------------------------------------------------------------------
// A workgroup takes 64 (or all 32) value rows of a head's state over a segment.
// Wave w has tokens 16 w .. of the tile for the read-out and value rows 16 w .. of
// the state.  Results are formed transposed, [s][t], [p][t], [n][p], so that each
// feeds the next product from registers (wkv7_linattn_device.h).
template <typename T, int N, int PB>
struct LaFwdShared {
    typedef LaStage<T, N> SK;
    typedef LaStage<T, PB> SV;
    // Two of everything, and one barrier a tile, where both fit twice into a unit's LDS.
    static constexpr int kBytes = (kLaChunk * (SK::kStride + SV::kStride) + PB * SK::kStride) * (int)sizeof(T);
    static constexpr int kBuffers = kBytes <= 28 * 1024 ? 2 : 1;
    T k[kBuffers][kLaChunk * SK::kStride];
    T v[kBuffers][kLaChunk * SV::kStride];
    T s[kBuffers][PB * SK::kStride];   // the state before the tile, [p][n], in the tokens' type
    LaDecay d[kBuffers];
};

template <typename T, int N, int PB>
__global__ __launch_bounds__(kLaThreads) void la_fwd_kernel(const LaArgs p) {
    typedef LaMat<T> M;
    typedef LaStage<T, N> SK;
    typedef LaStage<T, PB> SV;
    typedef LaFwdShared<T, N, PB> Shared;
    typedef typename M::Frag Frag;
    constexpr int NT = N / 16, PT = PB / 16, KS = N / 32, BUF = Shared::kBuffers;
    constexpr int kQ = KS * (int)sizeof(T) / 2;   // 16-byte loads of a lane's query
    __shared__ __attribute__((aligned(16))) Shared sm;
    const LaBlock w = la_block<PB>(p);
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, l16 = lane % 16;
    const LaRow row = la_row(p.rows, p.packed, p.tokens, p.T, w.b);
    const int64_t begin = (int64_t)w.r * p.seg_len;
    const bool tail = w.r == p.nseg - 1;
    const int64_t stop = begin + p.seg_len;
    const int end = (int)(tail || stop > row.len ? row.len : stop);          // tokens
    const int64_t zero_end = tail || stop > row.stored ? row.stored : stop;  // and places that are written
    const bool mine = wave < PT;
    const int prow = w.p0 + 16 * wave + l16;
    const size_t states = (size_t)p.B * p.H * p.P * N;
    f32x4 st[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) st[n] = zero4();
    if (mine) {
        const float* from = w.r > 0 ? p.seg_state + (w.r - 1) * states : p.s0;
        if (from) {
            from = state_at<N>(const_cast<float*>(from), p, w.b, w.h, prow);
#pragma unroll
            for (int n = 0; n < NT; ++n) st[n] = *reinterpret_cast<const f32x4*>(from + 16 * n + 4 * g);
        }
    }
    const int kh = w.h / (p.H / p.G);
    const int64_t krow = (int64_t)p.G * N, vrow = (int64_t)p.H * p.P;
    const int tiles = end > begin ? (int)((end - begin + kLaChunk - 1) / kLaChunk) : 0;
    const T* const Q = static_cast<const T*>(p.q);
    const T* const K = static_cast<const T*>(p.k);
    const T* const V = static_cast<const T*>(p.v);
    T* const Y = static_cast<T*>(p.y);
    SK rk;
    SV rv;
    LaLog<T> lg;
    vu4 rq[kQ];
    auto load = [&](int c) {
        const int64_t t0 = begin + (int64_t)c * kLaChunk;
        const int n = (int)(end - t0 < kLaChunk ? end - t0 : kLaChunk);
        const int64_t at = row.first + t0;
        const uint32_t kb = (uint32_t)(krow * sizeof(T));
        rk.load(rows_of(K + at * krow + kh * N, n, krow, N), kb);
        rv.load(rows_of(V + at * vrow + (int64_t)w.h * p.P + w.p0, n, vrow, PB), (uint32_t)(vrow * sizeof(T)));
        const auto qb = rows_of(Q + at * krow + kh * N, n, krow, N);
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int j = 0; j < kQ / KS; ++j)
                rq[i * (kQ / KS) + j] = __builtin_bit_cast(vu4, __builtin_amdgcn_raw_buffer_load_b128(
                    qb, (16 * wave + l16) * kb + (32 * i + 8 * g) * (uint32_t)sizeof(T) + 16 * j, 0, 0));
        if (wave == 0) lg.load(p, at + lane, w.h, lane < n);
    };
    auto put = [&](int buf) {
        rk.store(sm.k[buf]);
        rv.store(sm.v[buf]);
        if (wave == 0) put_decays(sm.d[buf], lg.x);
        const bool odd = __builtin_amdgcn_ballot_w64(rk.odd() || rv.odd()) != 0;
        if (lane == 0) sm.d[buf].odd[wave] = odd;
    };
    auto put_state = [&](int buf) {
        if (mine)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                M::put(sm.s[buf] + (16 * wave + l16) * SK::kStride + 16 * n + 4 * g, st[n]);
    };
    put_state(0);
    if (tiles > 0) {
        load(0);
        put(0);
    }
    for (int c = 0; c < tiles; ++c) {
        const int buf = BUF == 2 ? c & 1 : 0, nxt = BUF == 2 ? buf ^ 1 : 0;
        Frag qf[KS];
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            if constexpr (sizeof(T) == 2) qf[i] = __builtin_bit_cast(Frag, rq[i]);
            else qf[i] = M::cat(__builtin_bit_cast(f32x4, rq[2 * i]), __builtin_bit_cast(f32x4, rq[2 * i + 1]));
        }
        __syncthreads();
        const int64_t t0 = begin + (int64_t)c * kLaChunk;
        const int n_in = (int)(end - t0 < kLaChunk ? end - t0 : kLaChunk);
        const int n_out = (int)(zero_end - t0 < kLaChunk ? zero_end - t0 : kLaChunk);
        const T* const sk = sm.k[buf];
        const T* const sv = sm.v[buf];
        const LaDecay& d = sm.d[buf];
        const int64_t at = row.first + t0;
        if (p.ckpt && mine) {
            T* const m = static_cast<T*>(p.ckpt) +
                         (((row.ckpt + begin / kLaChunk + c) * p.H + w.h) * p.P + prow) * N;
#pragma unroll
            for (int n = 0; n < NT; ++n) M::put(m + 16 * n + 4 * g, st[n]);
        }
        if (c + 1 < tiles) load(c + 1);
        const auto yb = rows_of(Y + at * vrow + (int64_t)w.h * p.P + w.p0, n_out, vrow, PB);
        const uint32_t yrow = (uint32_t)(vrow * sizeof(T));
        const int odd = __builtin_amdgcn_readfirstlane(d.odd[0] | d.odd[1] | d.odd[2] | d.odd[3]);
        if (!odd) {
            // [s][t] of the wave's tokens t against those up to them.
            const int t = 16 * wave + l16;
            const float thi = d.hi[t], tlo = d.lo[t], tup = d.up[t];
            Frag pf[2];
#pragma unroll
            for (int j2 = 0; j2 < 2; ++j2) {
                typename M::Half h2[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int j = 2 * j2 + u;
                    f32x4 a = zero4();
                    if (j <= wave) {
#pragma unroll
                        for (int i = 0; i < KS; ++i)
                            a = M::mma(M::rows(sk + (16 * j + l16) * SK::kStride + 32 * i + 8 * g), qf[i], a);
                        const f32x4 shi = *reinterpret_cast<const f32x4*>(d.hi + 16 * j + 4 * g);
                        const f32x4 slo = *reinterpret_cast<const f32x4*>(d.lo + 16 * j + 4 * g);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float e = exp2_raw((thi - shi[q]) + (tlo - slo[q]));
                            a[q] = 16 * j + 4 * g + q <= t ? a[q] * e : 0.f;
                        }
                    }
                    // Rounded to the tokens' type for the product with v: an error of half a
                    // step of each weight, as large as y's own rounding.
                    h2[u] = M::half(a);
                }
                pf[j2] = M::cat(h2[0], h2[1]);
            }
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) {
                f32x4 o = zero4();
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    o = M::mma(M::rows(sm.s[buf] + (16 * pt + l16) * SK::kStride + 32 * i + 8 * g), qf[i], o);
                o *= tup;
                o = M::mma(columns<T>(sv + 16 * pt, SV::kStride, g, l16), pf[0], o);
                if (wave >= 2) o = M::mma(columns<T>(sv + 32 * SV::kStride + 16 * pt, SV::kStride, g, l16), pf[1], o);
                // nothing of a state that is not finite behind the row's last token
#pragma unroll
                for (int q = 0; q < 4; ++q) o[q] = t < n_in ? o[q] * p.scale : 0.f;
                const uint32_t off = t * yrow + (16 * pt + 4 * g) * (uint32_t)sizeof(T);
                if constexpr (sizeof(T) == 2)
                    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(vu2, cvt4(o)), yb, off, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(vu4, o), yb, off, 0, 0);
            }
            if (mine) {
                const float all = d.all;
#pragma unroll
                for (int n = 0; n < NT; ++n) st[n] *= all;
#pragma unroll
                for (int t1 = 0; t1 < kLaChunk; t1 += 32) {
                    f32x4 x[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        x[u] = M::wide(M::column(sv + (t1 + 16 * u) * SV::kStride + 16 * wave, SV::kStride, g, l16));
                        x[u] *= *reinterpret_cast<const f32x4*>(d.down + t1 + 16 * u + 4 * g);
                    }
                    Frag f[M::kParts];
                    split_parts<T>(x[0], x[1], f);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const Frag a = columns<T>(sk + t1 * SK::kStride + 16 * n, SK::kStride, g, l16);
#pragma unroll
                        for (int i = M::kParts - 1; i >= 0; --i) st[n] = M::mma(a, f[i], st[n]);
                    }
                }
            }
        } else if (mine) {
            // An infinity or a NaN among the tile's keys and values: token by token, so that it
            // reaches no token before its own (in a product it would meet their zero weights).
            for (int i = 0; i < n_out; ++i) {
                float y = 0.f;
                if (i < n_in) {
                    const float e = exp2_raw(d.hi[i] - (i > 0 ? d.hi[i - 1] : 0.f) + (d.lo[i] - (i > 0 ? d.lo[i - 1] : 0.f)));
                    const float v = Elem<T>::load1(sv + i * SV::kStride + 16 * wave + l16);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float4 k = Elem<T>::load4(sk + i * SK::kStride + 16 * n + 4 * g);
                        const float4 q = Elem<T>::load4(Q + (at + i) * krow + kh * N + 16 * n + 4 * g);
                        st[n][0] = fmaf(k.x, v, st[n][0] * e);
                        st[n][1] = fmaf(k.y, v, st[n][1] * e);
                        st[n][2] = fmaf(k.z, v, st[n][2] * e);
                        st[n][3] = fmaf(k.w, v, st[n][3] * e);
                        y = fmaf(st[n][3], q.w, fmaf(st[n][2], q.z, fmaf(st[n][1], q.y, fmaf(st[n][0], q.x, y))));
                    }
                    y = sum_rows4(y) * p.scale;
                }
                if (g == 0) Elem<T>::store1(Y + (at + i) * vrow + (int64_t)w.h * p.P + prow, y);
            }
        }
        if (BUF == 1) __syncthreads();
        put_state(nxt);
        if (c + 1 < tiles) put(nxt);
    }
    if (mine && tail && p.sT) {
        float* const to = state_at<N>(p.sT, p, w.b, w.h, prow);
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(to + 16 * n + 4 * g) = st[n];
    }
    // Places behind the last tile (of a padded row): 0.
    const int64_t from = begin + (int64_t)tiles * kLaChunk;
    constexpr int kPer = 16 / (int)sizeof(T);
    for (int64_t i = threadIdx.x; i < (zero_end - from) * (PB / kPer); i += kLaThreads)
        *reinterpret_cast<vu4*>(Y + (row.first + from + i / (PB / kPer)) * vrow + (int64_t)w.h * p.P + w.p0 +
                                i % (PB / kPer) * kPer) = vu4{0, 0, 0, 0};
}

// ---- one token ------------------------------------------------------------------
// N / 4 lanes per state row, four columns each; 4096 / N rows a workgroup (four of
// a lane's 16-byte loads in flight).  Bound by the states' bytes.
template <typename T, int N>
__global__ __launch_bounds__(256) void la_step_kernel(const LaStepArgs p) {
    constexpr int kLanes = N / 4, kRows = 4096 / N, kEach = 256 / kLanes;
    const unsigned blocks = ((unsigned)p.P + kRows - 1) / kRows;
    const unsigned pb = blockIdx.x % blocks, bh = blockIdx.x / blocks;
    const int h = (int)(bh % p.H), b = (int)(bh / p.H);
    const int c = threadIdx.x % kLanes * 4, r0 = (int)pb * kRows + threadIdx.x / kLanes;
    int64_t slot = b;
    bool live = true;
    if (p.slots) {
        slot = p.slots[b];
        live = slot >= 0 && slot < p.nslots;
        // A slot that an earlier row names too is that row's.
        bool twice = false;
        for (int i = threadIdx.x % 64; i < b; i += 64) twice |= p.slots[i] == slot;
        live = live && __builtin_amdgcn_ballot_w64(twice) == 0;
    }
    const float decay = exp2_raw((p.fixed ? static_cast<const float*>(p.g)[h]
                                          : Elem<T>::load1(static_cast<const T*>(p.g) + (size_t)b * p.H + h)) * kLog2e);
    const size_t kat = ((size_t)b * p.G + h / (p.H / p.G)) * N + c;
    const float4 k = Elem<T>::load4(static_cast<const T*>(p.k) + kat), q = Elem<T>::load4(static_cast<const T*>(p.q) + kat);
    float* const S = p.state + (((size_t)(live ? slot : 0) * p.H + h) * p.P) * N + c;
    float4 s[4];
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + i * kEach;
        if (live && r < p.P) {
            s[i] = *reinterpret_cast<const float4*>(S + (size_t)r * N);
            v[i] = Elem<T>::load1(static_cast<const T*>(p.v) + (size_t)bh * p.P + r);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + i * kEach;
        if (r >= p.P) continue;
        float y = 0.f;
        if (live) {
            s[i].x = fmaf(k.x, v[i], s[i].x * decay);
            s[i].y = fmaf(k.y, v[i], s[i].y * decay);
            s[i].z = fmaf(k.z, v[i], s[i].z * decay);
            s[i].w = fmaf(k.w, v[i], s[i].w * decay);
            *reinterpret_cast<float4*>(S + (size_t)r * N) = s[i];
            y = dot4(s[i], q);
        }
        y = lanes_sum<(kLanes < 16 ? kLanes : 16)>(y);
        if constexpr (kLanes == 32) y += __shfl_xor(y, 16);
        if (c == 0) Elem<T>::store1(static_cast<T*>(p.y) + (size_t)bh * p.P + r, y * p.scale);
    }
}

template <typename T, int N, int PB>
hipError_t fwd_block(const LaArgs& p, hipStream_t stream) {
    const unsigned blocks = (unsigned)p.B * p.H * (p.P / PB);
    if (p.nseg > 1) {
        la_sweep_kernel<T, N, PB, false, true><<<blocks * (p.nseg - 1), kLaThreads, 0, stream>>>(
            p, static_cast<const T*>(p.k), static_cast<const T*>(p.v), nullptr, p.seg_state, nullptr);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        la_join_kernel<<<(unsigned)(((size_t)p.B * p.H * p.P * N / 4 + 255) / 256), 256, 0, stream>>>(p, p.s0);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    la_fwd_kernel<T, N, PB><<<blocks * p.nseg, kLaThreads, 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T, int N, int PB>
hipError_t adjoint_block(const LaBwdArgs& q, hipStream_t stream) {
    const LaArgs& p = q.f;
    const unsigned blocks = (unsigned)p.B * p.H * (p.P / PB);
    const T* const Q = static_cast<const T*>(p.q);
    const T* const dY = static_cast<const T*>(q.dy);
    if (p.nseg > 1) {
        la_sweep_kernel<T, N, PB, true, true><<<blocks * (p.nseg - 1), kLaThreads, 0, stream>>>(
            p, Q, dY, nullptr, p.seg_state, nullptr);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        la_join_kernel<<<(unsigned)(((size_t)p.B * p.H * p.P * N / 4 + 255) / 256), 256, 0, stream>>>(p, q.dsT);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    la_sweep_kernel<T, N, PB, true, false><<<blocks * p.nseg, kLaThreads, 0, stream>>>(
        p, Q, dY, q.dsT, q.ds0, static_cast<T*>(q.adj));
    return hipGetLastError();
}

}  // namespace

#define WKV7_LA_SIZES(fn, T, p, q)                                                            \
    switch ((p).N) {                                                                          \
        case 32: return (p).P < 64 ? fn<T, 32, 32>(q, stream) : fn<T, 32, 64>(q, stream);     \
        case 64: return (p).P < 64 ? fn<T, 64, 32>(q, stream) : fn<T, 64, 64>(q, stream);     \
        case 128: return (p).P < 64 ? fn<T, 128, 32>(q, stream) : fn<T, 128, 64>(q, stream);  \
        default: return hipErrorInvalidValue;                                                 \
    }

hipError_t launch_la_forward(const LaArgs& p, hipStream_t stream) {
    if (p.bf16) {
        WKV7_LA_SIZES(fwd_block, bf16_t, p, p)
    } else {
        WKV7_LA_SIZES(fwd_block, float, p, p)
    }
}

hipError_t launch_la_adjoint(const LaBwdArgs& q, hipStream_t stream) {
    if (q.f.bf16) {
        WKV7_LA_SIZES(adjoint_block, bf16_t, q.f, q)
    } else {
        WKV7_LA_SIZES(adjoint_block, float, q.f, q)
    }
}

hipError_t launch_la_step(const LaStepArgs& p, hipStream_t stream) {
    const unsigned rows = 4096 / p.N;
    const unsigned grid = (unsigned)p.B * p.H * ((p.P + rows - 1) / rows);
#define WKV7_LA_STEP(N)                                                                       \
    case N:                                                                                   \
        if (p.bf16) la_step_kernel<bf16_t, N><<<grid, 256, 0, stream>>>(p);                   \
        else la_step_kernel<float, N><<<grid, 256, 0, stream>>>(p);                           \
        return hipGetLastError();
    switch (p.N) {
        WKV7_LA_STEP(32)
        WKV7_LA_STEP(64)
        WKV7_LA_STEP(128)
        default: return hipErrorInvalidValue;
    }
}

}  // namespace wkv7
