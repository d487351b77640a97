// wkv7_linattn_bwd.hip -- gradients of linear attention with one decay per head.
//
// The gradient D of the state runs through the tiles backwards (the reverse sweep
// of wkv7_linattn.hip); then every tile of 64 tokens stands alone.  With S before
// it, D behind it, W_ts = scale e^{G_t - G_s} for s <= t, else 0:
//   dq_t = sum_s W_ts (dy_t . v_s) k_s + scale e^{G_t} S^T dy_t
//   dk_s = sum_t W_ts (dy_t . v_s) q_t + e^{G_end - G_s} D^T v_s
//   dv_s = sum_t W_ts (q_t . k_s) dy_t + e^{G_end - G_s} D k_s
// and, every g_t being in the decay of what crosses from before t to t or behind,
//   dg_t = sum_{i >= t > s} M_is + sum_{i >= t} a_i + sum_{s < t} b_s + e^{G_end} <S, D>
// with M_is = W_is (q_i . k_s)(dy_i . v_s), a_i = q_i . (the state's part of dq_i),
// b_s = k_s . (D's part of dk_s): sums within the tile only, however long the row is.

#include "wkv7_linattn_device.h"

namespace wkv7 {

namespace {

template <typename T, int N, int PB>
struct LaBwdShared {
    typedef LaStage<T, N> SK;
    typedef LaStage<T, PB> SV;
    T q[kLaChunk * SK::kStride], k[kLaChunk * SK::kStride];
    T v[kLaChunk * SV::kStride], dy[kLaChunk * SV::kStride];
    T s[PB * SK::kStride], ds[PB * SK::kStride];   // [p][n]
    LaDecay d;
    // For dg: sums of M along its rows, by wave; the rest of what counts for all tokens up to
    // one (a, and M down its columns taken off), for those behind it (b), and for all.
    float row[4][kLaChunk], a[kLaChunk], b[kLaChunk], c[4];
    int odd_k[4];
};

// PB state rows of N on their way to LDS (64 rows of LaStage, or 32).
template <typename T, int N, int PB>
struct LaStateStage {
    static constexpr int kPieces = N * (int)sizeof(T) / 16;
    static constexpr int kLoads = PB * kPieces / kLaThreads;
    static constexpr int kStride = N + 16 / (int)sizeof(T);
    vu4 w[kLoads > 0 ? kLoads : 1];
    // Rows are one behind the other in memory.
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            w[i] = *reinterpret_cast<const vu4*>(reinterpret_cast<const char*>(p) + (i * kLaThreads + threadIdx.x) * 16);
        if (kLoads == 0 && threadIdx.x < PB * kPieces)
            w[0] = *reinterpret_cast<const vu4*>(reinterpret_cast<const char*>(p) + threadIdx.x * 16);
    }
    __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
        for (int i = 0; i < (kLoads > 0 ? kLoads : 1); ++i) {
            const int at = i * kLaThreads + threadIdx.x;
            if (kLoads > 0 || at < PB * kPieces)
                *reinterpret_cast<vu4*>(lds + at / kPieces * kStride + at % kPieces * (16 / (int)sizeof(T))) = w[i];
        }
    }
    // The lane's part of <this, o>.
    __device__ __forceinline__ float dot(const LaStateStage& o) const {
        float x = 0.f;
        if (kLoads > 0 || threadIdx.x < PB * kPieces) {
#pragma unroll
            for (int i = 0; i < (kLoads > 0 ? kLoads : 1); ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (sizeof(T) == 4) {
                        x = fmaf(__uint_as_float(w[i][j]), __uint_as_float(o.w[i][j]), x);
                    } else {
                        x = fmaf(bf16_lo(w[i][j]), bf16_lo(o.w[i][j]), x);
                        x = fmaf(bf16_hi(w[i][j]), bf16_hi(o.w[i][j]), x);
                    }
                }
        }
        return x;
    }
};

__device__ __forceinline__ float wave_sum(float x) { return sum_rows4(row16_sum(x)); }

// One tile of one group of heads (or of a part of them) per workgroup; the sums over
// the heads that share a key stay in registers.  Wave w has the tokens 16 w .. both as
// queries (against those before) and as keys (against those behind): as many products
// for each wave.
template <typename T, int N, int PB>
__global__ __launch_bounds__(kLaThreads) void la_bwd_kernel(const LaBwdArgs o, int blocks) {
    typedef LaMat<T> M;
    typedef LaStage<T, N> SK;
    typedef LaStage<T, PB> SV;
    typedef typename M::Frag Frag;
    typedef typename M::Half Half;
    constexpr int NT = N / 16, PT = PB / 16, KS = N / 32, PS = PB / 32;
    __shared__ __attribute__((aligned(16))) LaBwdShared<T, N, PB> sm;
    const LaArgs& p = o.f;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, l16 = lane % 16;
    unsigned i = blockIdx.x;
    const int kh = (int)(i % p.G);
    i /= p.G;
    const int part = (int)(i % o.split);
    i /= o.split;
    const int b = (int)(i / blocks), c0 = (int)(i % blocks);
    const LaRow row = la_row(p.rows, p.packed, p.tokens, p.T, b);
    const int shared = p.H / p.G, per = (shared + o.split - 1) / o.split;
    const int h_first = kh * shared + part * per;
    const int heads = shared - part * per < per ? shared - part * per : per;
    const int pblocks = p.P / PB, steps = heads * pblocks;
    const int64_t krow = (int64_t)p.G * N, vrow = (int64_t)p.H * p.P;
    const T* const V = static_cast<const T*>(p.v);
    const T* const dY = static_cast<const T*>(o.dy);
    const T* const CK = static_cast<const T*>(p.ckpt);
    const T* const AD = static_cast<const T*>(o.adj);
    // Every tile of the row whose number is c0 modulo `blocks` (more than one only where a
    // packed row is longer than the call says).
    for (int64_t c = c0; c * kLaChunk < row.stored; c += blocks) {
        const int64_t t0 = c * kLaChunk, at = row.first + t0;
        const int n_in = (int)(row.len - t0 < kLaChunk ? (row.len > t0 ? row.len - t0 : 0) : kLaChunk);
        const int n_out = (int)(row.stored - t0 < kLaChunk ? row.stored - t0 : kLaChunk);
        const int t = 16 * wave + l16;
        const bool in = t < n_in;
        f32x4 dq[NT], dk[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) dq[n] = dk[n] = zero4();
        SV rv, ry;
        LaStateStage<T, N, PB> rs, rd;
        LaLog<T> lg;
        auto load = [&](int step) {
            const int h = h_first + step / pblocks, p0 = step % pblocks * PB;
            const int64_t vat = at * vrow + (int64_t)h * p.P + p0;
            rv.load(rows_of(V + vat, n_in, vrow, PB), (uint32_t)(vrow * sizeof(T)));
            ry.load(rows_of(dY + vat, n_in, vrow, PB), (uint32_t)(vrow * sizeof(T)));
            const size_t sat = (((size_t)(row.ckpt + c) * p.H + h) * p.P + p0) * N;
            rs.load(CK + sat);
            rd.load(AD + sat);
            if (wave == 0) lg.load(p, at + lane, h, lane < n_in);
        };
        __syncthreads();   // the tile before has been read
        if (n_in > 0) {
            SK rq, rk;
            const uint32_t kb = (uint32_t)(krow * sizeof(T));
            rq.load(rows_of(static_cast<const T*>(p.q) + at * krow + kh * N, n_in, krow, N), kb);
            rk.load(rows_of(static_cast<const T*>(p.k) + at * krow + kh * N, n_in, krow, N), kb);
            load(0);
            rq.store(sm.q);
            rk.store(sm.k);
            const bool odd = __builtin_amdgcn_ballot_w64(rq.odd() || rk.odd()) != 0;
            if (lane == 0) sm.odd_k[wave] = odd;
        }
        f32x4 rsum[4];   // M's rows 16 j + 4 g .., the lane's column
        float asum = 0.f, bsum = 0.f, cdot = 0.f;
        for (int step = 0; step < (n_in > 0 ? steps : 0); ++step) {
            const int h = h_first + step / pblocks, p0 = step % pblocks * PB;
            const bool head_first = step % pblocks == 0, head_last = step % pblocks == pblocks - 1;
            if (step > 0) __syncthreads();
            rv.store(sm.v);
            ry.store(sm.dy);
            rs.store(sm.s);
            rd.store(sm.ds);
            if (head_first) {
                if (wave == 0) put_decays(sm.d, lg.x);
#pragma unroll
                for (int j = 0; j < 4; ++j) rsum[j] = zero4();
                asum = bsum = cdot = 0.f;
            }
            cdot += rs.dot(rd);
            const bool odd_v = __builtin_amdgcn_ballot_w64(rv.odd() || ry.odd()) != 0;
            if (lane == 0) sm.d.odd[wave] = odd_v;
            __syncthreads();
            if (step + 1 < steps) load(step + 1);
            const LaDecay& d = sm.d;
            const int odd = __builtin_amdgcn_readfirstlane(d.odd[0] | d.odd[1] | d.odd[2] | d.odd[3] | sm.odd_k[0] |
                                                           sm.odd_k[1] | sm.odd_k[2] | sm.odd_k[3]);
            const float up = d.up[t] * p.scale, down = d.down[t];
            const float thi = d.hi[t], tlo = d.lo[t];
            f32x4 dv[PT];
            // ---- the states' parts
            {
                // dy_t and v_t along the states' columns (the contraction's second order)
                Frag yc[PS], vc[PS];
#pragma unroll
                for (int j = 0; j < PS; ++j) {
                    const T* const y1 = sm.dy + t * SV::kStride + 32 * j + 4 * g;
                    const T* const v1 = sm.v + t * SV::kStride + 32 * j + 4 * g;
                    yc[j] = M::cat(M::four(y1), M::four(y1 + 16));
                    vc[j] = M::cat(M::four(v1), M::four(v1 + 16));
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    f32x4 x = zero4(), y = zero4();
#pragma unroll
                    for (int j = 0; j < PS; ++j) {
                        x = M::mma(columns<T>(sm.s + 32 * j * SK::kStride + 16 * n, SK::kStride, g, l16), yc[j], x);
                        y = M::mma(columns<T>(sm.ds + 32 * j * SK::kStride + 16 * n, SK::kStride, g, l16), vc[j], y);
                    }
                    x *= up;
                    y *= down;
                    const f32x4 qn = M::wide(M::four(sm.q + t * SK::kStride + 16 * n + 4 * g));
                    const f32x4 kn = M::wide(M::four(sm.k + t * SK::kStride + 16 * n + 4 * g));
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        asum = fmaf(qn[r], x[r], asum);
                        bsum = fmaf(kn[r], y[r], bsum);
                    }
                    dq[n] += x;
                    dk[n] += y;
                }
                Frag kf[KS];
#pragma unroll
                for (int j = 0; j < KS; ++j) kf[j] = M::rows(sm.k + t * SK::kStride + 32 * j + 8 * g);
#pragma unroll
                for (int m = 0; m < PT; ++m) {
                    dv[m] = zero4();
#pragma unroll
                    for (int j = 0; j < KS; ++j)
                        dv[m] = M::mma(M::rows(sm.ds + (16 * m + l16) * SK::kStride + 32 * j + 8 * g), kf[j], dv[m]);
                    dv[m] *= down;
                }
            }
            if (!odd) {
                // ---- the wave's tokens as queries: [s][t], s up to t
                {
                    Frag yf[PS], w[2];
#pragma unroll
                    for (int j = 0; j < PS; ++j) yf[j] = M::rows(sm.dy + t * SV::kStride + 32 * j + 8 * g);
#pragma unroll
                    for (int j2 = 0; j2 < 2; ++j2) {
                        Half h2[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int j = 2 * j2 + u;
                            f32x4 x = zero4();
                            if (j <= wave) {
#pragma unroll
                                for (int e = 0; e < PS; ++e)
                                    x = M::mma(M::rows(sm.v + (16 * j + l16) * SV::kStride + 32 * e + 8 * g), yf[e], x);
                                const f32x4 shi = *reinterpret_cast<const f32x4*>(d.hi + 16 * j + 4 * g);
                                const f32x4 slo = *reinterpret_cast<const f32x4*>(d.lo + 16 * j + 4 * g);
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    const float e = exp2_raw((thi - shi[r]) + (tlo - slo[r])) * p.scale;
                                    x[r] = 16 * j + 4 * g + r <= t ? x[r] * e : 0.f;
                                }
                            }
                            // Rounded to the tokens' type, as the weights of the forward: half a step of
                            // each, as large as the gradients' own rounding.
                            h2[u] = M::half(x);
                        }
                        w[j2] = M::cat(h2[0], h2[1]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        dq[n] = M::mma(columns<T>(sm.k + 16 * n, SK::kStride, g, l16), w[0], dq[n]);
                        if (wave >= 2)
                            dq[n] = M::mma(columns<T>(sm.k + 32 * SK::kStride + 16 * n, SK::kStride, g, l16), w[1], dq[n]);
                    }
                }
                // ---- and as keys: [t][s], s the wave's, t from s on
                {
                    Frag vf[PS], kf[KS], wb[2], wa[2];
#pragma unroll
                    for (int j = 0; j < PS; ++j) vf[j] = M::rows(sm.v + t * SV::kStride + 32 * j + 8 * g);
#pragma unroll
                    for (int j = 0; j < KS; ++j) kf[j] = M::rows(sm.k + t * SK::kStride + 32 * j + 8 * g);
#pragma unroll
                    for (int j2 = 0; j2 < 2; ++j2) {
                        Half hb[2], ha[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int j = 2 * j2 + u;
                            f32x4 x = zero4(), y = zero4();
                            if (j >= wave) {
#pragma unroll
                                for (int e = 0; e < PS; ++e)
                                    x = M::mma(M::rows(sm.dy + (16 * j + l16) * SV::kStride + 32 * e + 8 * g), vf[e], x);
#pragma unroll
                                for (int e = 0; e < KS; ++e)
                                    y = M::mma(M::rows(sm.q + (16 * j + l16) * SK::kStride + 32 * e + 8 * g), kf[e], y);
                                const f32x4 qhi = *reinterpret_cast<const f32x4*>(d.hi + 16 * j + 4 * g);
                                const f32x4 qlo = *reinterpret_cast<const f32x4*>(d.lo + 16 * j + 4 * g);
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    const int tt = 16 * j + 4 * g + r;
                                    const float e = exp2_raw((qhi[r] - thi) + (qlo[r] - tlo)) * p.scale;
                                    y[r] = tt >= t ? y[r] * e : 0.f;
                                    const float m = tt > t ? y[r] * x[r] : 0.f;
                                    x[r] = tt >= t ? x[r] * e : 0.f;
                                    rsum[j][r] += m;
                                    asum -= m;
                                }
                            }
                            hb[u] = M::half(x);
                            ha[u] = M::half(y);
                        }
                        wb[j2] = M::cat(hb[0], hb[1]);
                        wa[j2] = M::cat(ha[0], ha[1]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (wave < 2) dk[n] = M::mma(columns<T>(sm.q + 16 * n, SK::kStride, g, l16), wb[0], dk[n]);
                        dk[n] = M::mma(columns<T>(sm.q + 32 * SK::kStride + 16 * n, SK::kStride, g, l16), wb[1], dk[n]);
                    }
#pragma unroll
                    for (int m = 0; m < PT; ++m) {
                        if (wave < 2) dv[m] = M::mma(columns<T>(sm.dy + 16 * m, SV::kStride, g, l16), wa[0], dv[m]);
                        dv[m] = M::mma(columns<T>(sm.dy + 32 * SV::kStride + 16 * m, SV::kStride, g, l16), wa[1], dv[m]);
                    }
                }
            } else {
                // An infinity or a NaN in the tile: pair by pair, each lane its token, so that it
                // meets no weight of 0 of a pair that does not exist.
                for (int s = 0; s < n_in; ++s) {
                    float qk = 0.f, yv = 0.f;   // of the later token's query and dy, the earlier's key and value
                    const int late = s > t ? s : t, early = s > t ? t : s;
                    for (int e = 0; e < N; ++e)
                        qk = fmaf(Elem<T>::load1(sm.q + late * SK::kStride + e), Elem<T>::load1(sm.k + early * SK::kStride + e), qk);
                    for (int e = 0; e < PB; ++e)
                        yv = fmaf(Elem<T>::load1(sm.dy + late * SV::kStride + e), Elem<T>::load1(sm.v + early * SV::kStride + e), yv);
                    const float e = exp2_raw((d.hi[late] - d.hi[early]) + (d.lo[late] - d.lo[early])) * p.scale;
                    const float m = qk * e * yv;
                    if (in && s <= t) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            dq[n] += M::wide(M::four(sm.k + s * SK::kStride + 16 * n + 4 * g)) * (yv * e);
                        if (s < t && g == 0) asum += m;
                    }
                    if (in && s >= t) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            dk[n] += M::wide(M::four(sm.q + s * SK::kStride + 16 * n + 4 * g)) * (yv * e);
#pragma unroll
                        for (int n = 0; n < PT; ++n)
                            dv[n] += M::wide(M::four(sm.dy + s * SV::kStride + 16 * n + 4 * g)) * (qk * e);
                        if (s > t && g == 0) asum -= m;
                    }
                }
            }
            // ---- dv, and with the head's last block dg
            const auto vb = rows_of(static_cast<T*>(o.dv) + at * vrow + (int64_t)h * p.P + p0, n_out, vrow, PB);
#pragma unroll
            for (int m = 0; m < PT; ++m) {
                const uint32_t off = t * (uint32_t)(vrow * sizeof(T)) + (16 * m + 4 * g) * (uint32_t)sizeof(T);
                f32x4 x = dv[m];
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = in ? x[r] : 0.f;
                if constexpr (sizeof(T) == 2)
                    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(vu2, cvt4(x)), vb, off, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(vu4, x), vb, off, 0, 0);
            }
            if (o.dg && head_last) {
                const float a = sum_rows4(in ? asum : 0.f), bs = sum_rows4(in ? bsum : 0.f), cs = wave_sum(cdot);
                if (g == 0) {
                    sm.a[t] = a;
                    sm.b[t] = bs;
                }
                if (lane == 0) sm.c[wave] = cs;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j >= wave) {
                        f32x4 x;
#pragma unroll
                        for (int r = 0; r < 4; ++r) x[r] = row16_sum(rsum[j][r]);
                        if (l16 == 0) *reinterpret_cast<f32x4*>(sm.row[wave] + 16 * j + 4 * g) = x;
                    }
                }
                __syncthreads();
                if (wave == 0) {
                    // Lane l: what counts for token 63 - l, from behind it; what counts for token l, from
                    // before it.  In 64 bits: the rows and columns of M cancel where both lie on one side.
                    const int u = 63 - lane;
                    double x = sm.a[u];
#pragma unroll
                    for (int j = 0; j < 4; ++j) x += 16 * j <= u ? (double)sm.row[j][u] : 0.0;
                    x = wave_running_sum(x);
                    const double y = wave_running_sum(lane > 0 ? (double)sm.b[lane - 1] : 0.0);
                    const double all = (double)d.all * (((double)sm.c[0] + sm.c[1]) + ((double)sm.c[2] + sm.c[3]));
                    const float dg = (float)(x + __shfl(y, u) + all);
                    if (u < n_out) Elem<T>::store1(static_cast<T*>(o.dg) + (at + u) * p.H + h, u < n_in ? dg : 0.f);
                }
            }
        }
        if (n_in == 0) {
            // a padded tile: nothing but zeros
            for (int step = 0; step < steps; ++step) {
                const int h = h_first + step / pblocks, p0 = step % pblocks * PB;
                T* const dvp = static_cast<T*>(o.dv) + at * vrow + (int64_t)h * p.P + p0;
                constexpr int kPer = 16 / (int)sizeof(T);
                for (int e = threadIdx.x; e < n_out * (PB / kPer); e += kLaThreads)
                    *reinterpret_cast<vu4*>(dvp + e / (PB / kPer) * vrow + e % (PB / kPer) * kPer) = vu4{0, 0, 0, 0};
                if (o.dg && p0 == 0 && (int)threadIdx.x < n_out)
                    Elem<T>::store1(static_cast<T*>(o.dg) + (at + threadIdx.x) * p.H + h, 0.f);
            }
        }
        // ---- dq and dk, or this part's sums of them
        const int64_t kat = at * krow + kh * N;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dq[n][r] = in ? dq[n][r] : 0.f;
                dk[n][r] = in ? dk[n][r] : 0.f;
            }
        }
        if (o.split > 1) {
            const int64_t parts = (p.packed ? p.tokens : (int64_t)p.B * p.T) * krow * part;
            const auto qb = rows_of(o.part_q + parts + kat, n_out, krow, N), kb = rows_of(o.part_k + parts + kat, n_out, krow, N);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint32_t off = t * (uint32_t)(krow * 4) + (16 * n + 4 * g) * 4;
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(vu4, dq[n]), qb, off, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(vu4, dk[n]), kb, off, 0, 0);
            }
        } else {
            const auto qb = rows_of(static_cast<T*>(o.dq) + kat, n_out, krow, N), kb = rows_of(static_cast<T*>(o.dk) + kat, n_out, krow, N);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint32_t off = t * (uint32_t)(krow * sizeof(T)) + (16 * n + 4 * g) * (uint32_t)sizeof(T);
                if constexpr (sizeof(T) == 2) {
                    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(vu2, cvt4(dq[n])), qb, off, 0, 0);
                    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(vu2, cvt4(dk[n])), kb, off, 0, 0);
                } else {
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(vu4, dq[n]), qb, off, 0, 0);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(vu4, dk[n]), kb, off, 0, 0);
                }
            }
        }
    }
}

// dq and dk: the sums over the parts of a group's heads, in order.  Four values a thread;
// the second half of the grid takes dk.  Places of a packed tensor that no row covers hold
// no sums and stay as they are.
template <typename T>
__global__ __launch_bounds__(256) void la_parts_kernel(const LaBwdArgs o, int64_t values, unsigned half) {
    const LaArgs& p = o.f;
    const bool second = blockIdx.x >= half;
    const int64_t e = ((int64_t)(blockIdx.x - (second ? half : 0)) * 256 + threadIdx.x) * 4;
    if (e >= values) return;
    if (p.packed) {
        const int64_t token = e / ((int64_t)p.G * p.N);
        bool some = false;
        for (int b = 0; b < p.B && !some; ++b) {
            const LaRow row = la_row(p.rows, true, p.tokens, p.T, b);
            some = token >= row.first && token < row.first + row.len;
        }
        if (!some) return;
    }
    const float* const from = (second ? o.part_k : o.part_q) + e;
    f32x4 x = *reinterpret_cast<const f32x4*>(from);
    for (int i = 1; i < o.split; ++i) x += *reinterpret_cast<const f32x4*>(from + i * values);
    Elem<T>::store4(static_cast<T*>(second ? o.dk : o.dq) + e, make_float4(x[0], x[1], x[2], x[3]));
}

template <typename T, int N, int PB>
hipError_t bwd_block(const LaBwdArgs& q, hipStream_t stream) {
    const LaArgs& p = q.f;
    hipError_t e = launch_la_adjoint(q, stream);
    if (e != hipSuccess) return e;
    const int blocks = p.T > 0 ? (int)(((int64_t)p.T + kLaChunk - 1) / kLaChunk) : 1;
    la_bwd_kernel<T, N, PB><<<(unsigned)p.B * blocks * p.G * q.split, kLaThreads, 0, stream>>>(q, blocks);
    if ((e = hipGetLastError()) != hipSuccess || q.split == 1) return e;
    const int64_t values = (p.packed ? p.tokens : (int64_t)p.B * p.T) * p.G * N;
    const unsigned half = (unsigned)((values / 4 + 255) / 256);
    la_parts_kernel<T><<<2 * half, 256, 0, stream>>>(q, values, half);
    return hipGetLastError();
}

// Value rows at a time: 64, where the tiles of 64 fit a unit's LDS (not fp32 at N = 128).
template <typename T, int N>
hipError_t bwd_n(const LaBwdArgs& q, hipStream_t stream) {
    if constexpr (sizeof(T) == 4 && N == 128) return bwd_block<T, N, 32>(q, stream);
    else return q.f.P < 64 ? bwd_block<T, N, 32>(q, stream) : bwd_block<T, N, 64>(q, stream);
}

template <typename T>
hipError_t bwd_t(const LaBwdArgs& q, hipStream_t stream) {
    switch (q.f.N) {
        case 32: return bwd_n<T, 32>(q, stream);
        case 64: return bwd_n<T, 64>(q, stream);
        case 128: return bwd_n<T, 128>(q, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_la_backward(const LaBwdArgs& q, hipStream_t stream) {
    return q.f.bf16 ? bwd_t<bf16_t>(q, stream) : bwd_t<float>(q, stream);
}

}  // namespace wkv7
