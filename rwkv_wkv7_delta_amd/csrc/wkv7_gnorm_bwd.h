// wkv7_gnorm_bwd.h -- gradients of the group norm (formulas and layout in
// wkv7_gnorm_device.h), for the translation unit of each token type.
//
// With e the gradient of o (dy through the gate and the activation):
//   dgamma = sum e n,  dbeta = sum e (over the rows)
//   du = (f - n mean(f n) - mean f) / sqrt(var + eps),  f = gamma e
//   (mean f only where the mean was taken off)
//   dx, dz from du through the product with z sigmoid(z), or dz from dy.
// The moments are formed again from x: a second tensor of them would cost more bytes
// than the sums do time.  16384 rows of 2048 in one group, gate in front, without centring,
// bf16: 88 us, 3.8 TB/s, and 10 us for the parameters' sums; with centring 5 us more.  Two sums
// over a row, one after the other (with centring four), 213 registers a lane (two waves on a
// SIMD).  fp32: 140 us in all, 4.8 TB/s.

#pragma once

#include "wkv7_gnorm_device.h"
#include "wkv7_gnorm_dispatch.h"

namespace wkv7 {

namespace {

// What one channel needs once n is known: e, and its product with gamma.
// (q: sigmoid(z)).
template <int kGate, bool kSilu>
struct GnBack {
    float e, dgate;
    __device__ __forceinline__ GnBack(float n, float gamma, float beta, float z, float q, float dy) {
        e = dy;
        dgate = 0.f;
        if constexpr (kGate == 1 || kSilu) {
            const float o = fmaf(n, gamma, beta);
            const float a = kSilu ? sigmoid(o) : 1.f;
            if constexpr (kGate == 1) {
                dgate = dy * (o * a);
                e *= z * q;
            }
            if constexpr (kSilu) e *= a * fmaf(o, 1.f - a, 1.f);
        }
    }
};
// The gradient of z from that of z sigmoid(z), q = sigmoid(z).
__device__ __forceinline__ float gn_dz(float dgate, float z, float q) { return dgate * q * fmaf(z, 1.f - q, 1.f); }

template <typename T, int V, int P, int K, int kGate, bool kSilu>
__global__ __launch_bounds__(512) void gn_bwd_kernel(const GnArgs p) {
    constexpr int kBatch = 8;   // sums of a lane that meet in LDS at a time
    __shared__ float s_sum[8];
    __shared__ float s_part[kBatch][512];
    const GnPlace<P> at(p);
    const float inv = 1.f / p.W;
    const int64_t stride = (int64_t)p.plan.parts * p.plan.rows;
    const int64_t loops = (p.rows + stride - 1) / stride;
    float dg[K][V], db[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) dg[k][i] = db[k][i] = 0.f;
    // The next row is on its way while one is worked on.
    GnPiece<T, V> x1[K], z1[K], y1[K];
    auto load = [&](int64_t l) {
        const int64_t row = l * stride + at.side;
        const bool live = at.live && row < p.rows;
        const int64_t base = (live ? row : 0) * p.D + (int64_t)at.group * p.W;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * P + at.lane) * V;
            x1[k].load(static_cast<const T*>(p.x) + base + c, live && c < p.W);
            if constexpr (kGate != 0) z1[k].load(static_cast<const T*>(p.z) + base + c, live && c < p.W);
            y1[k].load(static_cast<const T*>(p.dy) + base + c, live && c < p.W);
        }
    };
    load(0);
    for (int64_t l = 0; l < loops; ++l) {
        const int64_t row = l * stride + at.side;
        const bool live = at.live && row < p.rows;
        const int64_t base = (live ? row : 0) * p.D + (int64_t)at.group * p.W;
        GnPiece<T, V> x[K], z[K], dy[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k] = x1[k];
            if constexpr (kGate != 0) z[k] = z1[k];
            dy[k] = y1[k];
        }
        load(l + 1);
        float n[K][V], f[K][V], q[K][V], dgate[K][V], sum = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                n[k][i] = x[k].get(i);
                if constexpr (kGate != 0) q[k][i] = sigmoid(z[k].get(i));
                if constexpr (kGate == 2) n[k][i] *= z[k].get(i) * q[k][i];
                sum += n[k][i];
            }
        const float mean = p.center ? gn_sum<P>(sum, s_sum) * inv : 0.f;
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                n[k][i] = (k * P + at.lane) * V + i < p.W ? n[k][i] - mean : 0.f;
                sum = fmaf(n[k][i], n[k][i], sum);
            }
        const float rstd = rsqrtf(fmaf(gn_sum<P>(sum, s_sum), inv, p.eps));
        float sf = 0.f, sfn = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * P + at.lane) * V;
            float g[V], b[V];
            gn_vector<V>(p.gamma ? p.gamma + at.group * p.W + c : nullptr, c < p.W, 1.f, g);
            if constexpr (kGate == 1 || kSilu)
                gn_vector<V>(p.beta ? p.beta + at.group * p.W + c : nullptr, c < p.W, 0.f, b);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                n[k][i] *= rstd;
                const GnBack<kGate, kSilu> r(n[k][i], g[i], kGate == 1 || kSilu ? b[i] : 0.f, kGate ? z[k].get(i) : 0.f,
                                             kGate ? q[k][i] : 0.f, dy[k].get(i));
                dgate[k][i] = r.dgate;
                dg[k][i] = live ? fmaf(r.e, n[k][i], dg[k][i]) : dg[k][i];
                db[k][i] = live ? db[k][i] + r.e : db[k][i];
                f[k][i] = r.e * g[i];
                sf += f[k][i];
                sfn = fmaf(f[k][i], n[k][i], sfn);
            }
        }
        sf = p.center ? gn_sum<P>(sf, s_sum) * inv : 0.f;
        sfn = gn_sum<P>(sfn, s_sum) * inv;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * P + at.lane) * V;
            if (!live || c >= p.W) continue;
            float dx[V], dz[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dx[i] = rstd * (f[k][i] - fmaf(n[k][i], sfn, sf));
                if constexpr (kGate != 0) {
                    const float zz = z[k].get(i);
                    dz[i] = gn_dz(kGate == 2 ? dx[i] * x[k].get(i) : dgate[k][i], zz, q[k][i]);
                    if constexpr (kGate == 2) dx[i] *= zz * q[k][i];
                }
            }
            store_piece<V>(static_cast<T*>(p.dx) + base, c, p.W, dx);
            if constexpr (kGate != 0) store_piece<V>(static_cast<T*>(p.dz) + base, c, p.W, dz);
        }
    }
    if (!p.part) return;
    // The rows side by side meet in LDS, in order; the workgroup leaves one partial row.
    const int ring = p.plan.groups * P;   // lanes of one of these rows
    float* const to = p.part + (size_t)(blockIdx.x / p.plan.blocks) * 2 * p.D + at.group * p.W;
    constexpr int kSums = 2 * K * V;
#pragma unroll
    for (int s0 = 0; s0 < kSums; s0 += kBatch) {
        __syncthreads();
#pragma unroll
        for (int s = s0; s < kSums && s < s0 + kBatch; ++s)
            s_part[s - s0][threadIdx.x] = s < K * V ? dg[s / V % K][s % V] : db[s / V % K][s % V];
        __syncthreads();
        if (at.live && at.row == 0) {
#pragma unroll
            for (int s = s0; s < kSums && s < s0 + kBatch; ++s) {
                const int c = (s / V % K * P + at.lane) * V + s % V;
                float sum = 0.f;
                for (int r = 0; r < p.plan.rows; ++r) sum += s_part[s - s0][threadIdx.x + r * ring];
                if (c < p.W) to[(s < K * V ? 0 : p.D) + c] = sum;
            }
        }
    }
}

template <typename T, int V, int kGate, bool kSilu>
__global__ __launch_bounds__(256) void gn_bwd_wide_kernel(const GnArgs p) {
    constexpr int P = 256;
    __shared__ float s_sum[8];
    const GnPlace<P> at(p);
    const float inv = 1.f / p.W;
    bool first = true;
    for (int64_t row = at.side; row < p.rows; row += p.plan.parts, first = false) {
        const int64_t base = row * p.D + (int64_t)at.group * p.W;
        auto value = [&](int c, float (&u)[V], GnPiece<T, V>& x, GnPiece<T, V>& z) {
            x.load(static_cast<const T*>(p.x) + base + c, true);
            z.load(static_cast<const T*>(p.z) + base + c, kGate != 0);
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] = kGate == 2 ? x.get(i) * silu(z.get(i)) : x.get(i);
        };
        float u[V], sum = 0.f;
        GnPiece<T, V> x, z, dy;
        for (int c = at.lane * V; c < p.W; c += P * V) {
            value(c, u, x, z);
#pragma unroll
            for (int i = 0; i < V; ++i) sum += u[i];
        }
        const float mean = p.center ? gn_sum<P>(sum, s_sum) * inv : 0.f;
        sum = 0.f;
        for (int c = at.lane * V; c < p.W; c += P * V) {
            value(c, u, x, z);
#pragma unroll
            for (int i = 0; i < V; ++i) sum = fmaf(u[i] - mean, u[i] - mean, sum);
        }
        const float rstd = rsqrtf(fmaf(gn_sum<P>(sum, s_sum), inv, p.eps));
        float sf = 0.f, sfn = 0.f;
        for (int c = at.lane * V; c < p.W; c += P * V) {
            value(c, u, x, z);
            dy.load(static_cast<const T*>(p.dy) + base + c, true);
            float g[V], b[V];
            gn_vector<V>(p.gamma ? p.gamma + (int64_t)at.group * p.W + c : nullptr, true, 1.f, g);
            gn_vector<V>(p.beta ? p.beta + (int64_t)at.group * p.W + c : nullptr, true, 0.f, b);
            float* const to = p.part ? p.part + (size_t)at.side * 2 * p.D + (int64_t)at.group * p.W + c : nullptr;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = (u[i] - mean) * rstd;
                const GnBack<kGate, kSilu> r(n, g[i], b[i], z.get(i), sigmoid(z.get(i)), dy.get(i));
                if (to) {   // this thread's channels in every row
                    to[i] = first ? r.e * n : fmaf(r.e, n, to[i]);
                    to[p.D + i] = first ? r.e : to[p.D + i] + r.e;
                }
                sf = fmaf(r.e, g[i], sf);
                sfn = fmaf(r.e * g[i], n, sfn);
            }
        }
        sf = p.center ? gn_sum<P>(sf, s_sum) * inv : 0.f;
        sfn = gn_sum<P>(sfn, s_sum) * inv;
        for (int c = at.lane * V; c < p.W; c += P * V) {
            value(c, u, x, z);
            dy.load(static_cast<const T*>(p.dy) + base + c, true);
            float g[V], b[V], dx[V], dz[V];
            gn_vector<V>(p.gamma ? p.gamma + (int64_t)at.group * p.W + c : nullptr, true, 1.f, g);
            gn_vector<V>(p.beta ? p.beta + (int64_t)at.group * p.W + c : nullptr, true, 0.f, b);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = (u[i] - mean) * rstd;
                const GnBack<kGate, kSilu> r(n, g[i], b[i], z.get(i), sigmoid(z.get(i)), dy.get(i));
                dx[i] = rstd * (r.e * g[i] - fmaf(n, sfn, sf));
                if constexpr (kGate != 0) {
                    dz[i] = gn_dz(kGate == 2 ? dx[i] * x.get(i) : r.dgate, z.get(i), sigmoid(z.get(i)));
                    if constexpr (kGate == 2) dx[i] *= silu(z.get(i));
                }
            }
            store_piece<V>(static_cast<T*>(p.dx) + base, c, p.W, dx);
            if constexpr (kGate != 0) store_piece<V>(static_cast<T*>(p.dz) + base, c, p.W, dz);
        }
    }
}

// dgamma and dbeta: the sums over the parts, in order; 16 channels of either by 16 lanes
// of parts a workgroup.
__global__ __launch_bounds__(256) void gn_params_kernel(const GnArgs p, int64_t sides) {
    __shared__ float s_sum[16][17];
    const int l = threadIdx.x % 16, k = threadIdx.x / 16;
    const int64_t c = (int64_t)blockIdx.x * 16 + l, all = 2 * (int64_t)p.D;
    float s = 0.f;
    if (c < all)
        for (int64_t i = k; i < sides; i += 16) s += p.part[i * all + c];
    s_sum[k][l] = s;
    __syncthreads();
    if (k == 0 && c < all) {
        for (int i = 1; i < 16; ++i) s += s_sum[i][l];
        float* const to = c < p.D ? p.dgamma : p.dbeta;
        if (to) to[c < p.D ? c : c - p.D] = s;
    }
}

template <typename T, int V, int P, int K, int kGate, bool kSilu>
hipError_t run(const GnArgs& p, hipStream_t stream) {
    const unsigned grid = p.plan.blocks * p.plan.parts;
    if (p.rows > 0) {
        if constexpr (K == 0) gn_bwd_wide_kernel<T, V, kGate, kSilu><<<grid, 256, 0, stream>>>(p);
        else gn_bwd_kernel<T, V, P, K, kGate, kSilu><<<grid, p.plan.threads, 0, stream>>>(p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!p.part) return hipSuccess;
    gn_params_kernel<<<(unsigned)((2 * (int64_t)p.D + 15) / 16), 256, 0, stream>>>(p, p.rows > 0 ? p.plan.parts : 0);
    return hipGetLastError();
}

}  // namespace

}  // namespace wkv7
