// wkv7_gnorm.hip -- the group norm over channels last with an activation and a
// gate, forward (formulas and layout in wkv7_gnorm_device.h).

#include "wkv7_gnorm_device.h"
#include "wkv7_gnorm_dispatch.h"

namespace wkv7 {

namespace {

template <typename T, int V, int P, int K, int kGate, bool kSilu>
__global__ __launch_bounds__(512) void gn_fwd_kernel(const GnArgs p) {
    __shared__ float s_sum[8];
    const GnPlace<P> at(p);
    const float inv = 1.f / p.W;
    const int64_t stride = (int64_t)p.plan.parts * p.plan.rows;
    const int64_t loops = (p.rows + stride - 1) / stride;
    for (int64_t l = 0; l < loops; ++l) {
        const int64_t row = l * stride + at.side;
        const bool live = at.live && row < p.rows;
        const int64_t base = (live ? row : 0) * p.D + (int64_t)at.group * p.W;
        GnPiece<T, V> x[K], z[K];
        float u[K][V], sum = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * P + at.lane) * V;
            x[k].load(static_cast<const T*>(p.x) + base + c, live && c < p.W);
            z[k].load(static_cast<const T*>(p.z) + base + c, kGate != 0 && live && c < p.W);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                u[k][i] = x[k].get(i);
                if constexpr (kGate == 2) u[k][i] *= silu(z[k].get(i));
                sum += u[k][i];
            }
        const float mean = p.center ? gn_sum<P>(sum, s_sum) * inv : 0.f;
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (k * P + at.lane) * V + i;
                u[k][i] = c < p.W ? u[k][i] - mean : 0.f;
                sum = fmaf(u[k][i], u[k][i], sum);
            }
        const float rstd = rsqrtf(fmaf(gn_sum<P>(sum, s_sum), inv, p.eps));
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * P + at.lane) * V;
            if (!live || c >= p.W) continue;
            float g[V], b[V], y[V];
            gn_vector<V>(p.gamma ? p.gamma + at.group * p.W + c : nullptr, true, 1.f, g);
            gn_vector<V>(p.beta ? p.beta + at.group * p.W + c : nullptr, true, 0.f, b);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                y[i] = fmaf(u[k][i] * rstd, g[i], b[i]);
                if constexpr (kSilu) y[i] = silu(y[i]);
                if constexpr (kGate == 1) y[i] *= silu(z[k].get(i));
            }
            store_piece<V>(static_cast<T*>(p.y) + base, c, p.W, y);
        }
    }
}

// Groups too wide for registers: a workgroup reads one again for each of its sums.
template <typename T, int V, int kGate, bool kSilu>
__global__ __launch_bounds__(256) void gn_fwd_wide_kernel(const GnArgs p) {
    constexpr int P = 256;
    __shared__ float s_sum[8];
    const GnPlace<P> at(p);
    const float inv = 1.f / p.W;
    for (int64_t row = at.side; row < p.rows; row += p.plan.parts) {
        const int64_t base = row * p.D + (int64_t)at.group * p.W;
        const T* const X = static_cast<const T*>(p.x) + base;
        const T* const Z = static_cast<const T*>(p.z) + base;
        auto value = [&](int c, float (&u)[V], GnPiece<T, V>& z) {
            GnPiece<T, V> x;
            x.load(X + c, true);
            z.load(Z + c, kGate != 0);
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] = kGate == 2 ? x.get(i) * silu(z.get(i)) : x.get(i);
        };
        float u[V], sum = 0.f;
        GnPiece<T, V> z;
        for (int c = at.lane * V; c < p.W; c += P * V) {
            value(c, u, z);
#pragma unroll
            for (int i = 0; i < V; ++i) sum += u[i];
        }
        const float mean = p.center ? gn_sum<P>(sum, s_sum) * inv : 0.f;
        sum = 0.f;
        for (int c = at.lane * V; c < p.W; c += P * V) {
            value(c, u, z);
#pragma unroll
            for (int i = 0; i < V; ++i) sum = fmaf(u[i] - mean, u[i] - mean, sum);
        }
        const float rstd = rsqrtf(fmaf(gn_sum<P>(sum, s_sum), inv, p.eps));
        for (int c = at.lane * V; c < p.W; c += P * V) {
            value(c, u, z);
            float g[V], b[V], y[V];
            gn_vector<V>(p.gamma ? p.gamma + (int64_t)at.group * p.W + c : nullptr, true, 1.f, g);
            gn_vector<V>(p.beta ? p.beta + (int64_t)at.group * p.W + c : nullptr, true, 0.f, b);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                y[i] = fmaf((u[i] - mean) * rstd, g[i], b[i]);
                if constexpr (kSilu) y[i] = silu(y[i]);
                if constexpr (kGate == 1) y[i] *= silu(z.get(i));
            }
            store_piece<V>(static_cast<T*>(p.y) + base, c, p.W, y);
        }
    }
}

template <typename T, int V, int P, int K, int kGate, bool kSilu>
hipError_t run(const GnArgs& p, hipStream_t stream) {
    const unsigned grid = p.plan.blocks * p.plan.parts;
    if constexpr (K == 0) gn_fwd_wide_kernel<T, V, kGate, kSilu><<<grid, 256, 0, stream>>>(p);
    else gn_fwd_kernel<T, V, P, K, kGate, kSilu><<<grid, p.plan.threads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gnorm_forward(const GnArgs& p, hipStream_t stream) {
    if (p.bf16) {
        WKV7_GN_BF16
    } else {
        WKV7_GN_F32
    }
    return hipErrorInvalidValue;
}

hipError_t launch_gnorm_backward(const GnArgs& p, hipStream_t stream) {
    return p.bf16 ? launch_gnorm_backward_bf16(p, stream) : launch_gnorm_backward_f32(p, stream);
}

}  // namespace wkv7
