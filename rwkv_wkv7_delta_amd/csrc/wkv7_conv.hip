// wkv7_conv.hip -- the short causal convolution along a sequence: prompts
// (forward), gradients, single tokens.
//
// Per channel d with W = 2, 3 or 4 taps:
//   pre_t = bias + sum_k weight[d][k] x_{t-(W-1)+k},   y_t = pre_t, or pre_t sigmoid(pre_t)
// with the W - 1 inputs before the first token from a state (zero without one);
// the state behind the sequence is its last W - 1 inputs.  W = 2 without the
// activation is a token shift (each channel mixes the previous token in).
//
// Bound by HBM: every kernel reads each token tensor once and writes each
// output once.  A thread owns a few neighbouring channels (16 bytes of a row
// where the width allows; rows of other widths element by element) and steps
// along a run of tokens with the last W - 1 inputs in registers, so that a
// token row is read by one run only, but for the W - 1 rows before a run.
// fp32 arithmetic, outputs rounded once.
//
// (8, 4096) tokens of 2560 channels, bf16, two taps: 74 us, 4.5 TB/s (a copy of
// 1 GiB reaches 5.1); (5, 1021) tokens of 1001 channels, fp32, four taps, one
// channel per lane: 12 us.

#include "wkv7_ssm_device.h"
#include "wkv7_ssm_internal.h"

namespace wkv7 {

namespace {

constexpr int kConvThreads = 256;

struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};

// Weights of the thread's channels, transposed to taps; zero behind the width.
template <int W, int V>
__device__ __forceinline__ void load_weights(const ConvArgs& p, int c, float (&w)[W][V], float (&bias)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const bool in = c + i < p.D;
        const size_t at = (size_t)(in ? c + i : 0);
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][i] = in ? p.weight[at * W + k] : 0.f;
        bias[i] = in && p.bias ? p.bias[at] : 0.f;
    }
}

// Input number t of batch row b (t in [1 - W, T)): the state before the first
// token.  The loaded piece holds valid memory's values for any t in that range.
template <typename T, int W, int V>
__device__ __forceinline__ void load_input(const ConvArgs& p, int b, int t, int c, Piece<T, V, true>& r, bool& zero) {
    const T* const X = static_cast<const T*>(p.x);
    const T* const S0 = static_cast<const T*>(p.s0);
    zero = t < 0 && !S0;
    if (t >= 0 || !S0) {
        r.load(X + ((size_t)b * p.T + (t > 0 ? t : 0)) * p.D, c, p.D);
    } else {
        r.load(S0 + ((size_t)b * (W - 1) + (t + W - 1)) * p.D, c, p.D);
    }
}

// The state behind each row: its last W - 1 inputs, copied, element `id` of
// [B][W - 1][D].
template <typename T, int W>
__device__ __forceinline__ void copy_state(const ConvArgs& p, int64_t id) {
    if (id >= (int64_t)p.B * (W - 1) * p.D) return;
    const int c = (int)(id % p.D);
    const int k = (int)(id / p.D % (W - 1)), b = (int)(id / p.D / (W - 1));
    const int t = row_length(p.lengths, b, p.T) - (W - 1) + k;
    T v = 0;
    if (t >= 0) v = static_cast<const T*>(p.x)[((size_t)b * p.T + t) * p.D + c];
    else if (p.s0) v = static_cast<const T*>(p.s0)[((size_t)b * (W - 1) + t + W - 1) * p.D + c];
    static_cast<T*>(p.sT)[id] = v;
}

// Workgroups from `runs_end` on copy the state: a launch of its own for that took
// 4 us more.
template <typename T, int W, int V>
__global__ __launch_bounds__(kConvThreads) void conv_fwd_kernel(const ConvArgs p, unsigned cols, unsigned runs,
                                                               int run, unsigned items, unsigned runs_end) {
    if (blockIdx.x >= runs_end) {
        copy_state<T, W>(p, (int64_t)(blockIdx.x - runs_end) * kConvThreads + threadIdx.x);
        return;
    }
    const unsigned id = blockIdx.x * kConvThreads + threadIdx.x;
    if (id >= items) return;
    const unsigned rr = id / cols;
    const int c = (int)(id % cols) * V;
    const int b = (int)(rr / runs), t0 = (int)(rr % runs) * run;
    const int t1 = t0 + run < p.T ? t0 + run : p.T;
    const int len = row_length(p.lengths, b, p.T);
    float w[W][V], bias[V], hist[W - 1][V];
    load_weights<W, V>(p, c, w, bias);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        Piece<T, V, true> r;
        bool zero;
        load_input<T, W, V>(p, b, t0 - (W - 1) + k, c, r, zero);
        const bool keep = !zero && t0 - (W - 1) + k < len;
#pragma unroll
        for (int i = 0; i < V; ++i) hist[k][i] = keep ? r.get(i) : 0.f;
    }
    const T* xp = static_cast<const T*>(p.x) + ((size_t)b * p.T + t0) * p.D;
    T* yp = static_cast<T*>(p.y) + ((size_t)b * p.T + t0) * p.D;
    constexpr int U = 4;   // rows loaded together
    for (int t = t0; t < t1; t += U) {
        Piece<T, V, true> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            r[u].load(xp + (size_t)(t + u < t1 ? u : t1 - 1 - t) * p.D, c, p.D);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u < t1) {
                const bool in = t + u < len;
                float out[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float x = r[u].get(i);
                    float pre = bias[i];
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) pre = fmaf(w[k][i], hist[k][i], pre);
                    pre = fmaf(w[W - 1][i], x, pre);
#pragma unroll
                    for (int k = 0; k + 1 < W - 1; ++k) hist[k][i] = hist[k + 1][i];
                    hist[W - 2][i] = x;
                    if (p.silu) pre *= sigmoid(pre);
                    out[i] = in ? pre : 0.f;
                }
                store_piece(yp + (size_t)u * p.D, c, p.D, out);
            }
        }
        xp += (size_t)U * p.D;
        yp += (size_t)U * p.D;
    }
}

// One token: y from the state and the input, the state moved on in place.
template <typename T, int W, int V>
__global__ __launch_bounds__(kConvThreads) void conv_step_kernel(const ConvArgs p, unsigned cols, unsigned items) {
    const unsigned id = blockIdx.x * kConvThreads + threadIdx.x;
    if (id >= items) return;
    const int c = (int)(id % cols) * V;
    const size_t b = id / cols;
    float w[W][V], bias[V], in[W][V], out[V];
    Piece<T, V, true> r[W];
    T* const S = static_cast<T*>(p.sT) + b * (W - 1) * p.D;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) r[k].load(S + (size_t)k * p.D, c, p.D);
    r[W - 1].load(static_cast<const T*>(p.x) + b * p.D, c, p.D);
    load_weights<W, V>(p, c, w, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float pre = bias[i];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            in[k][i] = r[k].get(i);
            pre = fmaf(w[k][i], in[k][i], pre);
        }
        out[i] = p.silu ? pre * sigmoid(pre) : pre;
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_piece(S + (size_t)k * p.D, c, p.D, in[k + 1]);
    store_piece(static_cast<T*>(p.y) + b * p.D, c, p.D, out);
}

// Gradients.  e_t = dy_t, times the activation's slope at pre_t:
//   dx_t = sum_k weight[k] e_{t+(W-1)-k} (+ dsT where x_t is in the last state)
//   dweight[k] = sum_t e_t x_{t-(W-1)+k},   dbias = sum_t e_t
// A wave takes 64 column pieces of one run of tokens, a workgroup four runs; a
// run steps W - 1 tokens past its end for the e that its last dx need, and the
// first run of a row gives ds0.  x and dy are read through buffers that end
// with the row's length (what is behind reads as 0, so e and dx there come out
// as 0), dx is written through one that holds the run's tokens: the loop has no
// condition per token.  (4, 4096) tokens of 2048 channels, bf16, four taps: 48 us,
// 4.2 TB/s, with four channels a lane and about 2048 waves (4096: 50 us; two
// channels a lane: 51 to 55 us).  The sums over a run stay in registers; the workgroup's
// four meet in LDS, the workgroups in a second kernel, in a fixed order.
template <typename T, int W, int V, bool kSilu>
__global__ __launch_bounds__(kConvThreads) void conv_bwd_kernel(const ConvBwdArgs q, unsigned cblocks, int runs) {
    constexpr int R = kConvThreads / 64, M = W + 1, H = W - 1, U = 4;
    __shared__ float s_part[R][M][64 * V];
    const ConvArgs& p = q.f;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const unsigned cb = blockIdx.x % cblocks, part = blockIdx.x / cblocks;
    const int c = (int)(cb * 64 + lane) * V;
    const int64_t r0 = (int64_t)part * R + wave;
    float w[W][V], bias[V], dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][i] = 0.f;
    }
    if (r0 < (int64_t)p.B * runs) {
        const int b = (int)(r0 / runs), rr = (int)(r0 % runs);
        const int t0 = rr * q.run, t1 = t0 + q.run < p.T ? t0 + q.run : p.T;
        const int len = row_length(p.lengths, b, p.T);
        load_weights<W, V>(p, c, w, bias);
        const int64_t row = (int64_t)p.D * (int)sizeof(T), base = ((int64_t)b * p.T + t0) * row;
        const int ahead = t1 + H < len ? t1 + H : len;   // the last input that is needed
        const int bytes = ahead > t0 ? (int)((ahead - t0) * row) : 0;
        const __amdgpu_buffer_rsrc_t x_rows = buffer_of(static_cast<const char*>(p.x) + base, bytes),
                                     dy_rows = buffer_of(static_cast<const char*>(q.dy) + base, bytes),
                                     dx_rows = buffer_of(static_cast<char*>(q.dx) + base, (int)((t1 - t0) * row));
        const bool dead = c >= p.D;
        const uint32_t step = dead ? 0 : (uint32_t)row;
        uint32_t at = dead ? kNowhere : c * (uint32_t)sizeof(T);
        // x and e of the W - 1 tokens before the group's, then the group's.
        float xw[H + U][V], ew[H + U][V];
#pragma unroll
        for (int k = 0; k < H; ++k) {
            Piece<T, V, true> r;
            bool zero;
            load_input<T, W, V>(p, b, t0 - H + k, c, r, zero);
            const bool keep = !zero && t0 - H + k < len;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                xw[k][i] = keep ? r.get(i) : 0.f;
                ew[k][i] = 0.f;
            }
        }
        const int inner = t1 < len ? t1 : len;   // the run's own tokens end here
        // A group of U tokens from t on; edge: some lie outside the run, or give
        // gradients of a state.
        auto group = [&](int t, auto edge_) {
            constexpr bool kEdge = decltype(edge_)::value;
            Piece<T, V, true> rx[U], ry[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                rx[u].load(x_rows, at + u * step);
                ry[u].load(dy_rows, at + u * step);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float g[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float x = rx[u].get(i);
                    float e = ry[u].get(i);
                    xw[H + u][i] = x;
                    if constexpr (kSilu) {
                        float pre = bias[i];
#pragma unroll
                        for (int k = 0; k < W; ++k) pre = fmaf(w[k][i], xw[u + k][i], pre);
                        const float s = sigmoid(pre);
                        e *= s * fmaf(pre, 1.f - s, 1.f);
                        // 0 behind the row's last token, whatever the taps make of its last inputs
                        if constexpr (kEdge) e = t + u < len ? e : 0.f;
                    }
                    ew[H + u][i] = e;
                    const bool own = !kEdge || t + u < inner;
#pragma unroll
                    for (int k = 0; k < W; ++k) dw[k][i] = own ? fmaf(e, xw[u + k][i], dw[k][i]) : dw[k][i];
                    db[i] += own ? e : 0.f;
                    // input t + u - (W-1) meets tap W-1 at its own token, tap 0 here
                    g[i] = w[0][i] * e;
#pragma unroll
                    for (int k = 0; k < H; ++k) g[i] = fmaf(w[H - k][i], ew[u + k][i], g[i]);
                }
                const int src = t + u - H;
                if constexpr (kEdge) {
                    const int k = src - (len - H);   // in the last state
                    if (q.dsT && k >= 0 && src < len && !dead) {
                        Piece<T, V, true> r;
                        r.load(static_cast<const T*>(q.dsT) + ((size_t)b * H + k) * p.D, c, p.D);
#pragma unroll
                        for (int i = 0; i < V; ++i) g[i] += r.get(i);
                    }
                    if (src < 0 && q.ds0)
                        store_piece(static_cast<T*>(q.ds0) + ((size_t)b * H + src + H) * p.D, c, p.D, g);
                }
                // inputs before the run's lie below the buffer's start: dropped
                store_piece<T, true>(dx_rows, at + u * step - H * step, 1, g);
            }
#pragma unroll
            for (int k = 0; k < H; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    xw[k][i] = xw[U + k][i];
                    ew[k][i] = ew[U + k][i];
                }
            at += U * step;
        };
        int t = t0;
        if (rr == 0) {
            group(t, Yes());
            t += U;
        }
        for (; t + U <= inner; t += U) group(t, No());
        for (; t < t1 + H; t += U) group(t, Yes());
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) s_part[wave][k][lane * V + i] = dw[k][i];
        s_part[wave][W][lane * V + i] = db[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 64 * V * M; e += kConvThreads) {
        const int cc = e / M, k = e % M;
        const int ch = (int)(cb * 64 * V) + cc;
        if (ch < p.D) {
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) s += s_part[r][k][cc];
            q.part[((size_t)part * p.D + ch) * M + k] = s;
        }
    }
}

// dweight and dbias: the sum over the parts, in order.  A workgroup takes 16
// elements of [D][W + 1], 16 lanes of parts each.
template <int W>
__global__ __launch_bounds__(256) void conv_params_kernel(const float* __restrict__ part, int parts, int D,
                                                          float* dweight, float* dbias) {
    constexpr int M = W + 1;
    __shared__ float s_sum[16][17];
    const size_t total = (size_t)D * M;
    const int l = threadIdx.x % 16, k = threadIdx.x / 16;
    const size_t e = (size_t)blockIdx.x * 16 + l;
    float s = 0.f;
    if (e < total)
        for (int i = k; i < parts; i += 16) s += part[i * total + e];
    s_sum[k][l] = s;
    __syncthreads();
    if (k == 0 && e < total) {
        for (int i = 1; i < 16; ++i) s += s_sum[i][l];
        const size_t c = e / M, t = e % M;
        if (t < W) dweight[c * W + t] = s;
        else if (dbias) dbias[c] = s;
    }
}

// Tokens of a forward run.  8, 16 and 32 for the two shapes named at the top: 74.5,
// 73.9, 72.3 us and 11.8, 12.0, 15.1 us.
constexpr int kRun = 16;

template <typename T, int W, int V>
hipError_t fwd_v(const ConvArgs& p, hipStream_t stream) {
    const unsigned cols = (unsigned)((p.D + V - 1) / V), runs = (unsigned)((p.T + kRun - 1) / kRun);
    const uint64_t items = (uint64_t)cols * runs * p.B;
    const uint64_t states = p.sT ? (uint64_t)p.B * (W - 1) * p.D : 0;
    if (items > (1ull << 31) || states > (1ull << 31)) return hipErrorInvalidValue;
    const unsigned runs_end = (unsigned)((items + kConvThreads - 1) / kConvThreads);
    const unsigned grid = runs_end + (unsigned)((states + kConvThreads - 1) / kConvThreads);
    if (grid == 0) return hipSuccess;
    conv_fwd_kernel<T, W, V><<<grid, kConvThreads, 0, stream>>>(p, cols, runs, kRun, (unsigned)items, runs_end);
    return hipGetLastError();
}

template <typename T, int W, int V>
hipError_t step_v(const ConvArgs& p, hipStream_t stream) {
    const unsigned cols = (unsigned)((p.D + V - 1) / V);
    const uint64_t items = (uint64_t)cols * p.B;
    if (items > (1ull << 31)) return hipErrorInvalidValue;
    const unsigned grid = (unsigned)((items + kConvThreads - 1) / kConvThreads);
    conv_step_kernel<T, W, V><<<grid, kConvThreads, 0, stream>>>(p, cols, (unsigned)items);
    return hipGetLastError();
}

template <typename T, int W, int V>
hipError_t bwd_v(const ConvBwdArgs& q, hipStream_t stream) {
    const ConvArgs& p = q.f;
    const unsigned cblocks = (unsigned)((p.D + 64 * V - 1) / (64 * V));
    const int runs = (p.T + q.run - 1) / q.run;
    if ((uint64_t)cblocks * q.parts > (1ull << 30)) return hipErrorInvalidValue;
    const dim3 grid(cblocks * q.parts);
    if (p.silu) conv_bwd_kernel<T, W, V, true><<<grid, kConvThreads, 0, stream>>>(q, cblocks, runs);
    else conv_bwd_kernel<T, W, V, false><<<grid, kConvThreads, 0, stream>>>(q, cblocks, runs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const size_t total = (size_t)p.D * (W + 1);
    conv_params_kernel<W><<<dim3((unsigned)((total + 15) / 16)), 256, 0, stream>>>(q.part, q.parts, p.D, q.dweight,
                                                                                q.dbias);
    return hipGetLastError();
}

// The gradient of the state when there are no tokens: sT = s0.
template <typename T>
__global__ __launch_bounds__(kConvThreads) void conv_pass_kernel(const T* __restrict__ from, T* to, uint64_t n) {
    const uint64_t id = (uint64_t)blockIdx.x * kConvThreads + threadIdx.x;
    if (id < n) to[id] = from ? from[id] : (T)0;
}

// Channels per thread: the widest piece, up to 16 bytes, that the rows are made of.
template <typename T, int W>
hipError_t fwd_w(const ConvArgs& p, hipStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    return p.D % V == 0         ? fwd_v<T, W, V>(p, stream)
           : p.D % (V / 2) == 0 ? fwd_v<T, W, V / 2>(p, stream)
           : p.D % 2 == 0       ? fwd_v<T, W, 2>(p, stream)
                                : fwd_v<T, W, 1>(p, stream);
}
template <typename T, int W>
hipError_t step_w(const ConvArgs& p, hipStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    return p.D % V == 0         ? step_v<T, W, V>(p, stream)
           : p.D % (V / 2) == 0 ? step_v<T, W, V / 2>(p, stream)
           : p.D % 2 == 0       ? step_v<T, W, 2>(p, stream)
                                : step_v<T, W, 1>(p, stream);
}
template <typename T, int W>
hipError_t bwd_w(const ConvBwdArgs& q, hipStream_t stream) {
    constexpr int V = 4;
    const uint64_t n = (uint64_t)q.f.B * (W - 1) * q.f.D;
    if (q.f.T == 0 && q.ds0 && n > 0) {
        conv_pass_kernel<T><<<dim3((unsigned)((n + kConvThreads - 1) / kConvThreads)), kConvThreads, 0, stream>>>(
            static_cast<const T*>(q.dsT), static_cast<T*>(q.ds0), n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return q.f.D % V == 0 ? bwd_v<T, W, V>(q, stream) : bwd_v<T, W, 1>(q, stream);
}

}  // namespace

#define WKV7_CONV_DISPATCH(fn, p, q)                                                          \
    switch ((p).W) {                                                                          \
        case 2: return (p).bf16 ? fn<bf16_t, 2>(q, stream) : fn<float, 2>(q, stream);         \
        case 3: return (p).bf16 ? fn<bf16_t, 3>(q, stream) : fn<float, 3>(q, stream);         \
        case 4: return (p).bf16 ? fn<bf16_t, 4>(q, stream) : fn<float, 4>(q, stream);         \
        default: return hipErrorInvalidValue;                                                 \
    }

hipError_t launch_conv_forward(const ConvArgs& p, hipStream_t stream) { WKV7_CONV_DISPATCH(fwd_w, p, p) }
hipError_t launch_conv_step(const ConvArgs& p, hipStream_t stream) { WKV7_CONV_DISPATCH(step_w, p, p) }
hipError_t launch_conv_backward(const ConvBwdArgs& q, hipStream_t stream) { WKV7_CONV_DISPATCH(bwd_w, q.f, q) }

}  // namespace wkv7
