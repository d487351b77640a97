// wkv7_ssm_bwd.hip -- gradients of the selective scan (formulas of the forward
// in wkv7_ssm.hip).
//
// With dy_t the gradient of the read-out before the gate, a_t = exp(D_t A) and
// g_t[n] the gradient of h_t[n]:
//   g_t = dy_t C_t + a_{t+1} g_{t+1}          (behind the last token: dhT)
//   dC_t[n] = sum_d dy_t h_t        dB_t[n] = sum_d g_t u_t    (the group's channels)
//   du_t = sum_n g_t B_t            r_t = g_t a_t h_{t-1}
//   dD_t = du_t x_t + sum_n r_t A   dA = sum_{b,t} r_t D_t
//   dx_t = du_t D_t + dy_t dskip    dskip: sum_{b,t} dy_t x_t   dh0 = a_0 g_0
// and the slope of the softplus on dD_t.
//
// The lanes own channels and states as in the forward, walking the 16-token
// tiles last to first.  A tile starts from the checkpoint of the state entering
// it: the lane steps its four states through the tile keeping a_t and h_t in
// registers (no state is read or written per token), then runs the adjoint
// back.  Sums over a channel's states are DPP sums over its P lanes.  Sums over
// channels (dB, dC) fold eight values over the wave's channel lanes at once:
// v_permlane32_swap and v_permlane16_swap halve the values as they add, DPP
// rotations add the rest; the waves meet in LDS, and the channel blocks of a
// group in a second kernel that adds their partial sums in a fixed order (no
// atomics).  dA and the per-channel vectors are summed over tiles in registers,
// over batch rows and segments by the second kernel.
//
// Time segments (few channels): the adjoint is affine too, carry_left =
// exp(A sum D) carry_right + e; a first launch finds e and sum D of every
// segment but the first, the second composes its own entry from dhT.

#include "wkv7_ssm_device.h"
#include "wkv7_ssm_internal.h"

namespace wkv7 {

namespace {

constexpr int kTile = kSsmChunk;
constexpr int kWaves = kSsmThreads / 64;

template <int N>
struct Shape {
    static constexpr int P = N / kSsmStates;              // lanes per channel
    static constexpr int CH = kSsmThreads / P;            // channels per workgroup
    static constexpr int EPT = CH * kTile / kSsmThreads;  // channels of a thread's row piece
    static constexpr int BC = kTile * N / kSsmThreads > 0 ? kTile * N / kSsmThreads : 1;
    static constexpr int YS = CH + 16;                    // row stride of the per-channel sums in LDS
};

template <typename T, int N, bool kVec>
struct Loaded {
    Piece<T, Shape<N>::EPT, kVec> x, dt, z, dy;
    Piece<T, Shape<N>::BC, true> b, c;
};

// Sums v[0..7] over the lanes of a wave that share lane % P: lane l returns in
// q[k] the sum of v[4k + 2 bit4(l) + bit5(l)].
template <int P>
__device__ __forceinline__ void fold8(const float (&v)[8], float (&q)[2]) {
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[2 * i]),
                                                        __float_as_uint(v[2 * i + 1]), false, false);
        w[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(w[2 * k]),
                                                        __float_as_uint(w[2 * k + 1]), false, false);
        float x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
        if (P <= 8) x += __builtin_amdgcn_update_dpp(0.0f, x, 0x128, 0xF, 0xF, false);   // row_ror 8
        if (P <= 4) x += __builtin_amdgcn_update_dpp(0.0f, x, 0x124, 0xF, 0xF, false);   // row_ror 4
        if (P <= 2) x += __builtin_amdgcn_update_dpp(0.0f, x, 0x122, 0xF, 0xF, false);   // row_ror 2
        q[k] = x;
    }
}

template <typename T, int N, bool kVec, bool kMap>
__global__ __launch_bounds__(kSsmThreads, 2) void ssm_bwd_kernel(const SsmBwdArgs q, int blocks) {
    using S = Shape<N>;
    constexpr int EPT = S::EPT, BC = S::BC, P = S::P, CH = S::CH;
    // Per token and channel: D, u, dy; then du, sum r A (and the read-out).
    __shared__ float2 s_du[kTile][CH];
    __shared__ float s_dy[kTile][CH];
    __shared__ __attribute__((aligned(16))) float s_b[kTile][N], s_c[kTile][N];
    __shared__ float s_o[kMap ? 1 : 3][kMap ? 1 : kTile][S::YS];
    __shared__ float s_red[kMap ? 1 : kWaves][kMap ? 1 : kTile][2 * N];

    const SsmArgs& p = q.f;
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    unsigned blk = blockIdx.x;
    const int j = blk % blocks;
    blk /= blocks;
    const int g = blk % p.G;
    blk /= p.G;
    const int b = blk % p.B, seg = (int)(blk / p.B) + (kMap ? 1 : 0);
    const int Dg = p.D / p.G;
    const int c0 = g * Dg + j * CH, cend = (g + 1) * Dg;
    const int t_begin = seg * p.seg_len;
    const int t_end = seg == p.nseg - 1 ? p.T : t_begin + p.seg_len;
    const int len = row_length(p.lengths, b, p.T);

    const int pt = tid / 16, pl = (tid % 16) * EPT, pc = c0 + pl;
    const int be = tid * BC, bt = be / N, bn = be % N;
    const bool has_bc = bt < kTile;
    const T* const X = static_cast<const T*>(p.x);
    const T* const DT = static_cast<const T*>(p.dt);
    const T* const Z = static_cast<const T*>(p.z);
    const T* const DY = static_cast<const T*>(q.dy);
    const T* const Bm = static_cast<const T*>(p.Bm);
    const T* const Cm = static_cast<const T*>(p.Cm);
    float bias[EPT], skip[EPT], sum_skip[EPT], sum_bias[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const int c = pc + i < cend ? pc + i : cend - 1;
        bias[i] = p.dt_bias ? p.dt_bias[c] : 0.f;
        skip[i] = p.dskip ? p.dskip[c] : 0.f;
        sum_skip[i] = sum_bias[i] = 0.f;
    }

    const int cl = tid / P, piece = tid % P, n0 = piece * kSsmStates, ch = c0 + cl;
    const bool live = ch < cend;
    const int chc = live ? ch : cend - 1;
    const size_t chn = ((size_t)b * p.D + chc) * N + n0;
    const size_t BDN = (size_t)p.B * p.D * N, BD = (size_t)p.B * p.D;
    const int nck = (p.T + kTile - 1) / kTile;
    float A[4], a2[4], dA[4] = {0.f, 0.f, 0.f, 0.f}, carry[4] = {0.f, 0.f, 0.f, 0.f}, dsum = 0.f;
    load_cols<4>(p.A + (size_t)chc * N + n0, A);
#pragma unroll
    for (int i = 0; i < 4; ++i) a2[i] = A[i] * kLog2e;
    if constexpr (!kMap) {
        if (q.dhT) load_cols<4>(q.dhT + chn, carry);
        for (int s = p.nseg - 1; s > seg; --s) {
            float e[4];
            load_cols<4>(p.seg_h + (s - 1) * BDN + chn, e);
            const float d = p.seg_d[(s - 1) * BD + chn / N];
#pragma unroll
            for (int i = 0; i < 4; ++i) carry[i] = fmaf(exp2_raw(d * a2[i]), carry[i], e[i]);
        }
    }

    auto load = [&](Loaded<T, N, kVec>& r, int t0) {
        const int t = t0 + pt < p.T ? t0 + pt : p.T - 1;
        const size_t row = ((size_t)b * p.T + t) * p.D;
        if (!kMap) r.x.load(X + row, pc, cend);
        r.dt.load(DT + row, pc, cend);
        r.dy.load(DY + row, pc, cend);
        if (Z) r.z.load(Z + row, pc, cend);
        if (has_bc) {
            const int tb = t0 + bt < p.T ? t0 + bt : p.T - 1;
            const size_t off = (((size_t)b * p.T + tb) * p.G + g) * N;
            if (!kMap) r.b.load(Bm + off, bn, N);
            r.c.load(Cm + off, bn, N);
        }
    };

    // The state entering the tile at t0.
    auto entry = [&](int t0, float (&h)[4]) {
        const size_t at = (((size_t)b * nck + t0 / kTile) * p.D + chc) * N + n0;
        if (p.ckpt_bits == 32) {
            load_cols<4>(static_cast<const float*>(p.ckpt) + at, h);
        } else {
            const char* const base = static_cast<const char*>(p.ckpt);
            decode8(*reinterpret_cast<const uint32_t*>(base + at),
                    reinterpret_cast<const float*>(base + ckpt_scale_offset((size_t)p.B * nck * p.D * N))[at / N], h);
        }
    };

    Loaded<T, N, kVec> cur;
    // The last tile (none when there are no tokens).
    const int t_last = t_begin < t_end ? t_begin + (t_end - t_begin - 1) / kTile * kTile : t_begin - kTile;
    if (t_begin < t_end) load(cur, t_last);
    for (int t0 = t_last; t0 >= t_begin; t0 -= kTile) {
        // ---- stage the tile -------------------------------------------------
        const bool in = t0 + pt < len && t0 + pt < t_end;
        float x[EPT], d[EPT], v[EPT], dy[EPT], dout[EPT], zz[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const bool on = in && pc + i < cend;
            x[i] = on ? cur.x.get(i) : 0.f;
            v[i] = cur.dt.get(i) + bias[i];
            d[i] = on ? (p.softplus ? softplus(v[i]) : v[i]) : 0.f;
            dout[i] = on ? cur.dy.get(i) : 0.f;
            zz[i] = Z && on ? cur.z.get(i) : 0.f;
            dy[i] = Z ? dout[i] * zz[i] * sigmoid(zz[i]) : dout[i];
            s_du[pt][pl + i] = make_float2(d[i], kMap ? 0.f : d[i] * x[i]);
            s_dy[pt][pl + i] = dy[i];
        }
        if (has_bc) {
            const bool inb = t0 + bt < len && t0 + bt < t_end;
#pragma unroll
            for (int i = 0; i < BC; ++i) {
                if (!kMap) s_b[bt][bn + i] = inb ? cur.b.get(i) : 0.f;
                s_c[bt][bn + i] = inb ? cur.c.get(i) : 0.f;
            }
        }
        __syncthreads();
        if (t0 > t_begin) load(cur, t0 - kTile);
        if constexpr (kMap) {
#pragma unroll
            for (int t = kTile - 1; t >= 0; --t) {
                const float dt = s_du[t][cl].x, dyt = s_dy[t][cl];
                const float4 c4 = *reinterpret_cast<const float4*>(&s_c[t][n0]);
                const float cc[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) carry[i] = exp2_raw(dt * a2[i]) * fmaf(dyt, cc[i], carry[i]);
                dsum += dt;
            }
        } else {
            // ---- the states of the tile again -------------------------------
            float h0[4], a[kTile][4], h[kTile][4];
            entry(t0, h0);
            float keep = 0.f;
#pragma unroll
            for (int t = 0; t < kTile; ++t) {
                const float2 du = s_du[t][cl];
                const float4 b4 = *reinterpret_cast<const float4*>(&s_b[t][n0]);
                const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[t][i] = exp2_raw(du.x * a2[i]);
                    h[t][i] = fmaf(a[t][i], t == 0 ? h0[i] : h[t - 1][i], du.y * bb[i]);
                }
                if (Z) {
                    const float4 c4 = *reinterpret_cast<const float4*>(&s_c[t][n0]);
                    const float y = group_sum<P>(dot4(make_float4(h[t][0], h[t][1], h[t][2], h[t][3]), c4));
                    keep = t % P == piece ? y : keep;
                    if (t % P == P - 1) s_o[2][t - (P - 1) + piece][cl] = keep;
                }
            }
            // ---- the adjoint, last token first ------------------------------
            float tA[4] = {0.f, 0.f, 0.f, 0.f}, keep0 = 0.f, keep1 = 0.f;
#pragma unroll
            for (int t = kTile - 1; t >= 0; --t) {
                const float2 du = s_du[t][cl];
                const float dyt = s_dy[t][cl];
                const float4 b4 = *reinterpret_cast<const float4*>(&s_b[t][n0]);
                const float4 c4 = *reinterpret_cast<const float4*>(&s_c[t][n0]);
                const float bb[4] = {b4.x, b4.y, b4.z, b4.w}, cc[4] = {c4.x, c4.y, c4.z, c4.w};
                float bc[8], sb = 0.f, sr = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float gr = fmaf(dyt, cc[i], carry[i]);
                    bc[i] = gr * du.y;
                    bc[4 + i] = dyt * h[t][i];
                    sb = fmaf(gr, bb[i], sb);
                    carry[i] = a[t][i] * gr;
                    const float r = carry[i] * (t == 0 ? h0[i] : h[t - 1][i]);
                    sr = fmaf(r, A[i], sr);
                    tA[i] = fmaf(r, du.x, tA[i]);
                }
                sb = group_sum<P>(sb);
                sr = group_sum<P>(sr);
                keep0 = t % P == piece ? sb : keep0;
                keep1 = t % P == piece ? sr : keep1;
                if (t % P == 0) {
                    s_o[0][t + piece][cl] = keep0;
                    s_o[1][t + piece][cl] = keep1;
                }
                float f[2];
                fold8<P>(bc, f);
                // Lanes whose low channel bits are 0 hold the sums of their states.
                if ((lane & 15) / P == 0) {
                    const int n = n0 + 2 * ((lane >> 4) & 1) + (lane >> 5);
                    s_red[wave][t][n] = f[0];
                    s_red[wave][t][N + n] = f[1];
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) dA[i] += tA[i];
        }
        __syncthreads();
        if constexpr (!kMap) {
            // ---- dB, dC of the tile -----------------------------------------
            for (int e = tid; e < kTile * 2 * N; e += kSsmThreads) {
                const int t = e / (2 * N), n = e % (2 * N);
                if (t0 + t < t_end) {
                    float s = 0.f;
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) s += s_red[w][t][n];
                    const size_t row = ((size_t)b * p.T + t0 + t) * p.G + g;
                    if (q.part_bc) {
                        q.part_bc[((size_t)j * p.B * p.T * p.G + row) * (2 * N) + n] = s;
                    } else if (n < N) {
                        Elem<T>::store1(static_cast<T*>(q.dBm) + row * N + n, s);
                    } else {
                        Elem<T>::store1(static_cast<T*>(q.dCm) + row * N + n - N, s);
                    }
                }
            }
            // ---- per token and channel --------------------------------------
            if (t0 + pt < t_end) {
                float dx[EPT], ddt[EPT], dz[EPT];
#pragma unroll
                for (int i = 0; i < EPT; ++i) {
                    const float du = s_o[0][pt][pl + i], sr = s_o[1][pt][pl + i];
                    dx[i] = fmaf(du, d[i], dy[i] * skip[i]);
                    const float dd = fmaf(du, x[i], sr);
                    ddt[i] = in ? (p.softplus ? dd * sigmoid(v[i]) : dd) : 0.f;
                    if (Z) {
                        const float y = fmaf(skip[i], x[i], s_o[2][pt][pl + i]), s = sigmoid(zz[i]);
                        dz[i] = dout[i] * y * (s * fmaf(zz[i], 1.f - s, 1.f));
                    }
                    sum_skip[i] = fmaf(dy[i], x[i], sum_skip[i]);
                    sum_bias[i] += ddt[i];
                }
                const size_t row = ((size_t)b * p.T + t0 + pt) * p.D;
                store_piece<kVec>(static_cast<T*>(q.dx) + row, pc, cend, dx);
                store_piece<kVec>(static_cast<T*>(q.ddt) + row, pc, cend, ddt);
                if (Z) store_piece<kVec>(static_cast<T*>(q.dz) + row, pc, cend, dz);
            }
        }
    }
    if constexpr (kMap) {
        if (live) {
            store_cols<4>(p.seg_h + (seg - 1) * BDN + chn, carry);
            if (n0 == 0) p.seg_d[(seg - 1) * BD + chn / N] = dsum;
        }
    } else {
        if (live) {
            store_cols<4>(q.part_a + (((size_t)seg * p.B + b) * p.D + ch) * N + n0, dA);
            if (seg == 0 && q.dh0) store_cols<4>(q.dh0 + chn, carry);
        }
        // The per-channel vectors: the sixteen threads of a row piece's channels
        // hold every sixteenth token each.
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            s_o[0][pt][pl + i] = sum_skip[i];
            s_o[1][pt][pl + i] = sum_bias[i];
        }
        __syncthreads();
        for (int c = tid; c < CH; c += kSsmThreads) {
            if (c0 + c < cend) {
                float s0 = 0.f, s1 = 0.f;
                for (int t = 0; t < kTile; ++t) {
                    s0 += s_o[0][t][c];
                    s1 += s_o[1][t][c];
                }
                *reinterpret_cast<float2*>(q.part_v + (((size_t)seg * p.B + b) * p.D + c0 + c) * 2) =
                    make_float2(s0, s1);
            }
        }
    }
}

// dB and dC: the sum of `blocks` partials per element, in order.  Four elements
// per thread (N is a multiple of 8).
template <typename T>
__global__ __launch_bounds__(256) void ssm_bc_kernel(const float* __restrict__ part, int blocks,
                                                     size_t rows, int N, T* dB, T* dC) {
    const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4, total = rows * 2 * N;
    if (at >= total) return;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < blocks; ++k) {
        float v[4];
        load_cols<4>(part + k * total + at, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += v[i];
    }
    const size_t row = at / (2 * N), n = at % (2 * N);
    Elem<T>::store4(n < (size_t)N ? dB + row * N + n : dC + row * N + n - N, make_float4(s[0], s[1], s[2], s[3]));
}

// dA, ddskip and ddt_bias: the sum over `parts` batch rows and segments.
// Element e of D N + 2 D: dA, then the two vectors interleaved.
__global__ __launch_bounds__(256) void ssm_params_kernel(const float* __restrict__ part_a,
                                                         const float* __restrict__ part_v, int parts, int D,
                                                         int N, float* dA, float* ddskip, float* ddt_bias) {
    const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x, DN = (size_t)D * N;
    if (e < DN) {
        float s = 0.f;
        for (int k = 0; k < parts; ++k) s += part_a[k * DN + e];
        dA[e] = s;
    } else if (e < DN + 2 * (size_t)D) {
        const size_t i = e - DN;
        float* const out = i % 2 == 0 ? ddskip : ddt_bias;
        if (!out) return;
        float s = 0.f;
        for (int k = 0; k < parts; ++k) s += part_v[k * 2 * (size_t)D + i];
        out[i / 2] = s;
    }
}

template <typename T, int N>
hipError_t launch_bwd(const SsmBwdArgs& q, hipStream_t stream) {
    using S = Shape<N>;
    const SsmArgs& p = q.f;
    const int Dg = p.D / p.G, blocks = (Dg + S::CH - 1) / S::CH;
    const unsigned per = (unsigned)p.B * p.G * blocks;
    const bool vec = Dg % S::EPT == 0;
    hipError_t e;
    if (p.nseg > 1 && per > 0) {
        const dim3 grid(per * (p.nseg - 1));
        if (vec) ssm_bwd_kernel<T, N, true, true><<<grid, kSsmThreads, 0, stream>>>(q, blocks);
        else ssm_bwd_kernel<T, N, false, true><<<grid, kSsmThreads, 0, stream>>>(q, blocks);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (per > 0) {
        const dim3 grid(per * p.nseg);
        if (vec) ssm_bwd_kernel<T, N, true, false><<<grid, kSsmThreads, 0, stream>>>(q, blocks);
        else ssm_bwd_kernel<T, N, false, false><<<grid, kSsmThreads, 0, stream>>>(q, blocks);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const size_t rows = (size_t)p.B * p.T * p.G;
    if (q.part_bc && rows > 0) {
        const size_t n = (rows * 2 * N / 4 + 255) / 256;
        ssm_bc_kernel<T><<<dim3((unsigned)n), 256, 0, stream>>>(q.part_bc, blocks, rows, N,
                                                                static_cast<T*>(q.dBm), static_cast<T*>(q.dCm));
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const size_t n = ((size_t)p.D * (N + 2) + 255) / 256;
    ssm_params_kernel<<<dim3((unsigned)n), 256, 0, stream>>>(q.part_a, q.part_v, p.B * p.nseg, p.D, N, q.dA,
                                                             q.ddskip, q.ddt_bias);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_backward(const SsmBwdArgs& q, hipStream_t stream) {
    const bool bf16 = q.f.bf16;
    switch (q.f.N) {
        case 8: return bf16 ? launch_bwd<bf16_t, 8>(q, stream) : launch_bwd<float, 8>(q, stream);
        case 16: return bf16 ? launch_bwd<bf16_t, 16>(q, stream) : launch_bwd<float, 16>(q, stream);
        case 32: return bf16 ? launch_bwd<bf16_t, 32>(q, stream) : launch_bwd<float, 32>(q, stream);
        case 64: return bf16 ? launch_bwd<bf16_t, 64>(q, stream) : launch_bwd<float, 64>(q, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace wkv7
