// wkv7_ssm.hip -- the selective state-space scan: prompts (forward) and single
// tokens (step).
//
// Per batch row, channel d (N states, its group's B and C) and token t:
//   D_t = softplus(dt_t + dt_bias) (or the sum itself), u_t = D_t x_t
//   h_t[n] = exp(D_t A[n]) h_{t-1}[n] + u_t B_t[n]
//   y_t = (sum_n C_t[n] h_t[n] + dskip x_t) * z_t sigmoid(z_t)
//
// A channel's N states lie over P = N / 4 lanes, four per lane, so a workgroup
// of 256 lanes takes 1024 / N channels of one group and one batch row.  It
// walks the tokens in tiles of 16: every thread loads a piece of one token row
// (x, dt, z) and of B and C, one tile ahead, forms D and u once per token and
// channel and leaves them in LDS as fp32; every lane then steps its four states
// through the tile (exponential as 2^(D A log2 e)); the read-out is summed over
// the channel's lanes by DPP and goes back through LDS to the threads that hold
// the row pieces, which add the skip term, gate and store whole pieces.
// Everything is fp32; only the stored outputs are rounded.
//
// Tokens at or behind a row's length take D = u = 0 and B = C = 0: the state
// passes unchanged (2^0 = 1), whatever the padding holds, and y is stored as 0.
//
// With few channels the sequence also runs in time segments: the recurrence is
// affine with a diagonal transition, so a segment maps its entry state h as
// exp(A sum D) h + e, e its final state from zero.  A first launch finds e and
// sum D of every segment but the last; the second composes its own entry state
// from them and h0 and runs its segment with outputs.

#include "wkv7_ssm_device.h"
#include "wkv7_ssm_internal.h"

namespace wkv7 {

namespace {

constexpr int kTile = kSsmChunk;

template <int N>
struct Shape {
    static constexpr int P = N / kSsmStates;              // lanes per channel
    static constexpr int CH = kSsmThreads / P;            // channels per workgroup
    static constexpr int EPT = CH * kTile / kSsmThreads;  // channels of a thread's row piece
    static constexpr int BC = kTile * N / kSsmThreads > 0 ? kTile * N / kSsmThreads : 1;
    static constexpr int YS = CH + 16;                    // row stride of the read-outs in LDS
};

// A thread's share of one tile as loaded.
template <typename T, int N>
struct Loaded {
    Piece<T, Shape<N>::EPT> x, dt, z;
    Piece<T, Shape<N>::BC> b, c;
};

template <typename T, int N, bool kVec, bool kMap>
__global__ __launch_bounds__(kSsmThreads) void ssm_fwd_kernel(const SsmArgs p, int blocks) {
    using S = Shape<N>;
    constexpr int EPT = S::EPT, BC = S::BC, P = S::P, CH = S::CH;
    __shared__ float2 s_du[2][kTile][CH];
    __shared__ __attribute__((aligned(16))) float s_b[2][kTile][N], s_c[2][kTile][N];
    __shared__ float s_y[2][kTile][S::YS];

    const int tid = threadIdx.x;
    unsigned blk = blockIdx.x;
    const int j = blk % blocks;
    blk /= blocks;
    const int g = blk % p.G;
    blk /= p.G;
    const int b = blk % p.B, seg = blk / p.B;
    const int Dg = p.D / p.G;
    const int c0 = g * Dg + j * CH, cend = (g + 1) * Dg;   // the group's channels end at cend
    const int t_begin = seg * p.seg_len;
    const int t_end = seg == p.nseg - 1 ? p.T : t_begin + p.seg_len;
    const int len = row_length(p.lengths, b, p.T);

    // The row piece this thread stages, and the B, C elements.
    const int pt = tid / 16, pc = c0 + (tid % 16) * EPT;
    const int be = tid * BC, bt = be / N, bn = be % N;
    const bool has_bc = bt < kTile;
    const T* const X = static_cast<const T*>(p.x);
    const T* const DT = static_cast<const T*>(p.dt);
    const T* const Z = static_cast<const T*>(p.z);
    const T* const Bm = static_cast<const T*>(p.Bm);
    const T* const Cm = static_cast<const T*>(p.Cm);
    float bias[EPT], skip[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const int c = pc + i < cend ? pc + i : cend - 1;
        bias[i] = p.dt_bias ? p.dt_bias[c] : 0.f;
        skip[i] = p.dskip ? p.dskip[c] : 0.f;
    }

    // The channel and states this lane steps.
    const int cl = tid / P, n0 = (tid % P) * kSsmStates, ch = c0 + cl;
    const bool live = ch < cend;
    const size_t chn = ((size_t)b * p.D + (live ? ch : cend - 1)) * N + n0;   // into [B][D][N]
    float a2[4], h[4] = {0.f, 0.f, 0.f, 0.f}, dsum = 0.f;
    {
        const float4 a = *reinterpret_cast<const float4*>(p.A + (size_t)(live ? ch : cend - 1) * N + n0);
        a2[0] = a.x * kLog2e; a2[1] = a.y * kLog2e; a2[2] = a.z * kLog2e; a2[3] = a.w * kLog2e;
    }
    if constexpr (!kMap) {
        if (p.h0) load_cols<4>(p.h0 + chn, h);
        const size_t BDN = (size_t)p.B * p.D * N, BD = (size_t)p.B * p.D;
        for (int s = 0; s < seg; ++s) {
            float e[4];
            load_cols<4>(p.seg_h + s * BDN + chn, e);
            const float d = p.seg_d[s * BD + chn / N];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = fmaf(exp2_raw(d * a2[i]), h[i], e[i]);
        }
    }

    auto load = [&](Loaded<T, N>& r, int t0) {
        const int t = t0 + pt < p.T ? t0 + pt : p.T - 1;
        const size_t row = ((size_t)b * p.T + t) * p.D;
        r.x.template load<kVec>(X + row, pc, cend);
        r.dt.template load<kVec>(DT + row, pc, cend);
        if (!kMap && Z) r.z.template load<kVec>(Z + row, pc, cend);
        if (has_bc) {
            const int tb = t0 + bt < p.T ? t0 + bt : p.T - 1;
            const size_t off = (((size_t)b * p.T + tb) * p.G + g) * N;
            r.b.template load<true>(Bm + off, bn, N);
            if (!kMap) r.c.template load<true>(Cm + off, bn, N);
        }
    };
    // The read-outs of the tile at t0 (in s_y[buf]) to y.
    T* const Y = static_cast<T*>(p.y);
    auto write_out = [&](const Piece<T, EPT>& xr, const Piece<T, EPT>& zr, int t0, int buf) {
        const int t = t0 + pt;
        if (t >= t_end) return;
        float out[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            float v = fmaf(skip[i], xr.get(i), s_y[buf][pt][(tid % 16) * EPT + i]);
            if (Z) {
                const float z = zr.get(i);
                v *= z * sigmoid(z);
            }
            out[i] = t < len ? v : 0.f;
        }
        store_piece<kVec>(Y + ((size_t)b * p.T + t) * p.D, pc, cend, out);
    };

    Loaded<T, N> cur;
    Piece<T, EPT> px, pz;   // the previous tile's x and z
    if (t_begin < t_end) load(cur, t_begin);
    const int nck = (p.T + kTile - 1) / kTile;
    int buf = 0;
    for (int t0 = t_begin; t0 < t_end; t0 += kTile, buf ^= 1) {
        {
            const bool in = t0 + pt < len && t0 + pt < t_end;
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const float v = cur.dt.get(i) + bias[i];
                const float d = p.softplus ? softplus(v) : v;
                s_du[buf][pt][(tid % 16) * EPT + i] =
                    in ? make_float2(d, d * cur.x.get(i)) : make_float2(0.f, 0.f);
            }
            if (has_bc) {
                const bool inb = t0 + bt < len && t0 + bt < t_end;
#pragma unroll
                for (int i = 0; i < BC; ++i) {
                    s_b[buf][bt][bn + i] = inb ? cur.b.get(i) : 0.f;
                    if (!kMap) s_c[buf][bt][bn + i] = inb ? cur.c.get(i) : 0.f;
                }
            }
        }
        __syncthreads();
        if constexpr (!kMap) {
            if (t0 > t_begin) write_out(px, pz, t0 - kTile, buf ^ 1);
            px = cur.x;
            pz = cur.z;
            if (p.ckpt_bits && live) {
                const size_t at = (((size_t)b * nck + t0 / kTile) * p.D + ch) * N + n0;
                if (p.ckpt_bits == 32) {
                    store_cols<4>(static_cast<float*>(p.ckpt) + at, h);
                } else {
                    float scale;
                    const uint32_t w = encode8<P>(h, scale);
                    *reinterpret_cast<uint32_t*>(static_cast<char*>(p.ckpt) + at) = w;
                    if (n0 == 0)
                        reinterpret_cast<float*>(static_cast<char*>(p.ckpt) +
                                                 ckpt_scale_offset((size_t)p.B * nck * p.D * N))[at / N] = scale;
                }
            }
        }
        if (t0 + kTile < t_end) load(cur, t0 + kTile);
        float keep = 0.f;
#pragma unroll
        for (int t = 0; t < kTile; ++t) {
            const float2 du = s_du[buf][t][cl];
            const float4 b4 = *reinterpret_cast<const float4*>(&s_b[buf][t][n0]);
            const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = fmaf(exp2_raw(du.x * a2[i]), h[i], du.y * bb[i]);
            if constexpr (kMap) {
                dsum += du.x;
            } else {
                const float4 c4 = *reinterpret_cast<const float4*>(&s_c[buf][t][n0]);
                const float y = group_sum<P>(dot4(make_float4(h[0], h[1], h[2], h[3]), c4));
                keep = t % P == tid % P ? y : keep;
                if (t % P == P - 1) s_y[buf][t - (P - 1) + tid % P][cl] = keep;
            }
        }
    }
    if constexpr (kMap) {
        if (live) {
            store_cols<4>(p.seg_h + (size_t)seg * p.B * p.D * N + chn, h);
            if (n0 == 0) p.seg_d[(size_t)seg * p.B * p.D + chn / N] = dsum;
        }
    } else {
        if (t_begin < t_end) {
            __syncthreads();
            write_out(px, pz, t_begin + (t_end - t_begin - 1) / kTile * kTile, buf ^ 1);
        }
        if (seg == p.nseg - 1 && p.hT && live) store_cols<4>(p.hT + chn, h);
    }
}

// One token on resident states, in place: bound by the states' bytes (read and
// written once, 16 bytes per lane).
template <typename T, int N>
__global__ __launch_bounds__(kSsmThreads) void ssm_step_kernel(const SsmArgs p) {
    constexpr int P = N / kSsmStates, CH = kSsmThreads / P;
    const int64_t ch = (int64_t)blockIdx.x * CH + threadIdx.x / P;   // over B * D
    if (ch >= (int64_t)p.B * p.D) return;
    const int n0 = (threadIdx.x % P) * kSsmStates;
    const int d = (int)(ch % p.D);
    const int64_t b = ch / p.D;
    const size_t bc = ((size_t)b * p.G + d / (p.D / p.G)) * N + n0;
    float a[4], h[4], bb[4], cc[4];
    load_cols<4>(p.A + (size_t)d * N + n0, a);
    load_cols<4>(p.hT + (size_t)ch * N + n0, h);
    load_cols<4>(static_cast<const T*>(p.Bm) + bc, bb);
    load_cols<4>(static_cast<const T*>(p.Cm) + bc, cc);
    const float x = Elem<T>::load1(static_cast<const T*>(p.x) + ch);
    const float v = Elem<T>::load1(static_cast<const T*>(p.dt) + ch) + (p.dt_bias ? p.dt_bias[d] : 0.f);
    const float rate = p.softplus ? softplus(v) : v, u = rate * x;
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = fmaf(exp2_raw(rate * (a[i] * kLog2e)), h[i], u * bb[i]);
        y = fmaf(cc[i], h[i], y);
    }
    store_cols<4>(p.hT + (size_t)ch * N + n0, h);
    y = group_sum<P>(y);
    if (n0 == 0) {
        if (p.dskip) y = fmaf(p.dskip[d], x, y);
        if (p.z) {
            const float z = Elem<T>::load1(static_cast<const T*>(p.z) + ch);
            y *= z * sigmoid(z);
        }
        Elem<T>::store1(static_cast<T*>(p.y) + ch, y);
    }
}

template <typename T, int N>
hipError_t launch_fwd(const SsmArgs& p, hipStream_t stream) {
    using S = Shape<N>;
    const int Dg = p.D / p.G, blocks = (Dg + S::CH - 1) / S::CH;
    const unsigned per = (unsigned)p.B * p.G * blocks;
    const bool vec = Dg % S::EPT == 0;   // every piece whole and aligned
    if (p.nseg > 1) {
        const dim3 grid(per * (p.nseg - 1));
        if (vec) ssm_fwd_kernel<T, N, true, true><<<grid, kSsmThreads, 0, stream>>>(p, blocks);
        else ssm_fwd_kernel<T, N, false, true><<<grid, kSsmThreads, 0, stream>>>(p, blocks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 grid(per * p.nseg);
    if (vec) ssm_fwd_kernel<T, N, true, false><<<grid, kSsmThreads, 0, stream>>>(p, blocks);
    else ssm_fwd_kernel<T, N, false, false><<<grid, kSsmThreads, 0, stream>>>(p, blocks);
    return hipGetLastError();
}

template <typename T, int N>
hipError_t launch_step(const SsmArgs& p, hipStream_t stream) {
    constexpr int CH = kSsmThreads * kSsmStates / N;
    const int64_t n = (int64_t)p.B * p.D;
    ssm_step_kernel<T, N><<<dim3((unsigned)((n + CH - 1) / CH)), kSsmThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_forward(const SsmArgs& p, hipStream_t stream) {
    switch (p.N) {
        case 8: return p.bf16 ? launch_fwd<bf16_t, 8>(p, stream) : launch_fwd<float, 8>(p, stream);
        case 16: return p.bf16 ? launch_fwd<bf16_t, 16>(p, stream) : launch_fwd<float, 16>(p, stream);
        case 32: return p.bf16 ? launch_fwd<bf16_t, 32>(p, stream) : launch_fwd<float, 32>(p, stream);
        case 64: return p.bf16 ? launch_fwd<bf16_t, 64>(p, stream) : launch_fwd<float, 64>(p, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_ssm_step(const SsmArgs& p, hipStream_t stream) {
    switch (p.N) {
        case 8: return p.bf16 ? launch_step<bf16_t, 8>(p, stream) : launch_step<float, 8>(p, stream);
        case 16: return p.bf16 ? launch_step<bf16_t, 16>(p, stream) : launch_step<float, 16>(p, stream);
        case 32: return p.bf16 ? launch_step<bf16_t, 32>(p, stream) : launch_step<float, 32>(p, stream);
        case 64: return p.bf16 ? launch_step<bf16_t, 64>(p, stream) : launch_step<float, 64>(p, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace wkv7
