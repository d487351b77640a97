// wkv7_ssm.hip -- the selective state-space scan: prompts (forward) and single
// tokens (step).
//
// Per batch row, channel d (N states, its group's B and C) and token t:
//   D_t = softplus(dt_t + dt_bias) (or the sum itself), u_t = D_t x_t
//   h_t[n] = exp(D_t A[n]) h_{t-1}[n] + u_t B_t[n]
//   y_t = (sum_n C_t[n] h_t[n] + dskip x_t) * z_t sigmoid(z_t)
//
// The layout over a workgroup is wkv7_ssm_tile.h's.  In interval i the staging
// waves leave D and u of tile i in LDS and finish tile i - 2: they add up the P
// partial read-outs of every token and channel, add the skip term, gate and
// store; they also write the checkpoints (8-bit codes are formed here).  The
// step waves run tile i - 1: per token and state a product for the exponent, a
// 2^x, the two products of the update and one of the read-out.  Everything is
// fp32; only the stored outputs are rounded.
//
// Bound by the vector ALU.  (8, 4096) tokens of 2048 channels, 16 states, bf16,
// with a gate: 259 us, against 105 us for its 0.54 GB at the rate of a large copy
// (5.1 TB/s).  A token of four states per lane takes 20 vector instructions, four
// of them exponentials, and a SIMD 41 ns at any occupancy: 168 us for the whole,
// and the staging waves' softplus and gate take most of the rest.  Measured
// against this split: two states per lane on eight step waves 275 us (the same
// products, twice the partial read-outs); the updates and read-outs as
// v_mfma_f32_4x4x1 (its broadcasts of A fit) 393 us, for these matrix instructions
// do not run beside the vector ALU here; priority for the staging waves 303 us
// where the plain order took 276.
//
// Tokens at or behind a row's length take D = u = 0 and B = C = 0: the state
// passes unchanged (2^0 = 1), whatever the padding holds, and y is stored as 0.
//
// With few channels the sequence also runs in time segments: the recurrence is
// affine with a diagonal transition, so a segment maps its entry state h as
// exp(A sum D) h + e, e its final state from zero.  A first launch finds e and
// sum D of every segment but the last; the second composes its own entry state
// from them and h0 and runs its segment with outputs.  (1, 16384) tokens of 768
// channels: 41 segments, 92 us, 40 of them in the first launch.

#include "wkv7_ssm_tile.h"

namespace wkv7 {

namespace {

// A staging thread's share of one tile as loaded.
template <typename T, int N, bool kVec>
struct Loaded {
    Piece<T, Shape<N, kSsmStates>::EPT, kVec> x, dt, z;
    Piece<T, Shape<N, kSsmStates>::BC, true> b, c;
};

template <typename T, int N, bool kVec, bool kMap, bool kCkpt>
__global__ __launch_bounds__(2 * kStepThreads) void ssm_fwd_kernel(const SsmArgs p, int blocks) {
    using S = Shape<N, kSsmStates>;
    constexpr int EPT = S::EPT, BC = S::BC, P = S::P, CH = S::CH;
    __shared__ __attribute__((aligned(16))) float2 s_du[2][kTile][CH];
    __shared__ __attribute__((aligned(16))) float s_b[2][kTile][N], s_c[2][kMap ? 1 : kTile][N];
    __shared__ __attribute__((aligned(16))) float s_y[2][kMap ? 1 : kTile][kMap ? 1 : P][S::YS];
    __shared__ __attribute__((aligned(16))) float s_h[2][kCkpt ? CH : 1][S::HS];   // states entering a tile

    const Place pos(blocks, p.G, p.B);
    const int g = pos.g, b = pos.b, seg = pos.seg;
    const int Dg = p.D / p.G;
    const int c0 = g * Dg + pos.j * CH, cend = (g + 1) * Dg;   // the group's channels end at cend
    const int t_begin = seg * p.seg_len;
    const int t_end = seg == p.nseg - 1 ? p.T : t_begin + p.seg_len;
    const int tiles = (t_end - t_begin + kTile - 1) / kTile;
    const int intervals = tiles + (kMap ? 0 : 2);

    if (threadIdx.x < kStepThreads) {
        // ---- step waves: tile i - 1 in interval i --------------------------------
        const StepLane<N, kSsmStates> at(threadIdx.x);
        const int ch = c0 + at.cl < cend ? c0 + at.cl : cend - 1;
        const bool live = c0 + at.cl < cend;
        const size_t chn = ((size_t)b * p.D + ch) * N + at.n0;   // into [B][D][N]
        float a2[4], h[4] = {0.f, 0.f, 0.f, 0.f}, dsum = 0.f;
        load_cols<4>(p.A + (size_t)ch * N + at.n0, a2);
#pragma unroll
        for (int i = 0; i < 4; ++i) a2[i] *= kLog2e;
        if constexpr (!kMap) {
            if (p.h0) load_cols<4>(p.h0 + chn, h);
            const size_t BDN = (size_t)p.B * p.D * N, BD = (size_t)p.B * p.D;
            through_segments<4>(h, a2, p.seg_h + chn, (int64_t)BDN, p.seg_d + chn / N, (int64_t)BD, seg);
        }
        // A wave whose channels all lie behind the group only keeps the barriers: what
        // is read of its sums is not stored.
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
        int i = 0;
        if (c0 + wave * 4 / P * 16 >= cend)
            for (; i < intervals; ++i) __syncthreads();
        for (; i < intervals; ++i) {
            __syncthreads();
            if (i >= tiles) continue;
            const int k = i & 1;
            float b4[4], c4[4];
            load_cols<4>(&s_b[k][at.t][at.n0], b4);
            if constexpr (!kMap) {
                load_cols<4>(&s_c[k][at.t][at.n0], c4);
                if constexpr (kCkpt) store_cols<4>(&s_h[k][at.cl][at.n0], h);
            }
            // All of the tile's D and u at once: read per token, each read's
            // latency showed between two tokens.
            float2 d16[kTile];
#pragma unroll
            for (int t = 0; t < kTile; ++t) d16[t] = s_du[k][t][at.cl];
            __builtin_amdgcn_sched_barrier(0);
            each_token([&](auto tok) {
                constexpr int t = decltype(tok)::v;
                const float2 du = d16[t];
                float a[4], x[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    a[n] = exp2_raw(du.x * a2[n]);
                    x[n] = row_bcast<t>(b4[n]) * du.y;
                }
                if constexpr (kMap) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) h[n] = fmaf(a[n], h[n], x[n]);
                    dsum += du.x;
                } else {
                    s_y[k][t][at.part][at.cl] = step_read<t>(h, a, x, c4);
                }
            });
        }
        if (live) {
            if constexpr (kMap) {
                store_cols<4>(p.seg_h + (size_t)seg * p.B * p.D * N + chn, h);
                if (at.n0 == 0) p.seg_d[(size_t)seg * p.B * p.D + chn / N] = dsum;
            } else if (seg == p.nseg - 1 && p.hT) {
                store_cols<4>(p.hT + chn, h);
            }
        }
        return;
    }

    // ---- staging waves: tile i in interval i, the outputs of tile i - 2 -------------
    const int tid = threadIdx.x - kStepThreads;
    const int len = row_length(p.lengths, b, p.T);
    // The thread's row piece: EPT neighbouring channels, or every sixteenth.
    constexpr int ES = kVec ? 1 : kApart;
    const int pt = tid / 16, pl = tid % 16 * (kVec ? EPT : 1);
    const int be = tid * BC, bt = be / N, bn = be % N;              // and its elements of B and C
    float bias[EPT], skip[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const int c = c0 + pl + ES * i < cend ? c0 + pl + ES * i : cend - 1;
        bias[i] = p.dt_bias ? p.dt_bias[c] : 0.f;
        skip[i] = p.dskip ? p.dskip[c] : 0.f;
    }
    const int nck = (p.T + kTile - 1) / kTile;
    const bool gate = p.z != nullptr;
    // The segment's tokens of a tensor as one buffer, from the workgroup's first
    // channel to the end of its group in the last row: one offset per thread moves
    // along all of them, rows behind the segment and pieces behind the group read
    // as 0 and are not written.  So nothing that touches memory in the loop below
    // is conditional, and each wait covers exactly the loads it needs.
    const bool full = kVec || EPT == 1;   // a piece lies inside its group or behind it
    const bool dead = c0 + pl >= cend;
    const int valid = full ? 1 : (cend - c0 - pl + ES - 1) / ES, here = cend - c0 < CH ? cend - c0 : CH;
    const uint32_t row = p.D * (uint32_t)sizeof(T), row_bc = p.G * N * (uint32_t)sizeof(T);
    const int tokens = t_end - t_begin;
    auto rows_of = [&](const void* base, bool on) {
        return buffer_of(static_cast<const char*>(base) + (((int64_t)b * p.T + t_begin) * p.D + c0) * (int)sizeof(T),
                         on && tokens > 0 ? (int)((tokens - 1) * row + (cend - c0) * (uint32_t)sizeof(T)) : 0);
    };
    auto rows_of_bc = [&](const void* base) {
        return buffer_of(static_cast<const char*>(base) + (((int64_t)b * p.T + t_begin) * p.G + g) * N * (int)sizeof(T),
                         tokens > 0 ? (int)((tokens - 1) * row_bc + N * (uint32_t)sizeof(T)) : 0);
    };
    const __amdgpu_buffer_rsrc_t x_rows = rows_of(p.x, true), dt_rows = rows_of(p.dt, true),
                                 z_rows = rows_of(gate ? p.z : p.x, gate), y_rows = rows_of(p.y, !kMap),
                                 b_rows = rows_of_bc(p.Bm), c_rows = rows_of_bc(p.Cm);
    const uint32_t step = dead ? 0 : kTile * row, step_bc = bt < kTile ? kTile * row_bc : 0;
    uint32_t at = dead ? kNowhere : pt * row + pl * (uint32_t)sizeof(T);
    uint32_t at_bc = bt < kTile ? bt * row_bc + bn * (uint32_t)sizeof(T) : kNowhere;
    uint32_t out_at = dead ? kNowhere : at - 2 * step;   // written two tiles later; before that, outside
    auto load = [&](Loaded<T, N, kVec>& r) {
        r.x.load(x_rows, at);
        r.dt.load(dt_rows, at);
        if constexpr (!kMap) r.z.load(z_rows, at);
        r.b.load(b_rows, at_bc);
        if constexpr (!kMap) r.c.load(c_rows, at_bc);
        at += step;
        at_bc += step_bc;
    };
    // The checkpoints of the segment: the thread's four states of channel hc, two
    // tiles behind.
    const int hc = tid / P, hn = (tid % P) * kSsmStates;
    const int blocks_here = (tokens + kTile - 1) / kTile;
    const bool wide = p.ckpt_bits == 32;
    __amdgpu_buffer_rsrc_t h_rows, code_rows, scale_rows;
    uint32_t code_at = 0, scale_at = 0;
    const uint32_t code_step = hc < here ? (uint32_t)p.D * N : 0, scale_step = hc < here && hn == 0 ? 4u * p.D : 0;
    if constexpr (kCkpt) {
        const int64_t crow = ((int64_t)b * nck + t_begin / kTile) * p.D + c0;   // the first tile's first channel
        const int size = blocks_here > 0 ? ((blocks_here - 1) * p.D + here) * N : 0;
        char* const base = static_cast<char*>(p.ckpt);
        h_rows = buffer_of(base + crow * N * 4, wide ? size * 4 : 0);
        code_rows = buffer_of(base + (wide ? 0 : crow * N), wide ? 0 : size);
        scale_rows = buffer_of(base + (wide ? 0 : ckpt_scale_offset((size_t)p.B * nck * p.D * N) + crow * 4),
                               wide || blocks_here == 0 ? 0 : ((blocks_here - 1) * p.D + here) * 4);
        code_at = hc < here ? (uint32_t)(hc * N + hn) - 2 * code_step : kNowhere / 4;
        scale_at = hc < here && hn == 0 ? 4u * hc - 2 * scale_step : kNowhere;
    }
    auto stage = [&](const Loaded<T, N, kVec>& r, int tile) {
        const int t0 = t_begin + tile * kTile, k = tile & 1;
        float d[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) d[i] = r.dt.get(i) + bias[i];
        if (p.softplus) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) d[i] = softplus(d[i]);
        }
        const int end = len < t_end ? len : t_end;
        if (t0 + kTile <= end) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) s_du[k][pt][pl + ES * i] = make_float2(d[i], d[i] * r.x.get(i));
            if (bt < kTile) {
#pragma unroll
                for (int i = 0; i < BC; ++i) {
                    s_b[k][bt][bn + i] = r.b.get(i);
                    if (!kMap) s_c[k][bt][bn + i] = r.c.get(i);
                }
            }
        } else {
            const bool in = t0 + pt < end, inb = t0 + bt < end;
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const float u = d[i] * r.x.get(i);
                s_du[k][pt][pl + ES * i] = make_float2(in ? d[i] : 0.f, in ? u : 0.f);
            }
            if (bt < kTile) {
#pragma unroll
                for (int i = 0; i < BC; ++i) {
                    s_b[k][bt][bn + i] = inb ? r.b.get(i) : 0.f;
                    if (!kMap) s_c[k][bt][bn + i] = inb ? r.c.get(i) : 0.f;
                }
            }
        }
    };
    // The read-outs of a stepped tile, and the checkpoint of the state entering it.
    auto write_out = [&](const Piece<T, EPT, kVec>& xr, const Piece<T, EPT, kVec>& zr, int tile) {
        const int t0 = t_begin + tile * kTile, k = tile & 1;
        float out[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) out[i] = s_y[k][pt][0][pl + ES * i];
#pragma unroll
        for (int q = 1; q < P; ++q)
#pragma unroll
            for (int i = 0; i < EPT; ++i) out[i] += s_y[k][pt][q][pl + ES * i];
#pragma unroll
        for (int i = 0; i < EPT; ++i) out[i] = fmaf(skip[i], xr.get(i), out[i]);
        if (gate) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) out[i] *= zr.get(i) * sigmoid(zr.get(i));
        }
        if (t0 + kTile > len) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) out[i] = t0 + pt < len ? out[i] : 0.f;
        }
        store_piece<T, kVec>(y_rows, out_at, valid, out);
        out_at += step;
        if constexpr (kCkpt) {
            float h[4], scale;
            load_cols<4>(&s_h[k][hc][hn], h);
            const uint32_t w = encode8<P>(h, scale);
            store_piece<float, true>(h_rows, code_at * 4, 1, h);
            __builtin_amdgcn_raw_buffer_store_b32(w, code_rows, code_at, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(scale), scale_rows, scale_at, 0, 0);
            code_at += code_step;
            scale_at += scale_step;
        }
    };

    // Two tiles of loads in flight, and the x and z of the two tiles whose
    // read-outs are still to come: four sets of registers in turn (moving a set
    // that is still being loaded would wait for it).  Behind the last tile and
    // before the first the loads and stores lie outside their buffers, and what is
    // staged is not read.
    Loaded<T, N, kVec> r0, r1, r2, r3;
    load(r0);
    load(r1);
    r2 = r0, r3 = r0;
    auto interval = [&](int i, const Loaded<T, N, kVec>& r, Loaded<T, N, kVec>& old) {
        stage(r, i);
        if constexpr (!kMap) write_out(old.x, old.z, i - 2);
        load(old);
        __syncthreads();
    };
    for (int i = 0; i < intervals; i += 4) {
        interval(i, r0, r2);
        if (i + 1 == intervals) break;
        interval(i + 1, r1, r3);
        if (i + 2 == intervals) break;
        interval(i + 2, r2, r0);
        if (i + 3 == intervals) break;
        interval(i + 3, r3, r1);
    }
}

// One token on resident states, in place: bound by the states' bytes (read and
// written once, 16 bytes per lane).  A lane takes four states of one channel in
// R batch rows, whose loads go out together and share A and the vectors.  256
// rows of 2560 channels, 16 states, bf16: 15.5 us for 90 MB, 5.8 TB/s.
constexpr int kStepRows = 4;

template <typename T, int N, int R>
__global__ __launch_bounds__(kSsmThreads) void ssm_step_kernel(const SsmArgs p) {
    constexpr int P = N / kSsmStates, CH = kSsmThreads / P;
    const unsigned cblocks = (unsigned)((p.D + CH - 1) / CH);
    const int d = (int)(blockIdx.x % cblocks) * CH + threadIdx.x / P;
    const int b0 = (int)(blockIdx.x / cblocks) * R;
    if (d >= p.D) return;
    const int n0 = (threadIdx.x % P) * kSsmStates, g = d / (p.D / p.G);
    float a2[4], h[R][4], bb[R][4], cc[R][4], x[R], v[R], z[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {   // rows behind the last are read as the last, and not written
        const size_t b = b0 + r < p.B ? b0 + r : p.B - 1;
        const size_t bd = b * p.D + d, bc = (b * p.G + g) * N + n0;
        load_cols<4>(p.hT + bd * N + n0, h[r]);
        load_cols<4>(static_cast<const T*>(p.Bm) + bc, bb[r]);
        load_cols<4>(static_cast<const T*>(p.Cm) + bc, cc[r]);
        x[r] = Elem<T>::load1(static_cast<const T*>(p.x) + bd);
        v[r] = Elem<T>::load1(static_cast<const T*>(p.dt) + bd);
        z[r] = p.z ? Elem<T>::load1(static_cast<const T*>(p.z) + bd) : 0.f;
    }
    load_cols<4>(p.A + (size_t)d * N + n0, a2);
#pragma unroll
    for (int i = 0; i < 4; ++i) a2[i] *= kLog2e;
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f, skip = p.dskip ? p.dskip[d] : 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (b0 + r >= p.B) break;
        const size_t bd = (size_t)(b0 + r) * p.D + d;
        const float rate = p.softplus ? softplus(v[r] + bias) : v[r] + bias, u = rate * x[r];
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[r][i] = fmaf(exp2_raw(rate * a2[i]), h[r][i], u * bb[r][i]);
            y = fmaf(cc[r][i], h[r][i], y);
        }
        store_cols<4>(p.hT + bd * N + n0, h[r]);
        y = fmaf(skip, x[r], group_sum<P>(y));
        if (p.z) y *= z[r] * sigmoid(z[r]);
        if (n0 == 0) Elem<T>::store1(static_cast<T*>(p.y) + bd, y);
    }
}

template <typename T, int N, bool kVec>
hipError_t launch_fwd_v(const SsmArgs& p, int blocks, hipStream_t stream) {
    constexpr int threads = 2 * kStepThreads;
    const unsigned per = (unsigned)p.B * p.G * blocks;
    if (p.nseg > 1) {
        ssm_fwd_kernel<T, N, kVec, true, false><<<dim3(per * (p.nseg - 1)), threads, 0, stream>>>(p, blocks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 grid(per * p.nseg);
    if (p.ckpt_bits && p.T > 0) ssm_fwd_kernel<T, N, kVec, false, true><<<grid, threads, 0, stream>>>(p, blocks);
    else ssm_fwd_kernel<T, N, kVec, false, false><<<grid, threads, 0, stream>>>(p, blocks);
    return hipGetLastError();
}

template <typename T, int N>
hipError_t launch_fwd(const SsmArgs& p, hipStream_t stream) {
    using S = Shape<N, kSsmStates>;
    const int Dg = p.D / p.G, blocks = (Dg + S::CH - 1) / S::CH;
    // Whole, aligned pieces where the width of a group holds them.
    return Dg % S::EPT == 0 ? launch_fwd_v<T, N, true>(p, blocks, stream)
                            : launch_fwd_v<T, N, false>(p, blocks, stream);
}

template <typename T, int N>
hipError_t launch_step(const SsmArgs& p, hipStream_t stream) {
    constexpr int CH = kSsmThreads * kSsmStates / N;
    const unsigned cblocks = (unsigned)((p.D + CH - 1) / CH);
    // One row per lane until the device is full: few rows are latency alone.  One and
    // four rows, at 64 workgroups (of one row) 2.2 and 3.3 us, at 2560 5.4 and 5.7, at
    // 4096 7.7 and 7.2, at 10240 16.6 and 15.5.
    if ((int64_t)cblocks * p.B < 4096)
        ssm_step_kernel<T, N, 1><<<dim3(cblocks * p.B), kSsmThreads, 0, stream>>>(p);
    else
        ssm_step_kernel<T, N, kStepRows>
            <<<dim3(cblocks * ((p.B + kStepRows - 1) / kStepRows)), kSsmThreads, 0, stream>>>(p);
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
