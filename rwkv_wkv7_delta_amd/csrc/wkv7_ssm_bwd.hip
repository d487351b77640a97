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
// The layout over a workgroup is wkv7_ssm_tile.h's, the tiles taken last to
// first.  A tile starts from the checkpoint of the state entering it (decoded by
// the staging waves): a step lane steps its states through the tile keeping a_t
// and h_t in registers (no state is read or written per token), then runs the
// adjoint back.  Sums over channels (dB, dC) fold a lane's values over the
// sixteen channels of its row by DPP, halving the values as they add; sums over
// states fold over the wave's rows by lane swaps; the rest meets in LDS, and the
// channel blocks of a group in a second kernel that adds their partial sums in a
// fixed order (no atomics).  dA and the per-channel vectors are summed over
// tiles in registers, over batch rows and segments by the second kernel.
//
// Bound by the vector ALU and the one step wave per SIMD that feeds it.  (4, 4096)
// tokens of 2048 channels, 16 states, bf16, gate, 8-bit checkpoints: 470 us and 24
// for the sums of the partial dB and dC (134 MB), against 92 us for the tensors' bytes
// (144 with those sums') and 163 us for the formulas' products alone, one lane per state.  A
// step wave takes 630 vector instructions per tile (two states and sixteen tokens
// per lane: 128 of them folds over channels, 48 swaps and adds over states), a
// staging wave 140: 370 us for both at their rates; the vector ALU is busy for 79 % of
// the time.  At 32 and 64 states a workgroup holds 16 channels, and the partial sums
// (537 MB and 1.07 GB at the same shape) outgrow the tensors: 820 + 130 and 1610 + 235
// us.  At 8 it holds 64, 128 workgroups for 256 compute units: 483 + 7 us.  Measured against
// this split: one state per lane on eight step waves 543 us where this took 521;
// the sums over states on v_mfma_f32_16x16x4 974 us; states and adjoint on four
// waves each, the states handed over in LDS and the exponentials taken twice, 540
// where this took 505.
//
// Time segments (few channels): the adjoint is affine too, carry_left =
// exp(A sum D) carry_right + e; a first launch finds e and sum D of every
// segment but the first, the second composes its own entry from dhT.

#include "wkv7_ssm_tile.h"

namespace wkv7 {

namespace {

// States per lane: two, so that the 2 x 16 states and transitions of a tile stay
// in registers beside everything else and a workgroup takes few enough channels
// to spread over the device; four at N = 64, whose channels would not fit a
// workgroup's sixteen rows otherwise.
template <int N>
constexpr int kStates = N == 64 ? 4 : 2;

template <typename T, int N, bool kVec>
struct Loaded {
    static constexpr int S = kStates<N>;
    Piece<T, Shape<N, S>::EPT, kVec> x, dt, z, dy;
    Piece<T, Shape<N, S>::BC, true> b, c;
    Piece<float, S, true> h;       // entry states: fp32,
    uint32_t codes, scale;         // or codes and their scale
};

// What a staging thread keeps of a tile until its gradients come back.
template <int EPT>
struct Kept {
    float x[EPT], d[EPT], slope[EPT], dy[EPT], w[EPT];   // w: dz per read-out
};

// Two folds of four values each over the sixteen lanes of every row: a step adds
// a lane's partner (row_ror:8, row_half_mirror, quad_perm) and, while there are
// several values, keeps one by a bit of the lane, which the bank masks of the DPP
// writes select.  Lane l returns the sum of value 2 bit2(l) + bit3(l) of each.
// Two folds at once, so that each fills the two instructions that must lie
// between writing a register and reading it through DPP in the other.
__device__ __forceinline__ void fold_row(const float (&v)[4], const float (&w)[4], float& y, float& z) {
    float x0, x1, u0, u1;
    asm("s_nop 1\n\t"
        "v_add_f32_dpp %0, %7, %7 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %1, %9, %9 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %2, %11, %11 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %3, %13, %13 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %0, %6, %6 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %1, %8, %8 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %2, %10, %10 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %3, %12, %12 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %4, %0, %0 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %5, %2, %2 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %4, %1, %1 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
        "v_add_f32_dpp %5, %3, %3 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
        "s_nop 0\n\t"
        "v_add_f32_dpp %4, %4, %4 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %5, %5, %5 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 0\n\t"
        "v_add_f32_dpp %4, %4, %4 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %5, %5, %5 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf"
        : "=&v"(x0), "=&v"(x1), "=&v"(u0), "=&v"(u1), "=&v"(y), "=&v"(z)
        : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(w[0]), "v"(w[1]), "v"(w[2]), "v"(w[3]));
}

// h = a g + x for two states, and the sum of (c broadcast from lane t of the row) h.
// As in the forward's step_read: the s_nop for a, which an exponential may just have
// written, the two updates in front of the products that read c through DPP.  The
// sums go into lane swaps (fold_rows): settled() first.
template <int t>
__device__ __forceinline__ float state_step(float& h0, float& h1, float g0, float g1, float a0, float a1, float x0,
                                            float x1, float c0, float c1) {
    float y;
    asm("s_nop 0\n\t"
        "v_fma_f32 %0, %5, %3, %7\n\t"
        "v_fma_f32 %1, %6, %4, %8\n\t"
        "v_mul_f32_dpp %2, %9, %0 row_newbcast:%11 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %2, %10, %1 row_newbcast:%11 row_mask:0xf bank_mask:0xf"
        : "=&v"(h0), "=&v"(h1), "=&v"(y)
        : "v"(g0), "v"(g1), "v"(a0), "v"(a1), "v"(x0), "v"(x1), "v"(c0), "v"(c1), "n"(t));
    return y;
}

// A swap may not read what one of the two instructions before it wrote; the compiler
// keeps that distance for its own instructions, not for state_step's sums.  Of each
// pair that is swapped the later one counts: the other was written a token earlier.
__device__ __forceinline__ void settled(float& y1, float& y3) { asm("s_nop 1" : "+v"(y1), "+v"(y3)); }

// One step of the adjoint for two states: g <- g + c dy (c broadcast from lane t of
// the row), v = (g u, dy h), the sum of (b broadcast) g, and g <- a g.  The two
// products in front keep the DPP operands c two instructions from whatever wrote
// them.  The sum meets a lane swap only together with the sum of r A, whose three
// products follow this.
template <int t>
__device__ __forceinline__ float adjoint_step(float& g0, float& g1, float (&v)[4], float c0, float c1, float b0,
                                              float b1, float dy, float u, float h0, float h1, float a0, float a1) {
    float sb;
    asm("v_mul_f32 %4, %11, %13\n\t"
        "v_mul_f32 %5, %11, %14\n\t"
        "v_fmac_f32_dpp %0, %7, %11 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %8, %11 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32 %2, %0, %12\n\t"
        "v_mul_f32_dpp %6, %9, %0 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32 %3, %1, %12\n\t"
        "v_mul_f32 %0, %15, %0\n\t"
        "v_fmac_f32_dpp %6, %10, %1 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
        "v_mul_f32 %1, %16, %1"
        : "+&v"(g0), "+&v"(g1), "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(sb)
        : "v"(c0), "v"(c1), "v"(b0), "v"(b1), "v"(dy), "v"(u), "v"(h0), "v"(h1), "v"(a0), "v"(a1), "n"(t));
    return sb;
}

// Sums of four values over the wave's four rows: row r returns the sum of value
// 0, 2, 1, 3 for r = 0, 1, 2, 3.
__device__ __forceinline__ float fold_rows(float v0, float v1, float v2, float v3) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v0), __float_as_uint(v1), false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v2), __float_as_uint(v3), false, false);
    const float p = __uint_as_float(a[0]) + __uint_as_float(a[1]), q = __uint_as_float(b[0]) + __uint_as_float(b[1]);
    const auto c = __builtin_amdgcn_permlane16_swap(__float_as_uint(p), __float_as_uint(q), false, false);
    return __uint_as_float(c[0]) + __uint_as_float(c[1]);
}

// A row of 64 sums, turned by 16 per token: neighbouring tokens' rows then lie on
// different banks.
__device__ __forceinline__ int turned(int t, int col) { return (col + 16 * t) & 63; }

// kDense: registers for two workgroups per compute unit (LDS holds two at N = 16
// and 32).  That fills each one's waits, but ties the schedule: with more than
// one workgroup per unit, (4, 1024) tokens of 768 channels, forward and
// backward, take 104 us with it and 112 without; one workgroup per unit, (4, 4096)
// of 2048 channels, 568 with it and 497 without (491 now).
template <typename T, int N, bool kVec, bool kMap, bool kGate, bool kDense>
__global__ __launch_bounds__(2 * kStepThreads, (kDense ? 4 : 2)) void ssm_bwd_kernel(const SsmBwdArgs q, int blocks) {
    constexpr int S = kStates<N>;
    using Sh = Shape<N, S>;
    constexpr int EPT = Sh::EPT, BC = Sh::BC, P = Sh::P, CH = Sh::CH, HS = Sh::HS;
    constexpr int PW = P / 4;                  // waves that share a channel
    constexpr int CG = CH / 16;                // groups of 16 channels
    constexpr int OS = 64;                     // row stride of the sums over states
    // A tile's inputs and its read-outs are live through four intervals (staged;
    // its states; its adjoint; its gradients), the rest through two.
    __shared__ __attribute__((aligned(16))) float2 s_du[4][kTile][CH];
    __shared__ __attribute__((aligned(16))) float s_dy[4][kTile][CH];
    __shared__ __attribute__((aligned(16))) float s_b[4][kMap ? 1 : kTile][N], s_c[4][kTile][N];
    __shared__ __attribute__((aligned(16))) float s_h[2][kMap ? 1 : CH][HS];
    // Per token: the read-out, the sums over a wave's states of du and of r A; and
    // the sums over 16 channels of dB and dC.
    __shared__ __attribute__((aligned(16))) float s_y[kGate && !kMap ? 4 : 1][kMap ? 1 : kTile][OS];
    __shared__ __attribute__((aligned(16))) float s_o[2][kMap ? 1 : 2][kMap ? 1 : kTile][OS];
    __shared__ __attribute__((aligned(16))) float s_red[2][kMap ? 1 : CG][kMap ? 1 : kTile][2 * N];

    const SsmArgs& p = q.f;
    const Place pos(blocks, p.G, p.B);
    const int g = pos.g, b = pos.b, j = pos.j, seg = pos.seg + (kMap ? 1 : 0);
    const int Dg = p.D / p.G;
    const int c0 = g * Dg + j * CH, cend = (g + 1) * Dg;
    const int t_begin = seg * p.seg_len;
    const int t_end = seg == p.nseg - 1 ? p.T : t_begin + p.seg_len;
    const int tiles = (t_end - t_begin + kTile - 1) / kTile;
    const int intervals = tiles + (kMap ? 0 : 3);
    const size_t BDN = (size_t)p.B * p.D * N, BD = (size_t)p.B * p.D;

    if (threadIdx.x < kStepThreads) {
        // ---- step waves, tiles counted from the end: in interval i + 1 the states of
        // ---- tile i and, interleaved with them, the adjoint of tile i - 1 ----------------
        const StepLane<N, S> at(threadIdx.x);
        const int wave = threadIdx.x / 64, l = threadIdx.x % 16, row = threadIdx.x / 16 % 4;
        const bool live = c0 + at.cl < cend;
        const int ch = live ? c0 + at.cl : cend - 1;
        const size_t chn = ((size_t)b * p.D + ch) * N + at.n0;
        float A[S], a2[S], dA[S], carry[S], dsum = 0.f;
        load_cols<S>(p.A + (size_t)ch * N + at.n0, A);
#pragma unroll
        for (int n = 0; n < S; ++n) {
            a2[n] = A[n] * kLog2e;
            dA[n] = carry[n] = 0.f;
        }
        if constexpr (!kMap) {
            if (q.dhT) load_cols<S>(q.dhT + chn, carry);
            // segments nseg - 1 down to seg + 1, kept at one less
            through_segments<S>(carry, a2, p.seg_h + (p.nseg - 2) * (int64_t)BDN + chn, -(int64_t)BDN,
                                p.seg_d + (p.nseg - 2) * (int64_t)BD + chn / N, -(int64_t)BD, p.nseg - 1 - seg);
            // A lane behind the group read its last channel's; it adds to the row's dB and dC,
            // and with D = u = dy = 0 from the staging waves every term of it is 0.
#pragma unroll
            for (int n = 0; n < S; ++n) carry[n] = live ? carry[n] : 0.f;
        }
        // Where the lane leaves its folded sums: row r of the wave holds value 0,
        // 2, 1, 3 of a fold over the rows; a lane of a row the state and dB or dC
        // (the values are (g u, dy h) of two states) that fold_row names.
        const int col = wave * 16 + l;
        const int second = row >> 1, later = row & 1;   // of (sb, sr), (t, t - 1)
        const int n_red = at.n0 + (l >> 3) + (l >> 2 & 1) * N;
        if constexpr (kMap) {
            for (int i = 0; i < intervals; ++i) {
                __syncthreads();
                if (i >= tiles) continue;
                const int k = i & 3;
                float c4[S];
                load_cols<S>(&s_c[k][at.t][at.n0], c4);
                each_token_back([&](auto tok) {
                    constexpr int t = decltype(tok)::v;
                    const float d = s_du[k][t][at.cl].x, dyt = s_dy[k][t][at.cl];
#pragma unroll
                    for (int n = 0; n < S; ++n)
                        carry[n] = exp2_raw(d * a2[n]) * (carry[n] + row_bcast<t>(c4[n]) * dyt);
                    dsum += d;
                });
            }
        } else {
            // A tile's transitions and states, from the state entering it.
            struct Tile {
                float a[kTile][S], h[kTile][S], h0[S], b[S], c[S];
            };
            float y4[4], v1[4], tA[S], sb1, sr1;
            auto begin = [&](Tile& w, int i) {
                load_cols<S>(&s_b[i & 3][at.t][at.n0], w.b);
                load_cols<S>(&s_c[i & 3][at.t][at.n0], w.c);
                load_cols<S>(&s_h[i & 1][at.cl][at.n0], w.h0);
            };
            auto states = [&](auto tok, Tile& w, int i) {
                constexpr int t = decltype(tok)::v;
                const float2 du = s_du[i & 3][t][at.cl];
                float y = 0.f, x[S];
                const float(&before)[S] = t == 0 ? w.h0 : w.h[t > 0 ? t - 1 : 0];
#pragma unroll
                for (int n = 0; n < S; ++n) {
                    w.a[t][n] = exp2_raw(du.x * a2[n]);
                    x[n] = row_bcast<t>(w.b[n]) * du.y;
                }
#pragma unroll
                for (int n = 0; n < S; n += 2) {
                    if constexpr (kGate) {
                        const float q = state_step<t>(w.h[t][n], w.h[t][n + 1], before[n], before[n + 1], w.a[t][n],
                                                      w.a[t][n + 1], x[n], x[n + 1], w.c[n], w.c[n + 1]);
                        y = n == 0 ? q : y + q;
                    } else {
                        w.h[t][n] = fmaf(w.a[t][n], before[n], x[n]);
                        w.h[t][n + 1] = fmaf(w.a[t][n + 1], before[n + 1], x[n + 1]);
                    }
                }
                if constexpr (kGate) {
                    y4[t % 4] = y;
                    // rows 0, 1, 2, 3 hold tokens t - 3, t - 1, t - 2, t
                    if constexpr (t % 4 == 3) {
                        settled(y4[1], y4[3]);
                        const int tok = t - 3 + 2 * later + second;
                        s_y[i & 3][tok][turned(tok, col)] = fold_rows(y4[0], y4[1], y4[2], y4[3]);
                    }
                }
            };
            auto adjoint = [&](auto tok, const Tile& w, int i) {
                constexpr int t = decltype(tok)::v;
                const int k = i & 1;
                const float2 du = s_du[i & 3][t][at.cl];
                const float dyt = s_dy[i & 3][t][at.cl];
                float v[S / 2][4], sb = 0.f, sr = 0.f;
#pragma unroll
                for (int n = 0; n < S; n += 2) {
                    const float s = adjoint_step<t>(carry[n], carry[n + 1], v[n / 2], w.c[n], w.c[n + 1], w.b[n], w.b[n + 1],
                                                    dyt, du.y, w.h[t][n], w.h[t][n + 1], w.a[t][n], w.a[t][n + 1]);
                    sb = n == 0 ? s : sb + s;
                }
#pragma unroll
                for (int n = 0; n < S; ++n) {
                    const float r = carry[n] * (t == 0 ? w.h0[n] : w.h[t > 0 ? t - 1 : 0][n]);
                    sr = n == 0 ? r * A[n] : fmaf(r, A[n], sr);
                    tA[n] = t == kTile - 1 ? r * du.x : fmaf(r, du.x, tA[n]);
                }
                float f0, f1;
                if constexpr (S == 4) {
                    fold_row(v[0], v[1], f0, f1);
                    s_red[k][at.cl / 16][t][n_red] = f0;
                    s_red[k][at.cl / 16][t][n_red + 2] = f1;
                }
                if constexpr (t % 2 == 1) {
                    sb1 = sb;
                    sr1 = sr;
#pragma unroll
                    for (int n = 0; n < 4; ++n) v1[n] = v[0][n];
                } else {   // value 0: (sb, t + 1), 1: (sr, t + 1), 2: (sb, t), 3: (sr, t)
                    s_o[k][second][t + 1 - later][turned(t + 1 - later, col)] = fold_rows(sb1, sr1, sb, sr);
                    if constexpr (S == 2) {
                        fold_row(v1, v[0], f0, f1);
                        s_red[k][at.cl / 16][t + 1][n_red] = f0;
                        s_red[k][at.cl / 16][t][n_red] = f1;
                    }
                }
            };
            // Two chains that do not depend on each other, a token of each in turn
            // (one wave to a SIMD beside a staging wave leaves a single chain's
            // latencies bare); as many states die on one side as are born on the
            // other.  The states behind the last tile are formed and not used.
            auto both = [&](const Tile& w, Tile& next, int i) {
                begin(next, i);
                each_token([&](auto tok) {
                    constexpr int t = decltype(tok)::v;
                    states(tok, next, i);
                    adjoint(Tok<kTile - 1 - t>(), w, i - 1);
                });
#pragma unroll
                for (int n = 0; n < S; ++n) dA[n] += tA[n];
            };
            Tile w0, w1;
            __syncthreads();
            begin(w0, 0);
            each_token([&](auto tok) { states(tok, w0, 0); });
            int i = 1;
            while (i <= tiles) {
                __syncthreads();
                both(w0, w1, i++);
                if (i > tiles) break;
                __syncthreads();
                both(w1, w0, i++);
            }
            for (; i < intervals; ++i) __syncthreads();
        }
        if (live) {
            if constexpr (kMap) {
                store_cols<S>(p.seg_h + (seg - 1) * BDN + chn, carry);
                if (at.n0 == 0) p.seg_d[(seg - 1) * BD + chn / N] = dsum;
            } else {
                store_cols<S>(q.part_a + (((size_t)seg * p.B + b) * p.D + ch) * N + at.n0, dA);
                if (seg == 0 && q.dh0) store_cols<S>(q.dh0 + chn, carry);
            }
        }
        if constexpr (!kMap) __syncthreads();
        return;
    }

    // ---- staging waves: the i-th tile from the end in interval i, the gradients of
    // ---- the (i - 3)-th ---------------------------------------------------------------
    const int tid = threadIdx.x - kStepThreads;
    const int len = row_length(p.lengths, b, p.T);
    constexpr int ES = kVec ? 1 : kApart;
    const int pt = tid / 16, pl = tid % 16 * (kVec ? EPT : 1);
    const int be = tid * BC, bt = be / N, bn = be % N;
    const int hc = tid * S / N, hn = tid * S % N;     // the thread's entry states
    float bias[EPT], skip[EPT], sum_skip[EPT], sum_bias[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const int c = c0 + pl + ES * i < cend ? c0 + pl + ES * i : cend - 1;
        bias[i] = p.dt_bias ? p.dt_bias[c] : 0.f;
        skip[i] = p.dskip ? p.dskip[c] : 0.f;
        sum_skip[i] = sum_bias[i] = 0.f;
    }
    // Buffers over the segment as in the forward, walked backwards: no memory access
    // in the loop is conditional.  Tiles before the first token lie below the
    // buffers' start, which as an unsigned offset is behind their end.
    const bool full = kVec || EPT == 1;
    const bool dead = c0 + pl >= cend;
    const int valid = full ? 1 : (cend - c0 - pl + ES - 1) / ES, here = cend - c0 < CH ? cend - c0 : CH;
    const int held = full ? (dead ? 0 : EPT) : valid;   // the thread's channels in the group
    const uint32_t row = p.D * (uint32_t)sizeof(T), row_bc = p.G * N * (uint32_t)sizeof(T);
    const int tokens = t_end - t_begin;
    auto rows_of = [&](const void* base) {
        return buffer_of(static_cast<const char*>(base) + (((int64_t)b * p.T + t_begin) * p.D + c0) * (int)sizeof(T),
                         tokens > 0 ? (int)((tokens - 1) * row + (cend - c0) * (uint32_t)sizeof(T)) : 0);
    };
    auto rows_of_bc = [&](const void* base, bool on) {
        return buffer_of(static_cast<const char*>(base) + (((int64_t)b * p.T + t_begin) * p.G + g) * N * (int)sizeof(T),
                         on && tokens > 0 ? (int)((tokens - 1) * row_bc + N * (uint32_t)sizeof(T)) : 0);
    };
    const int last = (tiles - 1) * kTile;   // the first tile's first token in the segment
    const uint32_t step = dead ? 0 : kTile * row, step_bc = bt < kTile ? kTile * row_bc : 0;
    uint32_t at = dead ? kNowhere : (last + pt) * row + pl * (uint32_t)sizeof(T);
    uint32_t at_bc = bt < kTile ? (last + bt) * row_bc + bn * (uint32_t)sizeof(T) : kNowhere;
    const __amdgpu_buffer_rsrc_t dt_rows = rows_of(p.dt), dy_rows = rows_of(q.dy), c_rows = rows_of_bc(p.Cm, true);
    __amdgpu_buffer_rsrc_t x_rows, z_rows, b_rows, h_rows, code_rows, scale_rows, dx_rows, ddt_rows, dz_rows, part_rows,
        db_rows, dc_rows;
    // Entry states: fp32, or codes and scales, of the thread's S states of channel hc.
    const int nck = (p.T + kTile - 1) / kTile;
    const bool wide = p.ckpt_bits == 32;
    const uint32_t code_step = hc < here ? (uint32_t)p.D * N : 0, scale_step = hc < here ? 4u * p.D : 0;
    uint32_t code_at = hc < here ? (tiles - 1) * code_step + hc * N + hn : kNowhere / 4;
    uint32_t scale_at = hc < here ? (tiles - 1) * scale_step + 4u * hc : kNowhere;
    // Gradients go out three tiles behind.  dB and dC: E neighbouring ones of the 2 N
    // values of a token per thread, or their partial sums [2 N].
    constexpr int E = kTile * 2 * N / kStepThreads;
    const int rt = tid * E / (2 * N), rn = tid * E % (2 * N);
    const uint32_t row_part = p.G * 2 * N * 4u, step_part = kTile * row_part, step_o = kTile * row_bc;
    uint32_t out_at = dead ? kNowhere : at + 3 * step;
    uint32_t part_at = (last + 3 * kTile + rt) * row_part + rn * 4u;
    uint32_t o_at = (last + 3 * kTile + rt) * row_bc + rn % N * (uint32_t)sizeof(T);
    if constexpr (kGate) z_rows = rows_of(p.z);
    if constexpr (!kMap) {
        const bool part = q.part_bc != nullptr;
        x_rows = rows_of(p.x);
        b_rows = rows_of_bc(p.Bm, true);
        dx_rows = rows_of(q.dx);
        ddt_rows = rows_of(q.ddt);
        if constexpr (kGate) dz_rows = rows_of(q.dz);
        const int64_t crow = ((int64_t)b * nck + t_begin / kTile) * p.D + c0;
        const int size = tiles > 0 ? ((tiles - 1) * p.D + here) * N : 0;
        const char* const base = static_cast<const char*>(p.ckpt);
        h_rows = buffer_of(base + crow * N * 4, wide ? size * 4 : 0);
        code_rows = buffer_of(base + (wide ? 0 : crow * N), wide ? 0 : size);
        scale_rows = buffer_of(base + (wide ? 0 : ckpt_scale_offset((size_t)p.B * nck * p.D * N) + crow * 4),
                               wide || tiles == 0 ? 0 : ((tiles - 1) * p.D + here) * 4);
        part_rows = buffer_of(q.part_bc + (((int64_t)j * p.B * p.T + (int64_t)b * p.T + t_begin) * p.G + g) * (2 * N),
                              part && tokens > 0 ? (int)((tokens - 1) * row_part + 2 * N * 4) : 0);
        db_rows = rows_of_bc(q.dBm, !part);
        dc_rows = rows_of_bc(q.dCm, !part);
    }
    auto load = [&](Loaded<T, N, kVec>& r) {
        r.dt.load(dt_rows, at);
        r.dy.load(dy_rows, at);
        if constexpr (kGate) r.z.load(z_rows, at);
        r.c.load(c_rows, at_bc);
        if constexpr (!kMap) {
            r.x.load(x_rows, at);
            r.b.load(b_rows, at_bc);
            r.h.load(h_rows, code_at * 4);
            if constexpr (S == 2) r.codes = __builtin_amdgcn_raw_buffer_load_b16(code_rows, code_at, 0, 0);
            else r.codes = __builtin_amdgcn_raw_buffer_load_b32(code_rows, code_at, 0, 0);
            r.scale = __builtin_amdgcn_raw_buffer_load_b32(scale_rows, scale_at, 0, 0);
        }
        at -= step;
        at_bc -= step_bc;
        code_at -= code_step;
        scale_at -= scale_step;
    };
    auto stage = [&](const Loaded<T, N, kVec>& r, Kept<EPT>& o, int i) {
        const int t0 = t_begin + last - i * kTile, k = i & 3;
        const int end = len < t_end ? len : t_end;
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            const float v = r.dt.get(e) + bias[e];
            // softplus and its slope 1 / (1 + exp(-v)) from one exponential
            const float ex = exp_raw(-fabsf(v)), w = 1.f + ex, inv = __builtin_amdgcn_rcpf(w);
            const float sp = fmaxf(v, 0.f) + fmaf(__builtin_amdgcn_logf(w), kLn2, ex - (w - 1.f));
            const float sl = inv * (v >= 0.f ? 1.f : ex);
            o.d[e] = p.softplus ? sp : v;
            o.slope[e] = p.softplus ? sl : 1.f;
            const float dout = r.dy.get(e);
            o.x[e] = kMap ? 0.f : r.x.get(e);
            if constexpr (kGate) {
                const float z = r.z.get(e), s = sigmoid(z);
                o.dy[e] = dout * (z * s);
                o.w[e] = dout * (s * fmaf(z, 1.f - s, 1.f));
            } else {
                o.dy[e] = dout;
            }
        }
        const bool partial = t0 + kTile > end;
        // Tokens behind the row's length; channels behind the group, whose rate would be
        // that of the last channel's bias alone, and their states could grow without limit.
        if (partial || here < CH) {
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                const bool on = t0 + pt < end && e < held;
                o.d[e] = on ? o.d[e] : 0.f;
                o.slope[e] = on ? o.slope[e] : 0.f;
                o.x[e] = on ? o.x[e] : 0.f;
                o.dy[e] = on ? o.dy[e] : 0.f;
                if constexpr (kGate) o.w[e] = on ? o.w[e] : 0.f;
            }
        }
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            s_du[k][pt][pl + ES * e] = make_float2(o.d[e], o.d[e] * o.x[e]);
            s_dy[k][pt][pl + ES * e] = o.dy[e];
        }
        if (bt < kTile) {
            const bool inb = !partial || t0 + bt < end;
#pragma unroll
            for (int e = 0; e < BC; ++e) {
                if constexpr (!kMap) s_b[k][bt][bn + e] = inb ? r.b.get(e) : 0.f;
                s_c[k][bt][bn + e] = inb ? r.c.get(e) : 0.f;
            }
        }
        if constexpr (!kMap) {
            const float sc = __uint_as_float(r.scale);
            float h[S];
#pragma unroll
            for (int n = 0; n < S; ++n) {
                const float code = (float)(int8_t)(r.codes >> (8 * n)) * sc, wide_h = r.h.get(n);
                h[n] = wide ? wide_h : code;
            }
            store_cols<S>(&s_h[i & 1][hc][hn], h);
        }
    };
    auto write_out = [&](const Kept<EPT>& o, int i) {
        const int k = i & 1;
        float dx[EPT], ddt[EPT], dz[EPT], s[E];
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            const int c = pl + ES * e, base = c / 16 * PW * 16 + c % 16;
            float du = s_o[k][0][pt][turned(pt, base)], sr = s_o[k][1][pt][turned(pt, base)];
#pragma unroll
            for (int w = 1; w < PW; ++w) {
                du += s_o[k][0][pt][turned(pt, base + 16 * w)];
                sr += s_o[k][1][pt][turned(pt, base + 16 * w)];
            }
            dx[e] = fmaf(du, o.d[e], o.dy[e] * skip[e]);
            ddt[e] = fmaf(du, o.x[e], sr) * o.slope[e];
            if constexpr (kGate) {
                float y = s_y[i & 3][pt][turned(pt, base)];
#pragma unroll
                for (int w = 1; w < PW; ++w) y += s_y[i & 3][pt][turned(pt, base + 16 * w)];
                dz[e] = o.w[e] * fmaf(skip[e], o.x[e], y);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            s[e] = s_red[k][0][rt][rn + e];
#pragma unroll
            for (int c = 1; c < CG; ++c) s[e] += s_red[k][c][rt][rn + e];
        }
        // Tokens behind the row's length: their products are 0 unless the channel's state or
        // gradient is not finite, their outputs 0 all the same.
        const int end = len < t_end ? len : t_end, t0 = t_begin + last - i * kTile;
        if (t0 + kTile > end) {
            const bool in = t0 + pt < end, inb = t0 + rt < end;
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                dx[e] = in ? dx[e] : 0.f;
                ddt[e] = in ? ddt[e] : 0.f;
                if constexpr (kGate) dz[e] = in ? dz[e] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) s[e] = inb ? s[e] : 0.f;
        }
        if (i >= 0 && i < tiles) {
#pragma unroll
            for (int e = 0; e < EPT; ++e) {
                sum_skip[e] = fmaf(o.dy[e], o.x[e], sum_skip[e]);
                sum_bias[e] += ddt[e];
            }
        }
        store_piece<T, kVec>(dx_rows, out_at, valid, dx);
        store_piece<T, kVec>(ddt_rows, out_at, valid, ddt);
        if constexpr (kGate) store_piece<T, kVec>(dz_rows, out_at, valid, dz);
        store_piece<float, true>(part_rows, part_at, 1, s);
        store_piece<T, true>(db_rows, o_at, rn < N, s);
        store_piece<T, true>(dc_rows, o_at, rn >= N, s);
        out_at -= step;
        part_at -= step_part;
        o_at -= step_o;
    };

    Loaded<T, N, kVec> r0, r1;
    Kept<EPT> k0 = {}, k1 = {}, k2 = {}, k3 = {};
    load(r0);
    load(r1);
    auto interval = [&](int i, Loaded<T, N, kVec>& r, Kept<EPT>& o, const Kept<EPT>& done) {
        if constexpr (!kMap) write_out(done, i - 3);
        stage(r, o, i);
        load(r);
        __syncthreads();
    };
    for (int i = 0; i < intervals; i += 4) {
        interval(i, r0, k0, k1);
        if (i + 1 == intervals) break;
        interval(i + 1, r1, k1, k2);
        if (i + 2 == intervals) break;
        interval(i + 2, r0, k2, k3);
        if (i + 3 == intervals) break;
        interval(i + 3, r1, k3, k0);
    }
    if constexpr (!kMap) {
        // The per-channel vectors: sixteen threads hold a channel's tokens.
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            s_o[0][0][pt][pl + ES * e] = sum_skip[e];
            s_o[0][1][pt][pl + ES * e] = sum_bias[e];
        }
        __syncthreads();
        if (tid < CH && c0 + tid < cend) {
            float s0 = 0.f, s1 = 0.f;
            for (int t = 0; t < kTile; ++t) {
                s0 += s_o[0][0][t][tid];
                s1 += s_o[0][1][t][tid];
            }
            *reinterpret_cast<float2*>(q.part_v + (((size_t)seg * p.B + b) * p.D + c0 + tid) * 2) = make_float2(s0, s1);
        }
    }
}

// The partial sums, each element's in order.  Workgroups below bc_blocks: dB and
// dC, the sum over the channel blocks, four elements per thread (N is a multiple
// of 8).  The rest: dA, ddskip and ddt_bias, the sum over `parts` batch rows and
// segments; element e of D N + 2 D is dA's, then the two vectors' interleaved.
template <typename T>
__global__ __launch_bounds__(256) void ssm_sums_kernel(const SsmBwdArgs q, int blocks, size_t rows, unsigned bc_blocks,
                                                       int parts) {
    const int N = q.f.N, D = q.f.D;
    if (blockIdx.x < bc_blocks) {
        const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4, total = rows * 2 * N;
        if (at >= total) return;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < blocks; k += 8) {   // eight loads in flight
            float v[8][4];
#pragma unroll
            for (int u = 0; u < 8; ++u) load_cols<4>(q.part_bc + (k + u < blocks ? k + u : blocks - 1) * total + at, v[u]);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (k + u < blocks) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i] += v[u][i];
                }
            }
        }
        const size_t row = at / (2 * N), n = at % (2 * N);
        T* const to = n < (size_t)N ? static_cast<T*>(q.dBm) + row * N + n : static_cast<T*>(q.dCm) + row * N + n - N;
        Elem<T>::store4(to, make_float4(s[0], s[1], s[2], s[3]));
        return;
    }
    const size_t e = (size_t)(blockIdx.x - bc_blocks) * 256 + threadIdx.x, DN = (size_t)D * N;
    const bool vec = e >= DN;
    if (e >= DN + 2 * (size_t)D) return;
    const size_t i = e - DN;
    float* const out = !vec ? q.dA + e : i % 2 == 0 ? (q.ddskip ? q.ddskip + i / 2 : nullptr)
                                                    : (q.ddt_bias ? q.ddt_bias + i / 2 : nullptr);
    if (!out) return;
    const float* const from = vec ? q.part_v + i : q.part_a + e;
    const size_t stride = vec ? 2 * (size_t)D : DN;
    float s = 0.f;
    for (int k = 0; k < parts; k += 8) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = from[(k + u < parts ? k + u : parts - 1) * stride];
#pragma unroll
        for (int u = 0; u < 8; ++u) s += k + u < parts ? v[u] : 0.f;
    }
    *out = s;
}

template <typename T, int N, bool kVec, bool kGate>
hipError_t launch_bwd_v(const SsmBwdArgs& q, int blocks, hipStream_t stream) {
    constexpr int threads = 2 * kStepThreads;
    const SsmArgs& p = q.f;
    const unsigned per = (unsigned)p.B * p.G * blocks;
    if (per == 0) return hipSuccess;
    if (p.nseg > 1) {
        ssm_bwd_kernel<T, N, kVec, true, kGate, false><<<dim3(per * (p.nseg - 1)), threads, 0, stream>>>(q, blocks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if constexpr (N == 16 || N == 32) {
        if (per * p.nseg > kUnits) {
            ssm_bwd_kernel<T, N, kVec, false, kGate, true><<<dim3(per * p.nseg), threads, 0, stream>>>(q, blocks);
            return hipGetLastError();
        }
    }
    ssm_bwd_kernel<T, N, kVec, false, kGate, false><<<dim3(per * p.nseg), threads, 0, stream>>>(q, blocks);
    return hipGetLastError();
}

template <typename T, int N>
hipError_t launch_bwd(const SsmBwdArgs& q, hipStream_t stream) {
    using S = Shape<N, kStates<N>>;
    const SsmArgs& p = q.f;
    const int Dg = p.D / p.G, blocks = (Dg + S::CH - 1) / S::CH;
    const bool vec = Dg % S::EPT == 0;
    hipError_t e = p.z ? (vec ? launch_bwd_v<T, N, true, true>(q, blocks, stream)
                              : launch_bwd_v<T, N, false, true>(q, blocks, stream))
                       : (vec ? launch_bwd_v<T, N, true, false>(q, blocks, stream)
                              : launch_bwd_v<T, N, false, false>(q, blocks, stream));
    if (e != hipSuccess) return e;
    const size_t rows = (size_t)p.B * p.T * p.G;
    const size_t bc = q.part_bc ? (rows * 2 * N / 4 + 255) / 256 : 0, rest = ((size_t)p.D * (N + 2) + 255) / 256;
    ssm_sums_kernel<T><<<dim3((unsigned)(bc + rest)), 256, 0, stream>>>(q, blocks, rows, (unsigned)bc, p.B * p.nseg);
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
