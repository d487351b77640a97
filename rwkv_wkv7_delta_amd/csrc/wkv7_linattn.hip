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
//
// With as many workgroups as compute units, bound by HBM and by the waves' own instructions
// alike: (8, 4096) tokens, 32 heads of 64, bf16: 126 to 130 us, 4.2 TB/s; reading and writing
// the same bytes in the same order, without arithmetic, takes 123.  With fewer, by a tile's
// products, exponentials and one barrier, 1.9 to 2.4 us (fp32, N = 32, P = 128: 4.2).  64 tokens a
// tile: at N = P = 64 its products with the state and within itself are as much work as each
// other.

#include "wkv7_linattn_device.h"

namespace wkv7 {

namespace {

// The head that a workgroup takes: neighbouring workgroups take heads of different
// groups, so that the heads that read the same keys come G apart (on one XCD where
// G is a multiple of 8).
__device__ __forceinline__ int head_of(int i, int H, int G) { return i % G * (H / G) + i / G; }

// A wave's role: to read out its tokens against kBlocks tiles of 16, or (0) to hold the state.
template <int kBlocks>
struct Blocks {
    static constexpr int value = kBlocks;
};

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
// (8, 4096) tokens, 40 heads of 64, bf16, in reverse with checkpoints: 197 us, 3.4 TB/s (what
// 320 workgroups on 256 units reach in this order).
// Forward (kReverse = false): S from k and v; reverse: its gradient D, from q and
// dy: D <- e^{G_end} D + scale sum_t (e^{G_t} dy_t) q_t^T.
// kSegment: what a segment leaves from zero, and its summed decay.  Else (the
// reverse only) D behind every tile is written, and the gradient of the first state; and
// <S, D> with the tile's checkpoint S, from D's 32 bits.
// Waves 0 to 3 hold the state, 16 value rows each (of 32: and half of the key columns), and
// move it on; waves 4 to 7 bring the tiles: two on their way from memory, one on its way to
// LDS while the others use the one before.
constexpr int kSweepStage = 256;

template <typename T, int N, int PB, bool kReverse, bool kSegment>
__global__ __launch_bounds__(kLaThreads) void la_sweep_kernel(const LaArgs p, const T* kk, const T* vv,
                                                                 const float* first, float* last, T* marks, float* both) {
    typedef LaMat<T> M;
    typedef LaStage<T, N, kSweepStage, kSweepStage> SK;
    typedef LaStage<T, PB, kSweepStage, kSweepStage> SV;
    constexpr int PT = PB / 16, NH = 4 / PT, NT = N / 16 / NH;
    constexpr int kBytes = kLaChunk * (SK::kStride + SV::kStride) * (int)sizeof(T);
    constexpr int BUF = kBytes <= 32 * 1024 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) T s_k[BUF][kLaChunk * SK::kStride];
    __shared__ __attribute__((aligned(16))) T s_v[BUF][kLaChunk * SV::kStride];
    __shared__ LaDecay s_d[BUF];
    // (checkpoints on their way to whole rows)
    constexpr bool kMarks = !kSegment && NH == 1 && sizeof(T) == 2;
    __shared__ __attribute__((aligned(16))) T s_own[4][kMarks ? LaRows16<T, N>::kSize : 8];
    const LaBlock w = la_block<PB>(p);
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, l16 = lane % 16;
    const LaRow row = la_row(p.rows, p.packed, p.tokens, p.T, w.b);
    const int seg = kReverse ? p.nseg - 1 - w.r : w.r;
    const int64_t begin = (int64_t)seg * p.seg_len;
    const int64_t stop = seg == p.nseg - 1 ? row.len : begin + p.seg_len;
    const int end = (int)(stop < row.len ? stop : row.len);
    const bool holds = wave < 4;
    const int ptile = wave % PT * 16, n0 = wave % 4 / PT * (NT * 16);
    const int prow = w.p0 + ptile + l16;
    f32x4 st[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) st[n] = zero4();
    const size_t states = (size_t)p.B * p.H * p.P * N;
    if (holds && !kSegment) {
        const float* from = w.r > 0 ? p.seg_state + (w.r - 1) * states : first;
        if (from) {
            from = state_at<N>(const_cast<float*>(from), p, w.b, w.h, prow) + n0;
#pragma unroll
            for (int n = 0; n < NT; ++n) st[n] = *reinterpret_cast<const f32x4*>(from + 16 * n + 4 * g);
        }
    }
    const int kh = w.h / (p.H / p.G);
    const int64_t krow = (int64_t)p.G * N, vrow = (int64_t)p.H * p.P;
    const int tiles = end > begin ? (int)((end - begin + kLaChunk - 1) / kLaChunk) : 0;
    constexpr bool kDeep = SK::kLoads + SV::kLoads <= 16;
    const auto tile_of = [&](int i) { return kReverse ? tiles - 1 - i : i; };
    // Deep: by twos, the last perhaps a tile without tokens, which changes nothing.
    const int turns = kDeep ? (tiles + 1) / 2 * 2 : tiles;
    double total = 0;
    if (holds) {
        // The 16 value rows of a tile's checkpoint; one tile ahead.
        vu4 part[kMarks ? 1 : NT];
        LaRows16<T, N> whole;
        const auto load_mark = [&](int i) __attribute__((always_inline)) {
            const auto r = buffer_of(static_cast<const T*>(p.ckpt) +
                                         (((row.ckpt + begin / kLaChunk + tile_of(i)) * p.H + w.h) * p.P + w.p0) * N,
                                     both && i < tiles ? PB * N * (int)sizeof(T) : 0);
            if constexpr (kMarks) {
                whole.load(r, N * sizeof(T), ptile);
            } else {
                const uint32_t at = ((ptile + l16) * N + n0 + 4 * g) * (uint32_t)sizeof(T);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if constexpr (sizeof(T) == 2) {
                        const vu2 x = __builtin_bit_cast(vu2, __builtin_amdgcn_raw_buffer_load_b64(r, at + 32 * n, 0, 0));
                        part[n] = vu4{x[0], x[1], 0, 0};
                    } else {
                        part[n] = __builtin_bit_cast(vu4, __builtin_amdgcn_raw_buffer_load_b128(r, at + 64 * n, 0, 0));
                    }
                }
            }
        };
        const auto mark = [&](int n) __attribute__((always_inline)) {   // as the wave holds D
            if constexpr (kMarks) return M::wide(M::four(s_own[wave] + l16 * LaRows16<T, N>::kStride + 16 * n + 4 * g));
            else if constexpr (sizeof(T) == 2) return unpack4(__builtin_bit_cast(bf16x4, vu2{part[n][0], part[n][1]}));
            else return __builtin_bit_cast(f32x4, part[n]);
        };
        if (!kSegment) load_mark(0);
        for (int i = 0; i < turns; ++i) {
            const int buf = BUF == 2 ? i & 1 : 0;
            __syncthreads();
            const LaDecay& d = s_d[buf];
            // (of a tile that there is not: nothing)
            const int64_t tile = row.ckpt + begin / kLaChunk + tile_of(i);
            const auto m = buffer_of(marks + ((tile * p.H + w.h) * p.P + w.p0) * N, i < tiles ? PB * N * (int)sizeof(T) : 0);
            typename M::Half h[NT];
            if (!kSegment) {
                float x = 0.f;
                if constexpr (kMarks) whole.put(s_own[wave]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const f32x4 e = mark(n);
#pragma unroll
                    for (int q = 0; q < 4; ++q) x = fmaf(e[q], st[n][q], x);
                }
                x = sum_rows4(row16_sum(x));
                load_mark(i + 1);
                const auto c = buffer_of(both + ((tile * p.H + w.h) * (p.P / PB) + w.p0 / PB) * 4, both && i < tiles ? 16 : 0);
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), c, lane == 0 ? 4 * wave : kNowhere, 0, 0);
                if constexpr (sizeof(T) == 2) {
                    pack_adjoint(st, g, h);
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n) h[n] = st[n];
                }
            }
            if (kSegment) total += d.sum;
            move_state<T, NT>(st, s_k[buf] + n0, SK::kStride, s_v[buf] + ptile, SV::kStride, kReverse ? d.up : d.down,
                              kReverse ? p.scale : 1.f, d.all, any_odd(d.odd), g, l16);
            if (!kSegment) store_mark<T, N>(s_own[wave], h, m, ptile, n0);
            if (BUF == 1) __syncthreads();
        }
    } else if (turns > 0) {
        struct Ahead {
            SK k;
            SV v;
            LaLog<T> g;
        } even, odd_;
        // No condition on the loads (tiles that there are not have no bytes): how many are
        // under way is then known to the code that waits for the older ones.
        auto load = [&](int i, Ahead& r) {
            const int64_t t0 = begin + (int64_t)tile_of(i) * kLaChunk;
            const int n = i >= tiles ? 0 : (int)(end - t0 < kLaChunk ? end - t0 : kLaChunk);
            const int64_t at = row.first + t0;
            r.k.load(rows_of(kk + at * krow + kh * N, n, krow, N), (uint32_t)(krow * sizeof(T)));
            r.v.load(rows_of(vv + at * vrow + (int64_t)w.h * p.P + w.p0, n, vrow, PB), (uint32_t)(vrow * sizeof(T)));
            r.g.load(p, at, w.h, n);
        };
        auto put = [&](int buf, const Ahead& r) {
            r.k.store(s_k[buf]);
            r.v.store(s_v[buf]);
            const bool odd = __builtin_amdgcn_ballot_w64((int)r.k.odd() | (int)r.v.odd()) != 0;
            if (lane == 0) {
                s_d[buf].odd[wave] = odd;
                s_d[buf].odd[wave - 4] = 0;
            }
            if (wave == 4) put_decays(s_d[buf], r.g.get());
        };
        auto turn = [&](int i, Ahead& r) {
            __syncthreads();
            if (BUF == 1) __syncthreads();
            put(BUF == 2 ? i & 1 ^ 1 : 0, r);
            load(i + (kDeep ? 3 : 2), r);
        };
        load(0, even);
        if (kDeep) load(1, odd_);
        put(0, even);
        load(kDeep ? 2 : 1, even);
        for (int i = 0; i < turns; i += kDeep ? 2 : 1) {
            turn(i, kDeep ? odd_ : even);
            if (kDeep) turn(i + 1, even);
        }
    }
    if (holds && last && (kSegment || w.r == p.nseg - 1)) {
        float* const to = state_at<N>(last + (kSegment ? w.r * states : 0), p, w.b, w.h, prow) + n0;
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
    constexpr int kAtOnce = 8;   // loads on their way while the chain waits for none
    for (int r0 = 0; r0 + 1 < p.nseg; r0 += kAtOnce) {
        f32x4 x[kAtOnce];
        float d[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int r = r0 + i + 1 < p.nseg ? r0 + i : r0;
            x[i] = *reinterpret_cast<const f32x4*>(p.seg_state + r * states + e);
            d[i] = exp2_raw((float)p.seg_decay[r * heads + head]);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (r0 + i + 1 < p.nseg) {
                s = s * d[i] + x[i];
                *reinterpret_cast<f32x4*>(p.seg_state + (r0 + i) * states + e) = s;
            }
        }
    }
}

// ---- prompts --------------------------------------------------------------------
// A workgroup takes 64 (or all 32) value rows of a head's state over a segment.  Waves 4 to 7
// hold the state, 16 value rows each (of 32: and half of the columns): each tile's queries read
// it out from its registers, in terms, then it is moved on.  Waves 0 to 3 read out the tile
// itself: wave w the tokens 16 w .. , to which it adds what the others read from the state, and
// stores them.  Results are formed transposed, [s][t], [p][t], [n][p], so that each feeds the
// next product from registers (wkv7_linattn_device.h); the state is both kinds of operand as it
// is held.  (Handed on through LDS for the others to read, in two bf16 terms, it cost 12 us of the
// prompts above: four waves each read all of it.)
template <typename T, int N, int PB, bool kMarks>
struct LaFwdShared {
    typedef LaStage<T, N> SK;
    typedef LaStage<T, PB> SV;
    static constexpr int kHalves = 64 / PB;      // waves that share value rows, with N / kHalves columns each
    static constexpr int kXStride = PB + 4;      // of a row of what is read from the state
    // Two of everything, and one barrier a tile, where that takes at most 128 KiB (registers leave
    // room for one workgroup on a unit in any case): (4, 2048) tokens, 32 heads of 128, bf16, 123
    // KiB: 100 us, with one set 110; (8, 2048), 32 heads of 64, fp32, 139 KiB: 279 and 185.
    static constexpr int kSet = kLaChunk * ((2 * SK::kStride + SV::kStride) * (int)sizeof(T) + kHalves * kXStride * 4);
    static constexpr int kBuffers = 2 * kSet <= 128 * 1024 ? 2 : 1;
    T k[kBuffers][kLaChunk * SK::kStride], q[kBuffers][kLaChunk * SK::kStride];
    T v[kBuffers][kLaChunk * SV::kStride];
    float x[kBuffers][kHalves][kLaChunk * kXStride];   // S q_t, [t][p]
    T own[4][LaRows16<T, PB>::kSize];   // a wave's results
    T mark[4][kMarks && sizeof(T) == 2 && PB == 64 ? LaRows16<T, N>::kSize : 8];   // a wave's state rows
    LaDecay d[kBuffers];
};

// (kMarks: with checkpoints.)
template <typename T, int N, int PB, bool kMarks>
__global__ __launch_bounds__(kLaThreads) void la_fwd_kernel(const LaArgs p) {
    typedef LaMat<T> M;
    typedef LaStage<T, N> SK;
    typedef LaStage<T, PB> SV;
    typedef LaRows16<T, N> SQ;
    typedef LaFwdShared<T, N, PB, kMarks> Shared;
    typedef typename M::Frag Frag;
    constexpr int PT = PB / 16, NT = N / 16 * PT / 4, KS = N / 32, BUF = Shared::kBuffers;
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
    // The state's wave: value rows ptile .., columns n0 ..
    const int ptile = wave % PT * 16, n0 = (wave % 4) / PT * (NT * 16);
    const int prow = w.p0 + ptile + l16;
    const size_t states = (size_t)p.B * p.H * p.P * N;
    const int kh = w.h / (p.H / p.G);
    const int64_t krow = (int64_t)p.G * N, vrow = (int64_t)p.H * p.P;
    const uint32_t kb = (uint32_t)(krow * sizeof(T)), vb = (uint32_t)(vrow * sizeof(T));
    const int tiles = end > begin ? (int)((end - begin + kLaChunk - 1) / kLaChunk) : 0;
    T* const Y = static_cast<T*>(p.y);
    // Two tiles are on their way from memory at any time (at a copy's rate, what a unit has
    // in flight has to cover about 2 us); one where the registers hold no more.
    struct Ahead {
        SK k;
        SV v;
        SQ q;
        LaLog<T> g;
    };
    constexpr bool kDeep = SK::kLoads + SV::kLoads + SQ::kEach <= 12;
    const auto tokens_of = [&](int c, int64_t to) {   // of tile c
        const int64_t n = to - (begin + (int64_t)c * kLaChunk);
        return (int)(n < 0 ? 0 : n < kLaChunk ? n : kLaChunk);
    };
    f32x4 st[NT];
    // A wave's whole way over the segment, by its role: the code that waits for older loads
    // has to know how many younger loads and stores there are, so no role's are conditional
    // for another and tiles that there are not are loaded as nothing.
    auto run = [&](auto blocks_) {
        constexpr int kBlocks = decltype(blocks_)::value;
        constexpr bool kReads = kBlocks > 0;
        const int t = 16 * wave + l16;   // the read-out's token
        Frag qf[KS];
        f32x4 o[PT];
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) o[pt] = zero4();
        float tup = 0.f;
        // Where the next tile to be loaded is, the next one to be stored, and the next state;
        // the tokens from there on.  Kept from turn to turn: formed anew from the tile's number
        // they were a sixth of a wave's instructions.
        int64_t at = row.first + begin;
        int left = end - (int)begin;
        const int64_t kat = at * krow + kh * N, vat = at * vrow + (int64_t)w.h * p.P + w.p0;
        const T* at_k = static_cast<const T*>(p.k) + kat;
        const T* at_q = static_cast<const T*>(p.q) + kat;
        const T* at_v = static_cast<const T*>(p.v) + vat;
        T* at_y = Y + vat;
        T* at_mark = static_cast<T*>(p.ckpt) + (((row.ckpt + begin / kLaChunk) * p.H + w.h) * p.P + w.p0) * N;
        auto load = [&](Ahead& r) {
            const int n = left < 0 ? 0 : left < kLaChunk ? left : kLaChunk;
            r.k.load(rows_of(at_k, n, krow, N), kb);
            r.v.load(rows_of(at_v, n, vrow, PB), vb);
            if constexpr (kReads) {
                r.q.load(rows_of(at_q, n, krow, N), kb, 16 * wave);
                if constexpr (kBlocks == 1) r.g.load(p, at, w.h, n);
            }
            at += kLaChunk;
            at_k += kLaChunk * krow;
            at_q += kLaChunk * krow;
            at_v += kLaChunk * vrow;
            left -= kLaChunk;
        };
        auto put = [&](int buf, const Ahead& r) {
            r.k.store(sm.k[buf]);
            r.v.store(sm.v[buf]);
            const bool odd = __builtin_amdgcn_ballot_w64((int)r.k.odd() | (int)r.v.odd()) != 0;
            sm.d[buf].odd[wave] = odd;   // (64 lanes alike: no branch)
            if constexpr (kReads) {
                if (kBlocks == 1) put_decays(sm.d[buf], r.g.get());
                T* const own = sm.q[buf] + 16 * wave * SQ::kStride;
                r.q.put(own);
#pragma unroll
                for (int i = 0; i < KS; ++i) qf[i] = M::rows(own + l16 * SQ::kStride + 32 * i + 8 * g);
            }
        };
        // Tile c's read-outs with what the state's waves found for them, to memory (before the
        // first tile: no rows).
        auto finish = [&](int c, int buf) {
            const int n_in = tokens_of(c, end), n_out = c < 0 ? 0 : tokens_of(c, zero_end);
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) {
                const float* const x1 = sm.x[buf][0] + t * Shared::kXStride + 16 * pt + 4 * g;
                f32x4 x = *reinterpret_cast<const f32x4*>(x1);
                if constexpr (Shared::kHalves == 2) x += *reinterpret_cast<const f32x4*>(x1 + kLaChunk * Shared::kXStride);
#pragma unroll
                for (int q = 0; q < 4; ++q) o[pt][q] = fmaf(x[q], tup, o[pt][q]) * p.scale;
            }
            // nothing of a state that is not finite behind the row's last token
            if (n_in < kLaChunk)
#pragma unroll
                for (int pt = 0; pt < PT; ++pt)
#pragma unroll
                    for (int q = 0; q < 4; ++q) o[pt][q] = t < n_in ? o[pt][q] : 0.f;
            LaRows16<T, PB>::store(sm.own[wave % 4], o,
                                   rows_of(at_y, n_out, vrow, PB), vb, 16 * wave);
            at_y += c < 0 ? 0 : kLaChunk * vrow;
        };
        auto turn = [&](int c, Ahead& r) {
            const int buf = BUF == 2 ? c & 1 : 0, nxt = BUF == 2 ? buf ^ 1 : 0;
            __syncthreads();
            const T* const sk = sm.k[buf];
            const T* const sv = sm.v[buf];
            const T* const sq = sm.q[buf];
            const LaDecay& d = sm.d[buf];
            const bool odd = any_odd(d.odd);
            if constexpr (kReads) {
                if (BUF == 2) finish(c - 1, nxt);
                const int n_in = tokens_of(c, end);
                const float thi = d.hi[t], tlo = d.lo[t];
                tup = d.up[t];
#pragma unroll
                for (int pt = 0; pt < PT; ++pt) o[pt] = zero4();
                if (!odd) {
                    // [s][t] of the wave's tokens t against those up to them.
                    Frag pf[2][M::kTerms];
#pragma unroll
                    for (int j2 = 0; j2 < 2; ++j2) {
                        typename M::Half h2[2][M::kTerms];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int j = 2 * j2 + u;
                            f32x4 a = zero4();
                            if (j < kBlocks) {
#pragma unroll
                                for (int i = 0; i < KS; ++i)
                                    a = M::mma(M::rows(sk + (16 * j + l16) * SK::kStride + 32 * i + 8 * g), qf[i], a);
                                const f32x4 shi = *reinterpret_cast<const f32x4*>(d.hi + 16 * j + 4 * g);
                                const f32x4 slo = *reinterpret_cast<const f32x4*>(d.lo + 16 * j + 4 * g);
#pragma unroll
                                for (int q = 0; q < 4; ++q) a[q] *= exp2_raw((thi - shi[q]) + (tlo - slo[q]));
                                if (j == kBlocks - 1)   // the triangle's edge
#pragma unroll
                                    for (int q = 0; q < 4; ++q) a[q] = 4 * g + q <= l16 ? a[q] : 0.f;
                            }
                            split_terms<T>(a, h2[u]);
                        }
#pragma unroll
                        for (int e = 0; e < M::kTerms; ++e) pf[j2][e] = M::cat(h2[0][e], h2[1][e]);
                    }
#pragma unroll
                    for (int pt = 0; pt < PT; ++pt) {
                        const Frag v0 = columns<T>(sv + 16 * pt, SV::kStride, g, l16);
#pragma unroll
                        for (int e = M::kTerms - 1; e >= 0; --e) o[pt] = M::mma(v0, pf[0][e], o[pt]);
                        if (kBlocks > 2) {
                            const Frag v1 = columns<T>(sv + 32 * SV::kStride + 16 * pt, SV::kStride, g, l16);
#pragma unroll
                            for (int e = M::kTerms - 1; e >= 0; --e) o[pt] = M::mma(v1, pf[1][e], o[pt]);
                        }
                    }
                } else {
                    // An infinity or a NaN among the tile's keys and values: pair by pair, each lane its
                    // token, so that it meets no weight of 0 of a token before its own.
                    for (int s = 0; s < n_in; ++s) {
                        float a = 0.f;
#pragma unroll 2
                        for (int n = 0; n < N; ++n)
                            a = fmaf(Elem<T>::load1(sk + s * SK::kStride + n), Elem<T>::load1(sq + t * SK::kStride + n), a);
                        a *= exp2_raw((thi - d.hi[s]) + (tlo - d.lo[s]));
#pragma unroll
                        for (int pt = 0; pt < PT; ++pt) {
                            const f32x4 x = M::wide(M::four(sv + s * SV::kStride + 16 * pt + 4 * g)) * a;
#pragma unroll
                            for (int q = 0; q < 4; ++q) o[pt][q] += s <= t ? x[q] : 0.f;
                        }
                    }
                }
            } else {
                // ---- the state read out, [p][t], as the lanes hold it
                constexpr int kDepth = (NT + 1) / 2;   // (of 16 columns: the other half zeros)
                Frag sf[kDepth][M::kTerms];
#pragma unroll
                for (int i = 0; i < kDepth; ++i) {
                    typename M::Half h2[2][M::kTerms];
#pragma unroll
                    for (int u = 0; u < 2; ++u) split_terms<T>(2 * i + u < NT ? st[2 * i + u] : zero4(), h2[u]);
#pragma unroll
                    for (int e = 0; e < M::kTerms; ++e) sf[i][e] = M::cat(h2[0][e], h2[1][e]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f32x4 x = zero4();
#pragma unroll
                    for (int i = 0; i < kDepth; ++i) {
                        const T* const q1 = sq + (16 * j + l16) * SK::kStride + n0 + 32 * i + 4 * g;
                        const Frag q2 = M::cat(M::four(q1), NT > 1 ? M::four(q1 + 16) : typename M::Half{});
#pragma unroll
                        for (int e = M::kTerms - 1; e >= 0; --e) x = M::mma(sf[i][e], q2, x);
                    }
                    *reinterpret_cast<f32x4*>(sm.x[buf][wave % 4 / PT] + (16 * j + l16) * Shared::kXStride + ptile + 4 * g) = x;
                }
                typename M::Half was[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) was[n] = M::half(st[n]);
                move_state<T, NT>(st, sk + n0, SK::kStride, sv + ptile, SV::kStride, d.down, 1.f, d.all, odd, g, l16);
                if constexpr (kMarks) {
                    store_mark<T, N>(sm.mark[wave - 4], was, buffer_of(at_mark, c < tiles ? PB * N * (int)sizeof(T) : 0), ptile, n0);
                    at_mark += (int64_t)p.H * p.P * N;
                }
            }
            if (BUF == 1) {
                __syncthreads();
                if constexpr (kReads) finish(c, 0);
            }
            put(nxt, r);
            load(r);
        };
        if constexpr (!kReads) {
#pragma unroll
            for (int n = 0; n < NT; ++n) st[n] = zero4();
            const float* from = w.r > 0 ? p.seg_state + (w.r - 1) * states : p.s0;
            if (from) {
                from = state_at<N>(const_cast<float*>(from), p, w.b, w.h, prow) + n0;
#pragma unroll
                for (int n = 0; n < NT; ++n) st[n] = *reinterpret_cast<const f32x4*>(from + 16 * n + 4 * g);
            }
        }
        if (tiles > 0) {
            Ahead even, odd_;
            load(even);
            if (kDeep) load(odd_);
            put(0, even);
            load(even);
            // Deep: by twos, the last perhaps a tile without tokens, which changes nothing.
            int c = 0;
            for (; c < tiles; c += kDeep ? 2 : 1) {
                turn(c, kDeep ? odd_ : even);
                if (kDeep) turn(c + 1, even);
            }
            if (BUF == 2) {
                __syncthreads();
                if constexpr (kReads) finish(c - 1, c - 1 & 1);
            }
        }
    };
    const bool reads = wave < 4;
    if (wave == 0) run(Blocks<1>());
    else if (wave == 1) run(Blocks<2>());
    else if (wave == 2) run(Blocks<3>());
    else if (wave == 3) run(Blocks<4>());
    else run(Blocks<0>());
    if (!reads && tail && p.sT) {
        float* const to = state_at<N>(p.sT, p, w.b, w.h, prow) + n0;
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
// a lane's 16-byte loads in flight).  Bound by the states' bytes: 256 rows of 40 heads of
// 64 x 64 take 73 us, 4.6 TB/s.  With slots every wave looks through the rows before its own
// for the same slot: 256, 4096 and 65536 rows of one head of 32 x 32 take 12, 21 and 2240 us,
// without slots 11, 12 and 98.
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
            p, static_cast<const T*>(p.k), static_cast<const T*>(p.v), nullptr, p.seg_state, nullptr, nullptr);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        la_join_kernel<<<(unsigned)(((size_t)p.B * p.H * p.P * N / 4 + 255) / 256), 256, 0, stream>>>(p, p.s0);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (p.ckpt) la_fwd_kernel<T, N, PB, true><<<blocks * p.nseg, kLaThreads, 0, stream>>>(p);
    else la_fwd_kernel<T, N, PB, false><<<blocks * p.nseg, kLaThreads, 0, stream>>>(p);
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
            p, Q, dY, nullptr, p.seg_state, nullptr, nullptr);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        la_join_kernel<<<(unsigned)(((size_t)p.B * p.H * p.P * N / 4 + 255) / 256), 256, 0, stream>>>(p, q.dsT);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    la_sweep_kernel<T, N, PB, true, false><<<blocks * p.nseg, kLaThreads, 0, stream>>>(
        p, Q, dY, q.dsT, q.ds0, static_cast<T*>(q.adj), q.both);
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
