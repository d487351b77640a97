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
//
// (8, 4096) tokens, 40 heads of 64, bf16: 377 to 415 us, 3.8 TB/s, behind a sweep of 197.  Bound
// by HBM and by the waves' own work (products, LDS, addresses), which overlap in part: with dk
// and dv on the same waves 527 us, of which the arithmetic alone took 394, the bytes alone 352
// (with weights and D in one bf16 term each; the second terms add 10 us, unpacking D 12).

#include "wkv7_linattn_device.h"

namespace wkv7 {

namespace {

// Twelve waves: four for dq, four for dk, four for dv; the last eight bring the tiles.
constexpr int kBwdThreads = 768, kBwdStage = 512, kBwdFirst = 256;
template <typename T, int W>
using LaBwdStage = LaStage<T, W, kBwdStage, kBwdFirst>;

template <typename T, int N, int PB>
struct LaBwdShared {
    typedef LaBwdStage<T, N> SK;
    typedef LaBwdStage<T, PB> SV;
    T q[kLaChunk * SK::kStride], k[kLaChunk * SK::kStride];
    T v[kLaChunk * SV::kStride], dy[kLaChunk * SV::kStride];
    T s[PB * SK::kStride], ds[LaMat<T>::kTerms][PB * SK::kStride];   // [p][n]; ds in terms
    // A wave's results on their way to whole rows (fp32 rows go there by themselves).
    T own[sizeof(T) == 2 ? 12 : 1][sizeof(T) == 2 ? LaRows16<T, (N > PB ? N : PB)>::kSize : 16];
    LaDecay d[2];                                  // of this head and the next
    // For dg, of this head and the one before: sums of M down its columns, by wave; a and M's
    // sums along its rows; b; the parts of <S, D>.
    struct {
        float col[4][kLaChunk], a[kLaChunk], b[kLaChunk], c[8];
    } g[2];
    int odd[8];
};

// PB state rows of N on their way to LDS (64 rows of LaStage, or 32).
template <typename T, int N, int PB>
struct LaStateStage {
    static constexpr int kPieces = N * (int)sizeof(T) / 16;
    static constexpr int kLoads = PB * kPieces / kBwdStage;
    static constexpr int kStride = N + 16 / (int)sizeof(T);
    vu4 w[kLoads > 0 ? kLoads : 1];
    __device__ __forceinline__ static int piece(int i) { return (i * kBwdStage + threadIdx.x - kBwdFirst) % (PB * kPieces); }
    // Rows are one behind the other in memory; none where there is no tile.
    __device__ __forceinline__ void load(const T* p, bool some) {
        const auto r = buffer_of(p, some ? PB * N * (int)sizeof(T) : 0);
#pragma unroll
        for (int i = 0; i < (kLoads > 0 ? kLoads : 1); ++i)
            w[i] = __builtin_bit_cast(vu4, __builtin_amdgcn_raw_buffer_load_b128(r, piece(i) * 16, 0, 0));
    }
    __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
        for (int i = 0; i < (kLoads > 0 ? kLoads : 1); ++i) {
            const int at = piece(i);
            *reinterpret_cast<vu4*>(lds + at / kPieces * kStride + at % kPieces * (16 / (int)sizeof(T))) = w[i];
        }
    }
    // An adjoint state as the sweep leaves it, in terms.
    vu4 term[sizeof(T) == 2 ? (kLoads > 0 ? kLoads : 1) : 1][2];
    __device__ __forceinline__ void unpack() {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < (kLoads > 0 ? kLoads : 1); ++i) unpack_adjoint(w[i], term[i]);
        }
    }
    __device__ __forceinline__ void store_terms(T (&lds)[LaMat<T>::kTerms][PB * kStride]) const {
        if constexpr (sizeof(T) == 4) {
            store(lds[0]);
        } else {
#pragma unroll
            for (int i = 0; i < (kLoads > 0 ? kLoads : 1); ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int at = piece(i);
                    *reinterpret_cast<vu4*>(lds[e] + at / kPieces * kStride + at % kPieces * 8) = term[i][e];
                }
        }
    }
};

// Decays between the lane's token and those of tile j: in register r, token 16 j + 4 g + r.
__device__ __forceinline__ f32x4 decays(const LaDecay& d, int j, int g, float hi, float lo, bool later) {
    const f32x4 ohi = *reinterpret_cast<const f32x4*>(d.hi + 16 * j + 4 * g);
    const f32x4 olo = *reinterpret_cast<const f32x4*>(d.lo + 16 * j + 4 * g);
    f32x4 e;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        e[r] = exp2_raw(later ? (ohi[r] - hi) + (olo[r] - lo) : (hi - ohi[r]) + (lo - olo[r]));
    return e;
}

// A wave's role.
template <int kRole>
struct Role {
    static constexpr int value = kRole;
};
constexpr int kDq = 0, kDk = 1, kDv = 2;

// What a workgroup has before it: a tile of one group of heads (or of a part of them), and of
// these one head and PB of its value rows.
struct LaUnit {
    // (no gaps between the members: copies of them would go through memory)
    int valid, part, step, steps;
    int n_in, n_out;        // the tile's tokens, and places that are written
    int64_t h;
    int64_t at;             // the tile's first token among all
    int64_t tile;           // its checkpoint's number
    int64_t kat, vat, sat;  // where its keys, values and states are, in elements
};

// Tiles of 64 tokens stand alone, so a workgroup goes from one to the next (as many
// workgroups as the device holds at once, in turn) with the next one's loads on their
// way while it computes.  Waves w, 4 + w and 8 + w have the tokens 16 w ..: as queries, for
// dq, against the keys before; as keys, for dk and for dv, against the queries behind.  Each
// SIMD has one of each.  The sums over the heads that share a key stay in registers.
template <typename T, int N, int PB>
__global__ __launch_bounds__(kBwdThreads) void la_bwd_kernel(const LaBwdArgs o, int blocks) {
    typedef LaMat<T> M;
    typedef LaBwdStage<T, N> SK;
    typedef LaBwdStage<T, PB> SV;
    typedef typename M::Frag Frag;
    typedef typename M::Half Half;
    constexpr int NT = N / 16, PT = PB / 16, KS = N / 32, PS = PB / 32;
    __shared__ __attribute__((aligned(16))) LaBwdShared<T, N, PB> sm;
    const LaArgs& p = o.f;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, l16 = lane % 16;
    const int w = wave % 4;
    const int shared = p.H / p.G, per = (shared + o.split - 1) / o.split, pblocks = p.P / PB;   // (1, 2 or 4)
    const int parts = p.P < 64 ? 4 : p.P / 16;   // of <S, D>
    const int krow = p.G * N, vrow = p.H * p.P;
    // The pointers are read from the kernel's arguments where they are used: kept in scalar
    // registers over the loop, they and the buffers made of them are more than there are.
    typedef const __attribute__((address_space(4))) LaBwdArgs* Args;
    const auto args = [&]() __attribute__((always_inline)) {
        Args a = (Args)__builtin_amdgcn_kernarg_segment_ptr();
        asm volatile("" : "+s"(a));
        return a;
    };
    const int t = 16 * w + l16;   // the lane's token
    // Results of the wave's 16 tokens, rows of W, n of the tile's written.
    const auto store_rows = [&](auto& x, T* to, int n, int64_t stride) __attribute__((always_inline)) {
        constexpr int W = 16 * (int)(sizeof(x) / sizeof(f32x4));
        const auto r = rows_of(to, n, stride, W);
        const uint32_t bytes = (uint32_t)(stride * (int64_t)sizeof(T));
        if constexpr (sizeof(T) == 2) {
            LaRows16<T, W>::store(sm.own[wave], x, r, bytes, 16 * w);
        } else {
#pragma unroll
            for (int e = 0; e < W / 16; ++e)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(vu4, x[e]), r, t * bytes + (16 * e + 4 * g) * 4, 0, 0);
        }
    };
    // n rows of W zeros, by all threads.
    const auto zero_rows = [&](auto* to, int n, int64_t stride, int W) __attribute__((always_inline)) {
        constexpr int kSize = (int)sizeof(*to);
        const auto r = rows_of(to, n, stride, W);
        const int pieces = W * kSize / 16;
        for (int from = 0; from < kLaChunk * pieces; from += kBwdThreads) {
            const int e = from + (int)threadIdx.x, row = e / pieces;
            __builtin_amdgcn_raw_buffer_store_b128(vu4{0, 0, 0, 0}, r, row < kLaChunk
                ? row * (uint32_t)(stride * kSize) + e % pieces * 16 : kNowhere, 0, 0);
        }
    };
    const auto first_of_head = [&](const LaUnit& u) __attribute__((always_inline)) { return (u.step & (pblocks - 1)) == 0; };
    const auto to_next_step = [&](LaUnit& u) __attribute__((always_inline)) {
        ++u.step;
        u.h += first_of_head(u);
        u.vat += PB;
        u.sat += PB * N;
    };
    // A wave's whole way, by its role (so that the code that waits for loads knows how many
    // stores were issued behind them).
    auto run = [&](auto role_) __attribute__((always_inline)) {
    constexpr int kRole = decltype(role_)::value;
    // Units are numbered row by row, tile by tile, part by part, group by group: this
    // workgroup's, and the distance to its next one, digit by digit.
    int at_kh, at_part, at_c, at_b, by_kh, by_part, by_c, by_b;
    const auto digits = [&](unsigned i, int& kh, int& part, int& c, int& b) __attribute__((always_inline)) {
        kh = (int)(i % p.G);
        i /= p.G;
        part = (int)(i % o.split);
        i /= o.split;
        c = (int)(i % blocks);
        b = (int)(i / blocks);
    };
    digits(blockIdx.x, at_kh, at_part, at_c, at_b);
    digits(gridDim.x, by_kh, by_part, by_c, by_b);
    const auto skip = [&]() __attribute__((always_inline)) {
        at_kh += by_kh;
        int over = at_kh >= p.G;
        at_kh -= over ? p.G : 0;
        at_part += by_part + over;
        over = at_part >= o.split;
        at_part -= over ? o.split : 0;
        at_c += by_c + over;
        over = at_c >= blocks;
        at_c -= over ? blocks : 0;
        at_b += by_b + over;
    };
    int64_t tile = -1;   // of the unit's row, the last one taken
    // The next unit with tokens.  A unit is every tile of a row whose number is c0 modulo
    // `blocks` (more than one only where a packed row is longer than the call says); tiles of
    // padding get their zeros here.
    auto advance = [&]() __attribute__((always_inline)) {
        LaUnit u;
        u.valid = 0;
        for (; at_b < p.B; skip(), tile = -1) {
            const LaRow row = la_row(p.rows, p.packed, p.tokens, p.T, at_b);
            tile = tile < 0 ? at_c : tile + blocks;
            if (tile * kLaChunk >= row.stored) continue;
            const int t0 = (int)tile * kLaChunk, kh = at_kh;
            u.part = at_part;
            u.at = row.first + t0;
            u.n_in = row.len - t0 < kLaChunk ? (row.len > t0 ? row.len - t0 : 0) : kLaChunk;
            u.n_out = row.stored - t0 < kLaChunk ? row.stored - t0 : kLaChunk;
            u.step = 0;
            const int heads = shared - u.part * per < per ? shared - u.part * per : per;
            u.steps = heads * pblocks;
            u.h = kh * shared + u.part * per;
            u.kat = u.at * krow + kh * N;
            u.vat = u.at * vrow + u.h * p.P;
            u.tile = row.ckpt + tile;
            u.sat = (u.tile * vrow + u.h * p.P) * N;
            if (u.n_in > 0) {
                u.valid = 1;
                break;
            }
            // (through buffers, which end behind the last row: the lanes stay together)
            for (; u.step < u.steps; to_next_step(u)) {
                zero_rows(static_cast<T*>(args()->dv) + u.vat, u.n_out, vrow, PB);
                if (!o.dg || !first_of_head(u)) continue;
                const auto r = rows_of(static_cast<T*>(args()->dg) + u.at * p.H + u.h, u.n_out, p.H, 1);
                const uint32_t at = threadIdx.x < kLaChunk ? threadIdx.x * p.H * (uint32_t)sizeof(T) : kNowhere;
                if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16((unsigned short)0, r, at, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b32(0u, r, at, 0, 0);
            }
            if (o.split > 1) {
                const int64_t to = (p.packed ? p.tokens : (int64_t)p.B * p.T) * krow * u.part + u.kat;
                zero_rows(args()->part_q + to, u.n_out, krow, N);
                zero_rows(args()->part_k + to, u.n_out, krow, N);
            } else {
                zero_rows(static_cast<T*>(args()->dq) + u.kat, u.n_out, krow, N);
                zero_rows(static_cast<T*>(args()->dk) + u.kat, u.n_out, krow, N);
            }
        }
        return u;
    };
    SK rq, rk;
    SV rv, ry;
    LaStateStage<T, N, PB> rs, rd;
    LaLog<T> lg;
    float both1 = 0.f;   // (of the next unit)
    auto load = [&](const LaUnit& u) __attribute__((always_inline)) {
        const int n = u.valid ? u.n_in : 0, n_qk = u.step == 0 ? n : 0;
        const uint32_t kb = (uint32_t)krow * sizeof(T), vb = (uint32_t)vrow * sizeof(T);
        const Args a = args();
        if constexpr (kRole == kDq) {
            lg.load(p, u.at, (int)u.h, n);
            // with a head's first step, its parts of <S, D>, one to a lane
            const auto r = buffer_of(a->both + (u.tile * p.H + u.h) * parts, o.dg && n > 0 && first_of_head(u) ? 4 * parts : 0);
            both1 = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, 4 * lane, 0, 0));
            return;
        }
        rq.load(rows_of(static_cast<const T*>(a->f.q) + u.kat, n_qk, krow, N), kb);
        rk.load(rows_of(static_cast<const T*>(a->f.k) + u.kat, n_qk, krow, N), kb);
        rv.load(rows_of(static_cast<const T*>(a->f.v) + u.vat, n, vrow, PB), vb);
        ry.load(rows_of(static_cast<const T*>(a->dy) + u.vat, n, vrow, PB), vb);
        rs.load(static_cast<const T*>(a->f.ckpt) + u.sat, u.valid);
        rd.load(static_cast<const T*>(a->adj) + u.sat, u.valid);
    };
    // dg of a head once the sums over its tile are in LDS, by one wave.  Lane l: what counts
    // for token 63 - l, from behind it; what counts for token l, from before it.  In 64 bits:
    // the rows and columns of M cancel where both lie on one side.
    // (the head whose dg is still to be written)
    int64_t behind_at = 0;
    int behind_h = 0, behind_in = 0, behind_out = 0, behind_buf = 0;
    float behind_all = 0.f;
    auto finish_dg = [&]() __attribute__((always_inline)) {
        const int u = 63 - lane;
        const auto& sg = sm.g[behind_buf];
        double x = sg.a[u];
#pragma unroll
        for (int j = 0; j < 4; ++j) x -= u < 16 * j + 16 ? (double)sg.col[j][u] : 0.0;
        x = wave_running_sum(x);
        const double y = wave_running_sum(lane > 0 ? (double)sg.b[lane - 1] : 0.0);
        double both = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) both += sg.c[j];   // (0 behind the last)
        const float dg = (float)(x + __shfl(y, u) + behind_all * both);
        if (u < behind_out) Elem<T>::store1(static_cast<T*>(args()->dg) + (behind_at + u) * p.H + behind_h, u < behind_in ? dg : 0.f);
    };
    const auto after = [&](const LaUnit& u) __attribute__((always_inline)) {
        LaUnit n = u;
        if (!u.valid) return n;
        to_next_step(n);
        return n.step == n.steps ? advance() : n;
    };
    LaUnit u = advance();
    if (!u.valid) return;
    LaUnit next = after(u);
    load(u);
    if (kRole == kDq && wave == 0) put_decays(sm.d[0], lg.get());
    int dbuf = 0, gbuf = 0;
    bool waits = false;   // a head's dg
    f32x4 sum[NT];        // dq or dk of the lane's token
    float asum = 0.f, csum = 0.f;
    bool odd_qk = false;
    while (u.valid) {
        const int n_in = u.n_in, n_out = u.n_out;
        const bool in = t < n_in;
        const bool head_first = first_of_head(u), head_last = ((u.step + 1) & (pblocks - 1)) == 0;
        if constexpr (kRole != kDq) rd.unpack();
        __syncthreads();   // the tiles before have been read
        if (u.step == 0) {
            if constexpr (kRole != kDq) {
                rq.store(sm.q);
                rk.store(sm.k);
                odd_qk = rq.odd() || rk.odd();
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) sum[n] = zero4();
        }
        if (head_first) asum = csum = 0.f;
        csum += both1;
        if constexpr (kRole != kDq) {
            rv.store(sm.v);
            ry.store(sm.dy);
            rs.store(sm.s);
            rd.store_terms(sm.ds);
            const bool odd_lane = __builtin_amdgcn_ballot_w64(odd_qk || rv.odd() || ry.odd()) != 0;
            if (lane == 0) sm.odd[wave - 4] = odd_lane;
        }
        __syncthreads();
        load(next);
        if (kRole == kDq && waits && wave == 1) finish_dg();
        waits = false;
        const LaDecay& d = sm.d[dbuf];
        const bool odd = any_odd(sm.odd);
        const float thi = d.hi[t], tlo = d.lo[t];
        // An infinity or a NaN in the tile (odd): pair by pair, each lane its token, so that it
        // meets no weight of 0 of a pair that does not exist.  The products of token `late` as
        // a query with `early` as a key, the second with the pair's weight.
        const auto qk_of = [&](int late, int early) {
            float x = 0.f;
#pragma unroll 2
            for (int e = 0; e < N; ++e)
                x = fmaf(Elem<T>::load1(sm.q + late * SK::kStride + e), Elem<T>::load1(sm.k + early * SK::kStride + e), x);
            return x;
        };
        const auto yv_of = [&](int late, int early) {
            float x = 0.f;
#pragma unroll 2
            for (int e = 0; e < PB; ++e)
                x = fmaf(Elem<T>::load1(sm.dy + late * SV::kStride + e), Elem<T>::load1(sm.v + early * SV::kStride + e), x);
            return x;
        };
        const auto weight = [&](int late, int early) {
            return exp2_raw((d.hi[late] - d.hi[early]) + (d.lo[late] - d.lo[early])) * p.scale;
        };
        // A product with weights in terms.
        const auto weighted = [&](const Frag& rows, const Frag (&wt)[M::kTerms], f32x4& to) __attribute__((always_inline)) {
#pragma unroll
            for (int e = M::kTerms - 1; e >= 0; --e) to = M::mma(rows, wt[e], to);
        };
        // A row times x, where there is such a pair: chosen, not branched around, so that all
        // lanes stay together beside the matrix instructions.
        const auto add = [&](bool pair, const T* from, float x, auto& to) __attribute__((always_inline)) {
#pragma unroll
            for (int n = 0; n < (int)(sizeof(to) / sizeof(f32x4)); ++n) {
                const f32x4 y = M::wide(M::four(from + 16 * n + 4 * g)) * x;
#pragma unroll
                for (int r = 0; r < 4; ++r) to[n][r] += pair ? y[r] : 0.f;
            }
        };
        if constexpr (kRole == kDq) {
            // ---- the state's part
            const float up = d.up[t] * p.scale;
            Frag yf[PS];   // dy_t, along the states' columns (the contraction's second order)
#pragma unroll
            for (int j = 0; j < PS; ++j) {
                const T* const y1 = sm.dy + t * SV::kStride + 32 * j + 4 * g;
                yf[j] = M::cat(M::four(y1), M::four(y1 + 16));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                f32x4 x = zero4();
#pragma unroll
                for (int j = 0; j < PS; ++j)
                    x = M::mma(columns<T>(sm.s + 32 * j * SK::kStride + 16 * n, SK::kStride, g, l16), yf[j], x);
                x *= up;
                const f32x4 qn = M::wide(M::four(sm.q + t * SK::kStride + 16 * n + 4 * g));
#pragma unroll
                for (int r = 0; r < 4; ++r) asum = fmaf(qn[r], x[r], asum);
                sum[n] += x;
            }
            if (!odd) {
                // ---- and the tile's: [s][t], s up to t; and M
                Frag wt[2][M::kTerms], qf[KS];
#pragma unroll
                for (int j = 0; j < PS; ++j) yf[j] = M::rows(sm.dy + t * SV::kStride + 32 * j + 8 * g);
#pragma unroll
                for (int j = 0; j < KS; ++j) qf[j] = M::rows(sm.q + t * SK::kStride + 32 * j + 8 * g);
#pragma unroll
                for (int j2 = 0; j2 < 2; ++j2) {
                    Half h2[2][M::kTerms];
#pragma unroll
                    for (int u2 = 0; u2 < 2; ++u2) {
                        const int j = 2 * j2 + u2;
                        f32x4 x = zero4();
                        if (j <= w) {
#pragma unroll
                            for (int e = 0; e < PS; ++e)
                                x = M::mma(M::rows(sm.v + (16 * j + l16) * SV::kStride + 32 * e + 8 * g), yf[e], x);
                            x *= decays(d, j, g, thi, tlo, false) * p.scale;
                            if (j == w)   // the triangle's edge
#pragma unroll
                                for (int r = 0; r < 4; ++r) x[r] = 4 * g + r <= l16 ? x[r] : 0.f;
                            if (o.dg) {
                                f32x4 m = zero4();
#pragma unroll
                                for (int e = 0; e < KS; ++e)
                                    m = M::mma(M::rows(sm.k + (16 * j + l16) * SK::kStride + 32 * e + 8 * g), qf[e], m);
                                m *= x;
                                if (j == w)   // (a token with itself is on no side of a decay)
#pragma unroll
                                    for (int r = 0; r < 4; ++r) m[r] = 4 * g + r < l16 ? m[r] : 0.f;
                                asum += (m[0] + m[1]) + (m[2] + m[3]);
#pragma unroll
                                for (int r = 0; r < 4; ++r) m[r] = row16_sum(m[r]);
                                f32x4* const to = reinterpret_cast<f32x4*>(sm.g[gbuf].col[w] + 16 * j + 4 * g);
                                *to = head_first ? m : *to + m;   // (16 lanes alike: no branch)
                            }
                        }
                        split_terms<T>(x, h2[u2]);
                    }
#pragma unroll
                    for (int e = 0; e < M::kTerms; ++e) wt[j2][e] = M::cat(h2[0][e], h2[1][e]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    weighted(columns<T>(sm.k + 16 * n, SK::kStride, g, l16), wt[0], sum[n]);
                    if (w >= 2) weighted(columns<T>(sm.k + 32 * SK::kStride + 16 * n, SK::kStride, g, l16), wt[1], sum[n]);
                }
            } else {
                for (int s = 0; s < kLaChunk; ++s) {
                    const bool pair = in && s <= t && s < n_in;
                    const float yv = yv_of(t, s) * weight(t, s);
                    add(pair, sm.k + s * SK::kStride, yv, sum);
                    float m = qk_of(t, s) * yv;
                    m = pair && s < t ? m : 0.f;
                    asum += g == 0 ? m : 0.f;
                    m = row16_sum(m);
                    float* const to = sm.g[gbuf].col[w] + s;
                    *to = head_first ? m : *to + m;   // (64 lanes alike)
                }
            }
        } else if constexpr (kRole == kDk) {
            const float down = d.down[t];
            Frag vf[PS];
#pragma unroll
            for (int j = 0; j < PS; ++j) {
                const T* const v1 = sm.v + t * SV::kStride + 32 * j + 4 * g;
                vf[j] = M::cat(M::four(v1), M::four(v1 + 16));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                f32x4 x = zero4();
#pragma unroll
                for (int e = M::kTerms - 1; e >= 0; --e)
#pragma unroll
                    for (int j = 0; j < PS; ++j)
                        x = M::mma(columns<T>(sm.ds[e] + 32 * j * SK::kStride + 16 * n, SK::kStride, g, l16), vf[j], x);
                x *= down;
                const f32x4 kn = M::wide(M::four(sm.k + t * SK::kStride + 16 * n + 4 * g));
#pragma unroll
                for (int r = 0; r < 4; ++r) asum = fmaf(kn[r], x[r], asum);   // b
                sum[n] += x;
            }
            if (!odd) {
                // ---- and the tile's: [t][s], t from s on
                Frag wt[2][M::kTerms];
#pragma unroll
                for (int j = 0; j < PS; ++j) vf[j] = M::rows(sm.v + t * SV::kStride + 32 * j + 8 * g);
#pragma unroll
                for (int j2 = 0; j2 < 2; ++j2) {
                    Half h2[2][M::kTerms];
#pragma unroll
                    for (int u2 = 0; u2 < 2; ++u2) {
                        const int j = 2 * j2 + u2;
                        f32x4 x = zero4();
                        if (j >= w) {
#pragma unroll
                            for (int e = 0; e < PS; ++e)
                                x = M::mma(M::rows(sm.dy + (16 * j + l16) * SV::kStride + 32 * e + 8 * g), vf[e], x);
                            x *= decays(d, j, g, thi, tlo, true) * p.scale;
                            if (j == w)
#pragma unroll
                                for (int r = 0; r < 4; ++r) x[r] = 4 * g + r >= l16 ? x[r] : 0.f;
                        }
                        split_terms<T>(x, h2[u2]);
                    }
#pragma unroll
                    for (int e = 0; e < M::kTerms; ++e) wt[j2][e] = M::cat(h2[0][e], h2[1][e]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (w < 2) weighted(columns<T>(sm.q + 16 * n, SK::kStride, g, l16), wt[0], sum[n]);
                    weighted(columns<T>(sm.q + 32 * SK::kStride + 16 * n, SK::kStride, g, l16), wt[1], sum[n]);
                }
            } else {
                for (int s = 0; s < n_in; ++s)   // the query's token
                    add(in && s >= t, sm.q + s * SK::kStride, yv_of(s, t) * weight(s, t), sum);
            }
        } else {
            const float down = d.down[t];
            f32x4 dv[PT];
            Frag kf[KS];
#pragma unroll
            for (int j = 0; j < KS; ++j) kf[j] = M::rows(sm.k + t * SK::kStride + 32 * j + 8 * g);
#pragma unroll
            for (int m = 0; m < PT; ++m) {
                dv[m] = zero4();
#pragma unroll
                for (int e = M::kTerms - 1; e >= 0; --e)
#pragma unroll
                    for (int j = 0; j < KS; ++j)
                        dv[m] = M::mma(M::rows(sm.ds[e] + (16 * m + l16) * SK::kStride + 32 * j + 8 * g), kf[j], dv[m]);
                dv[m] *= down;
            }
            if (!odd) {
                Frag wt[2][M::kTerms];
#pragma unroll
                for (int j2 = 0; j2 < 2; ++j2) {
                    Half h2[2][M::kTerms];
#pragma unroll
                    for (int u2 = 0; u2 < 2; ++u2) {
                        const int j = 2 * j2 + u2;
                        f32x4 x = zero4();
                        if (j >= w) {
#pragma unroll
                            for (int e = 0; e < KS; ++e)
                                x = M::mma(M::rows(sm.q + (16 * j + l16) * SK::kStride + 32 * e + 8 * g), kf[e], x);
                            x *= decays(d, j, g, thi, tlo, true) * p.scale;
                            if (j == w)
#pragma unroll
                                for (int r = 0; r < 4; ++r) x[r] = 4 * g + r >= l16 ? x[r] : 0.f;
                        }
                        split_terms<T>(x, h2[u2]);
                    }
#pragma unroll
                    for (int e = 0; e < M::kTerms; ++e) wt[j2][e] = M::cat(h2[0][e], h2[1][e]);
                }
#pragma unroll
                for (int m = 0; m < PT; ++m) {
                    if (w < 2) weighted(columns<T>(sm.dy + 16 * m, SV::kStride, g, l16), wt[0], dv[m]);
                    weighted(columns<T>(sm.dy + 32 * SV::kStride + 16 * m, SV::kStride, g, l16), wt[1], dv[m]);
                }
            } else {
                for (int s = 0; s < n_in; ++s)
                    add(in && s >= t, sm.dy + s * SV::kStride, qk_of(s, t) * weight(s, t), dv);
            }
#pragma unroll
            for (int m = 0; m < PT; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) dv[m][r] = in ? dv[m][r] : 0.f;
            store_rows(dv, static_cast<T*>(args()->dv) + u.vat, n_out, vrow);
        }
        if (o.dg && head_last) {
            auto& sg = sm.g[gbuf];
            const float a = sum_rows4(in ? asum : 0.f);
            if constexpr (kRole == kDq) {
                if (g == 0) sg.a[t] = a;
                if (wave == 0 && lane < 8) sg.c[lane] = csum;
            } else if (kRole == kDk && g == 0) {
                sg.b[t] = a;
            }
            behind_at = u.at;
            behind_h = (int)u.h;
            behind_in = n_in;
            behind_out = n_out;
            behind_buf = gbuf;
            behind_all = d.all;
            waits = true;
            gbuf ^= 1;
        }
        // ---- dq or dk, or this part's sums of them, behind the last step (before: no rows)
        if constexpr (kRole != kDv) {
            const int n = u.step + 1 == u.steps ? n_out : 0;
            f32x4 x[NT];
#pragma unroll
            for (int e = 0; e < NT; ++e)
#pragma unroll
                for (int r = 0; r < 4; ++r) x[e][r] = in ? sum[e][r] : 0.f;
            if (o.split > 1) {
                const int64_t skipped = (p.packed ? p.tokens : (int64_t)p.B * p.T) * krow * u.part;
                const auto to = rows_of((kRole == kDq ? args()->part_q : args()->part_k) + skipped + u.kat, n, krow, N);
#pragma unroll
                for (int e = 0; e < NT; ++e)
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(vu4, x[e]), to,
                                                           t * (uint32_t)krow * 4 + (16 * e + 4 * g) * 4, 0, 0);
            } else {
                store_rows(x, static_cast<T*>(kRole == kDq ? args()->dq : args()->dk) + u.kat, n, krow);
            }
        }
        // The next head's decays, where the other waves still compute.
        if (next.valid && first_of_head(next)) {
            dbuf ^= 1;
            if (kRole == kDq && wave == 0) put_decays(sm.d[dbuf], lg.get());
        }
        u = next;
        next = after(u);
    }
    if (waits) {
        __syncthreads();
        if (kRole == kDq && wave == 1) finish_dg();
    }
    };
    if (wave < 4) run(Role<kDq>());
    else if (wave < 8) run(Role<kDk>());
    else run(Role<kDv>());
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
    const unsigned units = (unsigned)p.B * blocks * p.G * q.split;
    const unsigned most = 256;   // one workgroup to a compute unit
    la_bwd_kernel<T, N, PB><<<units < most ? units : most, kBwdThreads, 0, stream>>>(q, blocks);
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
