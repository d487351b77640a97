// wkv7_slots.hip -- copies between the slots of a cache of states, and its compaction.
//
// Bytes only: a cache is [planes][slots][row].  Bound by HBM: each moved row is read and
// written once, 16 bytes a lane and access, four of them under way.  Rows of another size
// than whole 16 bytes begin anywhere: their accesses are not aligned, and their last bytes go
// one by one (7 planes of 50 moves of 60 002 bytes: 9 us, by pairs of bytes 17).
// 12 planes of 48 copies of 192 KiB: 47 us, 4.8 TB/s (a copy of 1 GiB reaches 5.1).

#include "wkv7_device.h"
#include "wkv7_slots_internal.h"

namespace wkv7 {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;                  // pieces that a lane has on their way
constexpr int kPart = kThreads * kAhead;   // pieces of a row that a workgroup takes
constexpr int kPairs = 1024;               // pairs of a list that have workgroups of their own
constexpr int kSeen = 1 << 18;             // slots of the map of targets at a time: a bit each

typedef uint32_t Piece __attribute__((ext_vector_type(4)));
typedef Piece LoosePiece __attribute__((aligned(1)));

// Whether pair i counts: a target that exists, and a source that does or -1 (zeros).
__device__ __forceinline__ bool pair_ok(const SlotsArgs& p, int src, int dst) {
    return dst >= 0 && dst < p.slots && src >= -1 && src < p.from_slots;
}

// Words of the table of targets.
__host__ __device__ inline int seen_words(int slots) { return ((slots < kSeen ? slots : kSeen) + 31) / 32; }

// Pieces [c0, c0 + kPart) of row `src` of one plane to row `dst`; with the last of them the
// row's bytes behind whole pieces.  A lane always has the same bytes of a row.
template <bool kWhole>
__device__ __forceinline__ void move_part(const SlotsArgs& p, int plane, int src, int dst, int64_t c0) {
    const char* const from = static_cast<const char*>(p.from) + ((int64_t)plane * p.from_slots + (src < 0 ? 0 : src)) * p.bytes;
    char* const to = static_cast<char*>(p.pool) + ((int64_t)plane * p.slots + dst) * p.bytes;
    const int64_t pieces = p.bytes / 16;
    Piece x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int64_t c = c0 + i * kThreads + threadIdx.x;
        x[i] = Piece{0, 0, 0, 0};
        if (src >= 0 && c < pieces) {
            if constexpr (kWhole) x[i] = reinterpret_cast<const Piece*>(from)[c];
            else x[i] = *reinterpret_cast<const LoosePiece*>(from + c * 16);
        }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int64_t c = c0 + i * kThreads + threadIdx.x;
        if (c < pieces) {
            if constexpr (kWhole) reinterpret_cast<Piece*>(to)[c] = x[i];
            else *reinterpret_cast<LoosePiece*>(to + c * 16) = x[i];
        }
    }
    if constexpr (!kWhole) {
        const int64_t at = pieces * 16 + threadIdx.x;
        if (c0 <= pieces && pieces < c0 + kPart && at < p.bytes) to[at] = src < 0 ? 0 : from[at];
    }
}

// Pair by pair, in order, as the contract says: a lane has its bytes of every row to
// itself, so what it wrote for one pair is there for the next.  That is one row after the
// other; where no target is named twice and none is a source, the pairs do not touch and
// each has a workgroup of its own.  Every workgroup looks that up, the same way: it marks
// the targets in a table of bits, of as many slots as there are (of more than kSeen, 32 KiB
// of LDS, kSeen at a time, the lists read again for each).  Of longer lists a workgroup takes
// several pairs, so that the lists are not read more often than they are long: 65536 pairs of
// rows of 4 KiB in a cache of 140000 slots 0.34 ms (with a workgroup for each pair 6.2), of 64
// bytes in one of 2^22, sixteen tables, 2.5 ms (141).  With one table of 8192 bits for all
// slots, where two far ones can share a bit, 1024 pairs of 4 KiB among 20000 slots went one
// after the other, 687 us where these take 8.
template <bool kWhole>
__global__ __launch_bounds__(kThreads) void slots_copy_kernel(const SlotsArgs p, unsigned parts) {
    extern __shared__ uint32_t s_seen[];
    __shared__ int s_met;
    const unsigned part = blockIdx.x % parts, rest = blockIdx.x / parts;
    const int plane = (int)(rest % p.planes), pair = (int)(rest / p.planes);
    const int64_t c0 = (int64_t)part * kPart;
    if (p.n > 1) {
        if (threadIdx.x == 0) s_met = 0;
        const int words = seen_words(p.slots);
        for (int first = 0; first < p.slots; first += kSeen) {
            for (int i = threadIdx.x; i < words; i += kThreads) s_seen[i] = 0;
            __syncthreads();
            const auto here = [&](int slot) { return slot >= first && slot - first < kSeen; };
            bool met = false;
            for (int i = threadIdx.x; i < p.n; i += kThreads) {
                const int s = p.src[i], d = p.dst[i];
                if (pair_ok(p, s, d) && here(d)) {
                    const uint32_t bit = 1u << (d % 32);
                    met |= (atomicOr(&s_seen[(d - first) / 32], bit) & bit) != 0;
                }
            }
            __syncthreads();
            if (p.from == p.pool)
                for (int i = threadIdx.x; i < p.n; i += kThreads) {
                    const int s = p.src[i], d = p.dst[i];
                    if (pair_ok(p, s, d) && s != d && here(s)) met |= (s_seen[(s - first) / 32] >> (s % 32) & 1) != 0;
                }
            if (met) s_met = 1;
            __syncthreads();
            if (s_met) break;
        }
        if (s_met) {
            if (pair != 0) return;
            for (int i = 0; i < p.n; ++i) {
                const int s = p.src[i], d = p.dst[i];
                if (pair_ok(p, s, d) && (s != d || p.from != p.pool)) move_part<kWhole>(p, plane, s, d, c0);
            }
            return;
        }
    }
    for (int64_t i = pair; i < p.n; i += gridDim.x / parts / p.planes) {
        const int s = p.src[i], d = p.dst[i];
        if (pair_ok(p, s, d) && (s != d || p.from != p.pool)) move_part<kWhole>(p, plane, s, d, c0);
    }
}

// Which slots move: with `count` kept ones, those behind the first `count` places fill the
// free ones among these, both in order, so that no slot is moved twice and none that is
// read is written.  One workgroup; a thread takes a run of slots.
constexpr int kScan = 1024;
__device__ __forceinline__ int block_before(int x, int* lds, int& total) {
    lds[threadIdx.x] = x;
    __syncthreads();
    for (int d = 1; d < kScan; d *= 2) {
        const int y = threadIdx.x >= (unsigned)d ? lds[threadIdx.x - d] : 0;
        __syncthreads();
        lds[threadIdx.x] += y;
        __syncthreads();
    }
    total = lds[kScan - 1];
    const int r = lds[threadIdx.x] - x;
    __syncthreads();
    return r;
}
__global__ __launch_bounds__(kScan) void slots_plan_kernel(const SlotsArgs p) {
    __shared__ int s_run[kScan];
    const int run = (p.slots + kScan - 1) / kScan;
    const int64_t a64 = (int64_t)threadIdx.x * run;
    const int a = (int)(a64 < p.slots ? a64 : p.slots), e = a + run < p.slots ? a + run : p.slots;
    int kept = 0, count, holes = 0, late = 0, all;
    for (int i = a; i < e; ++i) kept += p.keep[i] != 0;
    block_before(kept, s_run, count);
    for (int i = a; i < e; ++i) {
        const bool k = p.keep[i] != 0;
        holes += !k && i < count;
        late += k && i >= count;
    }
    int h = block_before(holes, s_run, all), l = block_before(late, s_run, all);
    for (int i = a; i < e; ++i) {
        const bool k = p.keep[i] != 0;
        if (!k && i < count) p.pairs[p.slots + h++] = i;
        if (k && i >= count) p.pairs[l++] = i;
        if (!k) p.moved[i] = -1;
        else if (i < count) p.moved[i] = i;
    }
    if (threadIdx.x == 0) {
        p.pairs[2 * (size_t)p.slots] = all;
        p.count[0] = count;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < all; i += kScan) p.moved[p.pairs[i]] = p.pairs[p.slots + i];
}

// The moves, and zeros behind the last kept slot if wanted.  A slot that is moved is read
// here and cleared only by its own workgroup's part, behind its copy.
template <bool kWhole>
__global__ __launch_bounds__(kThreads) void slots_move_kernel(const SlotsArgs p, unsigned parts) {
    const unsigned part = blockIdx.x % parts, rest = blockIdx.x / parts;
    const int plane = (int)(rest % p.planes), i = (int)(rest / p.planes);
    const int64_t c0 = (int64_t)part * kPart;
    if (!p.clear) {
        // workgroup i: move i (at most half of the slots move)
        if (i < p.pairs[2 * (size_t)p.slots]) move_part<kWhole>(p, plane, p.pairs[i], p.pairs[p.slots + i], c0);
        return;
    }
    // workgroup i: slot i
    if (i < p.count[0]) return;
    const int n = p.pairs[2 * (size_t)p.slots];
    if (p.keep[i] != 0) {
        int lo = 0, hi = n - 1;   // its place among the moved ones, which are in order
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (p.pairs[mid] < i) lo = mid + 1;
            else hi = mid;
        }
        move_part<kWhole>(p, plane, i, p.pairs[p.slots + lo], c0);
    }
    move_part<kWhole>(p, plane, -1, i, c0);
}

}  // namespace

#define WKV7_SLOTS(kernel, rows, lds)                                                         \
    {                                                                                         \
        const unsigned parts = (unsigned)(((p.bytes + 15) / 16 + kPart - 1) / kPart);         \
        const unsigned grid = parts * p.planes * (unsigned)(rows);                            \
        if (p.bytes % 16 == 0) kernel<true><<<grid, kThreads, lds, stream>>>(p, parts);       \
        else kernel<false><<<grid, kThreads, lds, stream>>>(p, parts);                        \
        return hipGetLastError();                                                             \
    }

hipError_t launch_slots_copy(const SlotsArgs& p, hipStream_t stream) {
    WKV7_SLOTS(slots_copy_kernel, p.n < kPairs ? p.n : kPairs, p.n > 1 ? seen_words(p.slots) * sizeof(uint32_t) : 0)
}

hipError_t launch_slots_compact(const SlotsArgs& p, hipStream_t stream) {
    slots_plan_kernel<<<1, kScan, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.planes == 0 || p.bytes == 0) return e;
    const int rows = p.clear ? p.slots : (p.slots + 1) / 2;
    WKV7_SLOTS(slots_move_kernel, rows, 0)
}

}  // namespace wkv7
