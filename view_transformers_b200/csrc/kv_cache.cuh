// Shared definitions of the paged key/value cache kernels: arguments, sequence tables, what a
// token sees, and how the attention's work is split over blocks.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace bsa {
namespace kv {

constexpr int kUnit = 128;   // keys per work unit

struct CacheArgs {
    int seqs, heads, kv_heads, pshift, pages, max_pages;
    const int32_t* table;
    const int32_t* kv_len;
};

struct AttnArgs {
    CacheArgs c;
    int group;                 // query heads per key/value head
    int rows;                  // packed rows of q and out
    int unit, window, sink;
    const int32_t* cu;
    const void* k;
    const void* v;
    const uint8_t* ks;
    const uint8_t* vs;
    const __nv_bfloat16* q;
    long long q_stride;
    __nv_bfloat16* out;
    long long out_stride;
    float* lse;
    float* part;               // partial results: [teams][2][R][M] rows of 64 + 1 floats
    int* desc;                 // [teams] records of kDesc ints: the item a team leaves unfinished
    int max_teams, R;          // R blocks of a team walk the same keys, each for its own query tile
    int mr;                    // rows of a query tile (at most the M of its kernel)
    int min_run;               // fewest units worth a team of its own
    int32_t* status;
};
constexpr int kDesc = 8;       // valid, first row, tokens, kv head, row group, last team

struct Seq {
    int row0, n, len;          // first packed row, new tokens, cached tokens
};

// Table values are clamped to what the buffers hold; `report` records a bad one.
__device__ __forceinline__ Seq load_seq(const CacheArgs& c, const int32_t* cu, int rows, int s, int32_t* status,
                                        bool report) {
    const int c0 = cu[s], c1 = cu[s + 1], len = c.kv_len[s];
    const int cap = c.max_pages << c.pshift;
    Seq q;
    q.row0 = min(max(c0, 0), rows);
    q.n = min(max(c1, q.row0), rows) - q.row0;
    q.len = min(max(len, 0), cap);
    if (report && (c0 < 0 || c1 < c0 || c1 > rows || len < 0 || len > cap || q.n > q.len))
        record_error(status, BSA_ERR_DEVICE_BOUNDS);
    return q;
}

// Positions [lo, hi) and, with a window, [0, min(sink, lo)) are what the token at position p
// sees. lo and hi do not fall as p grows.
__device__ __forceinline__ void visible(const AttnArgs& a, int len, int p, int& lo, int& hi) {
    lo = 0;
    hi = len;
    if (a.unit == 0) return;
    if (p < 0) {
        hi = 0;
        return;
    }
    const long long f = p / a.unit;
    hi = (int)min((long long)len, (f + 1) * a.unit);
    if (a.window > 0) lo = (int)min((long long)hi, max(0ll, (f - a.window + 1) * a.unit));
}

// The key units that the tokens [i0, i1] of a sequence's chunk need, in order: units
// [0, n_sink), then [t_lo, t_lo + count - n_sink).
struct Span {
    int n_sink, t_lo, count;
    int lo_min, hi_max;        // positions that some token may see (besides the sink)
    int lo_max, hi_min;        // [lo_max, hi_min) is seen by every token
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, const Seq& q, int i0, int i1) {
    Span s;
    visible(a, q.len, q.len - q.n + i0, s.lo_min, s.hi_min);
    visible(a, q.len, q.len - q.n + i1, s.lo_max, s.hi_max);
    s.t_lo = s.lo_min / kUnit;
    const int sink = min(a.sink, s.lo_min);
    s.n_sink = min((sink + kUnit - 1) / kUnit, s.t_lo);
    s.count = s.n_sink + max(0, (s.hi_max + kUnit - 1) / kUnit - s.t_lo);
    return s;
}
__device__ __forceinline__ int unit_of(const Span& s, int j) { return j < s.n_sink ? j : s.t_lo + (j - s.n_sink); }

// Work is counted in units of 128 keys. An item is one row group (R query tiles of mr rows; a
// row is one query head of one token, the heads of a group next to each other) of one key/value
// head, with at least one unit, so that rows that see nothing are written too. The units of all
// items in the order sequence, head, row group are dealt out to the teams in equal runs: a team
// finishes the items that lie inside its run and leaves partial results of the (at most two)
// that cross its ends, which the merge kernel joins in a fixed order.
__device__ __forceinline__ int group_count(const AttnArgs& a, const Seq& q) {
    const int tiles = (q.n * a.group + a.mr - 1) / a.mr;
    return (tiles + a.R - 1) / a.R;
}
// rows [r0, r1) of a sequence's chunk
__device__ __forceinline__ Span rows_span(const AttnArgs& a, const Seq& q, int r0, int r1) {
    return span_of(a, q, r0 / a.group, (min(r1, q.n * a.group) - 1) / a.group);
}
__device__ __forceinline__ Span group_span(const AttnArgs& a, const Seq& q, int rg) {
    const int r0 = rg * a.R * a.mr;
    return rows_span(a, q, r0, r0 + a.R * a.mr);
}

struct Start {
    int s, h, rg;
    int teams;         // teams that have work
    long long item;    // first unit of the item
    long long total;   // units of all items
};

__device__ __forceinline__ long long shfl_up64(long long v, int d) { return __shfl_up_sync(0xffffffffu, v, d); }

// Fills pre[s] = units of sequences 0 .. s - 1 (pre[seqs] = total) and finds the item of the first
// unit of a team. Whole block; `list` holds seqs + 1 ints. All in shared memory.
__device__ __forceinline__ void plan(const AttnArgs& a, int team, long long* pre, int* list, Start* st) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    const int S = a.c.seqs;
    if (tid == 0) list[S] = 0;
    __syncthreads();
    for (int s = tid; s < S; s += nt) {
        const Seq q = load_seq(a.c, a.cu, a.rows, s, a.status, blockIdx.x == 0);
        const int ng = group_count(a, q);
        long long u = 0;
        if (a.unit == 0) {
            u = ng > 0 ? (long long)ng * max(1, group_span(a, q, 0).count) : 0;
        } else if (ng <= 8) {
            for (int g = 0; g < ng; ++g) u += max(1, group_span(a, q, g).count);
        } else {
            list[atomicAdd(&list[S], 1)] = s;   // long chunks: one warp each, below
        }
        pre[s] = u * a.c.kv_heads;
    }
    __syncthreads();
    for (int x = warp; x < list[S]; x += nw) {
        const int s = list[x];
        const Seq q = load_seq(a.c, a.cu, a.rows, s, nullptr, false);
        const int ng = group_count(a, q);
        long long u = 0;
        for (int g = lane; g < ng; g += 32) u += max(1, group_span(a, q, g).count);
        for (int d = 16; d > 0; d >>= 1) u += __shfl_xor_sync(0xffffffffu, u, d);
        if (lane == 0) pre[s] = u * a.c.kv_heads;
    }
    __syncthreads();
    if (warp == 0) {
        long long base = 0;
        for (int s0 = 0; s0 < S; s0 += 32) {
            const long long own = s0 + lane < S ? pre[s0 + lane] : 0;
            long long v = own;
            for (int d = 1; d < 32; d <<= 1) {
                const long long o = shfl_up64(v, d);
                if (lane >= d) v += o;
            }
            if (s0 + lane < S) pre[s0 + lane] = base + v - own;
            base += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) pre[S] = base;
        __syncwarp();
        Start r;
        r.teams = (int)max(1ll, min((long long)a.max_teams, base / a.min_run));
        const long long u0 = team < r.teams ? base * team / r.teams : base;
        int lo = 0, hi = S;                     // last sequence with pre[s] <= u0 that has units
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= u0) lo = mid; else hi = mid;
        }
        r.s = lo;
        r.total = base;
        r.h = r.rg = 0;
        r.item = pre[lo];
        if (u0 < base) {
            const Seq q = load_seq(a.c, a.cu, a.rows, lo, nullptr, false);
            const long long per_head = (pre[lo + 1] - pre[lo]) / a.c.kv_heads;
            const long long off = u0 - pre[lo];
            r.h = (int)(off / per_head);
            r.item += (long long)r.h * per_head;
            long long rest = off - (long long)r.h * per_head;
            const int ng = group_count(a, q);
            for (int g0 = 0; g0 < ng; g0 += 32) {
                const long long own = g0 + lane < ng ? max(1, group_span(a, q, g0 + lane).count) : 0;
                long long v = own;
                for (int d = 1; d < 32; d <<= 1) {
                    const long long o = shfl_up64(v, d);
                    if (lane >= d) v += o;
                }
                const unsigned in = __ballot_sync(0xffffffffu, g0 + lane < ng && rest < v);
                if (in) {
                    const int at = __ffs(in) - 1;
                    r.rg = g0 + at;
                    r.item += __shfl_sync(0xffffffffu, v - own, at);
                    break;
                }
                const long long all = __shfl_sync(0xffffffffu, v, 31);
                rest -= all;
                r.item += all;
            }
        }
        if (lane == 0) *st = r;
    }
    __syncthreads();
}

// Walks the segments (item, run of its units) of one team. Every role of a block runs its own
// copy over the same tables.
struct Walk {
    const AttnArgs& a;
    long long u, u1, item;     // next unit, end of the team's run, first unit of the item
    int s, h, rg, ng;
    Seq q;
    Span span;                 // of the whole row group
    int j0, j1;                // this segment's units within the item
    bool has_start, has_end;   // the segment holds the item's first, last unit
    int teams;
    __device__ __forceinline__ Walk(const AttnArgs& args, const Start& st, int team) : a(args) {
        teams = st.teams;
        u = team < teams ? st.total * team / teams : st.total;
        u1 = team < teams ? st.total * (team + 1) / teams : st.total;
        item = st.item;
        s = st.s;
        h = st.h;
        rg = st.rg;
        q.row0 = q.n = q.len = 0;
        ng = 0;
        if (u < u1) enter();
    }
    __device__ __forceinline__ void enter() {
        q = load_seq(a.c, a.cu, a.rows, s, nullptr, false);
        ng = group_count(a, q);
    }
    // the next segment; false when the run is done
    __device__ __forceinline__ bool next() {
        if (u >= u1) return false;
        while (rg >= ng) {     // past the last row group of a head, or an empty sequence
            rg = 0;
            if (ng == 0 || ++h >= a.c.kv_heads) {
                h = 0;
                if (++s >= a.c.seqs) return false;
                enter();
            }
        }
        span = group_span(a, q, rg);
        const int cnt = max(1, span.count);
        j0 = (int)(u - item);
        j1 = (int)(min(item + cnt, u1) - item);
        has_start = j0 == 0;
        has_end = j1 == cnt;
        return j1 > j0;        // false only if the tables changed under the call
    }
    // to the end of the segment; its fields stay
    __device__ __forceinline__ void done() {
        u = item + j1;
        if (has_end) {
            item = u;
            ++rg;
        }
    }
    // last team that holds units of the item that ends at unit `end`
    __device__ __forceinline__ int last_team(long long end, long long total) const {
        int t = (int)((end * teams + total - 1) / total) - 1;
        while (t + 1 < teams && total * (t + 1) / teams < end) ++t;
        while (t > 0 && total * t / teams >= end) --t;
        return t;
    }
};

// Where a block keeps the partial result of a segment: run 0 of a team for the item that
// began in an earlier team, run 1 for the item that it leaves unfinished.
template <int M>
__device__ __forceinline__ float* part_at(const AttnArgs& a, int team, int run, int member) {
    return a.part + ((long long)(team * 2 + run) * a.R + member) * (M * 65);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^(byte - 127), the scale that a scale byte stands for; 255 stands for NaN (a row that held
// infinite or NaN elements)
__device__ __forceinline__ float pow2_of(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7fc00000u) : pow2_of(byte);
}

}  // namespace kv
}  // namespace bsa
