// Shared definitions of the paged key/value cache kernels: arguments, sequence tables, what a
// token sees, and how the attention's work is split over blocks.
#pragma once

#include <atomic>
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

// Division of 0 <= n < 2^31 by a divisor that the host knows: with s = ceil(log2 d) and
// mul = ceil(2^(31 + s) / d), n mul / 2^(31 + s) is at most 2^-s <= 1 / d above n / d. The split of the
// work is all divisions, one after the other, and a block's first load waits for them.
struct Div {
    int d = 1;
    uint32_t mul = 0, shift = 0;
    Div() = default;
    explicit Div(int divisor) : d(divisor) {
        if (d <= 1) return;
        int s = 0;
        while ((1ll << s) < d) ++s;
        mul = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
        shift = s - 1;
    }
    __device__ __forceinline__ int of(int n) const { return mul == 0u ? n : (int)(__umulhi((uint32_t)n, mul) >> shift); }
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
    Div by_group, by_unit, by_mr, by_R, by_teams;
    int32_t* status;
    void set_divisors() {
        by_group = Div(group);
        by_unit = Div(unit);
        by_mr = Div(mr);
        by_R = Div(R);
        by_teams = Div(max_teams);
    }
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
    const long long f = a.by_unit.of(p);
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
__device__ __forceinline__ Span span_of(const AttnArgs& a, Seq q, int i0, int i1) {
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
    return a.by_R.of(a.by_mr.of(q.n * a.group + a.mr - 1) + a.R - 1);
}
// rows [r0, r1) of a sequence's chunk
__device__ __forceinline__ Span rows_span(const AttnArgs& a, const Seq& q, int r0, int r1) {
    return span_of(a, q, a.by_group.of(r0), a.by_group.of(min(r1, q.n * a.group) - 1));
}
__device__ __forceinline__ Span group_span(const AttnArgs& a, const Seq& q, int rg) {
    const int r0 = rg * a.R * a.mr;
    return rows_span(a, q, r0, r0 + a.R * a.mr);
}

struct Start {
    int s, h, rg;
    Seq q;                     // sequence s
    int teams;                 // teams that have work
    int item;                  // first unit of the item
    int total;                 // units of all items
    int run, wide;             // the first `wide` teams get run + 1 units, the others run
    __device__ __forceinline__ int first_unit(int team) const { return run * team + min(team, wide); }
    // the team that holds unit u
    __device__ __forceinline__ int team_of(int u) const {
        const int w = wide * (run + 1);
        return u < w ? u / (run + 1) : wide + (u - w) / run;
    }
    __device__ __forceinline__ void deal(const AttnArgs& a, int units) {
        total = units;
        teams = max(1, min(a.max_teams, units));
        run = units < a.max_teams ? min(units, 1) : a.by_teams.of(units);
        wide = units - run * teams;
    }
};

// inclusive sum over the lanes up to this one
__device__ __forceinline__ int lane_scan(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}
__device__ __forceinline__ int lane_sum(int v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

constexpr int kMostUnits = 1 << 30;
// Units of one head that are more than any call may have, and whose sum over a warp is an int.
constexpr int kTooMany = kMostUnits / 32 + 4096;

// Units of one key/value head of a sequence with few row groups (many: far set instead).
__device__ __forceinline__ int head_units(const AttnArgs& a, const Seq& q, bool& far) {
    const int ng = group_count(a, q);
    int u = 0;
    if (a.unit == 0) {
        u = ng > 0 ? (int)min((long long)ng * max(1, group_span(a, q, 0).count), (long long)kTooMany) : 0;
    } else if (ng <= 4) {
        for (int g = 0; g < ng; ++g) u += max(1, group_span(a, q, g).count);
    } else {
        far = true;
    }
    return u;
}
// the same of a sequence with many row groups, by a whole warp
__device__ __forceinline__ int head_units_warp(const AttnArgs& a, const Seq& q, int lane) {
    const int ng = group_count(a, q);
    int u = 0;
    for (int g = lane; g < ng && u < kTooMany; g += 32) u += max(1, group_span(a, q, g).count);
    u = min(u, kTooMany);
    return lane_sum(u);
}
// the item of unit u0, which lies in the sequence r.q that starts at unit `base` (whole warp)
__device__ __forceinline__ void find_item(const AttnArgs& a, int base, int per_head, int u0, int lane, Start& r) {
    r.h = (u0 - base) / per_head;
    r.item = base + r.h * per_head;
    r.rg = 0;
    const int ng = group_count(a, r.q);
    if (ng == 1) return;
    int rest = u0 - r.item;
    for (int g0 = 0; g0 < ng; g0 += 32) {
        const int own = g0 + lane < ng ? max(1, group_span(a, r.q, g0 + lane).count) : 0;
        const int v = lane_scan(own, lane);
        const unsigned in = __ballot_sync(0xffffffffu, g0 + lane < ng && rest < v);
        if (in) {
            const int at = __ffs(in) - 1;
            r.rg = g0 + at;
            r.item += __shfl_sync(0xffffffffu, v - own, at);
            return;
        }
        const int all = __shfl_sync(0xffffffffu, v, 31);
        rest -= all;
        r.item += all;
    }
}

static __device__ __noinline__ Start plan_many(const AttnArgs& a, int team, int* pre, int* list, Start* st);

// The split of the work, for this block's team. Up to 32 sequences: every warp by itself,
// without shared memory or a barrier. More: the whole block, through pre (seqs + 1 ints), list
// (seqs + 1 ints) and *st in shared memory. Refused: more than 2^25 units in one sequence, over all
// its key/value heads, so that sums over 32 of them stay inside 2^30; more than 2^30 in all.
__device__ __forceinline__ Start plan(const AttnArgs& a, int team, int* pre, int* list, Start* st) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int S = a.c.seqs;
    if (S > 32) return plan_many(a, team, pre, list, st);
    Start r;
    r.s = r.h = r.rg = r.item = 0;
    r.q.row0 = r.q.n = r.q.len = 0;
    {
        Seq q;
        q.row0 = q.n = q.len = 0;
        if (lane < S) q = load_seq(a.c, a.cu, a.rows, lane, a.status, blockIdx.x == 0 && warp == 0);
        bool far = false;
        int u = head_units(a, q, far);
        for (unsigned m = __ballot_sync(0xffffffffu, far); m; m &= m - 1) {
            const int s = __ffs(m) - 1;
            Seq o;
            o.row0 = __shfl_sync(0xffffffffu, q.row0, s);
            o.n = __shfl_sync(0xffffffffu, q.n, s);
            o.len = __shfl_sync(0xffffffffu, q.len, s);
            const int v = head_units_warp(a, o, lane);
            if (lane == s) u = v;
        }
        const float most = (float)u * (float)a.c.kv_heads;   // 32 such sums stay inside 2^31
        const bool over = __any_sync(0xffffffffu, most > (float)(kMostUnits / 32));
        const int head = u;
        u *= a.c.kv_heads;
        const int v = lane_scan(u, lane);
        const int total = __shfl_sync(0xffffffffu, v, 31);
        if (over && threadIdx.x == 0) record_error(a.status, BSA_ERR_UNSUPPORTED);
        r.deal(a, over ? 0 : total);
        const int u0 = team < r.teams ? r.first_unit(team) : r.total;
        const unsigned in = __ballot_sync(0xffffffffu, v > u0 && u > 0);
        if (in && u0 < r.total) {
            r.s = __ffs(in) - 1;
            r.q.row0 = __shfl_sync(0xffffffffu, q.row0, r.s);
            r.q.n = __shfl_sync(0xffffffffu, q.n, r.s);
            r.q.len = __shfl_sync(0xffffffffu, q.len, r.s);
            find_item(a, __shfl_sync(0xffffffffu, v - u, r.s), __shfl_sync(0xffffffffu, head, r.s), u0, lane, r);
        }
        return r;
    }
}

static __device__ __noinline__ Start plan_many(const AttnArgs& a, int team, int* pre, int* list, Start* st) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    const int S = a.c.seqs;
    if (tid == 0) list[S] = 0;
    __syncthreads();
    for (int s = tid; s < S; s += nt) {
        const Seq q = load_seq(a.c, a.cu, a.rows, s, a.status, blockIdx.x == 0);
        bool far = false;
        pre[s] = head_units(a, q, far);
        if (far) list[atomicAdd(&list[S], 1)] = s;
    }
    __syncthreads();
    for (int x = warp; x < list[S]; x += nw) {
        const int s = list[x];
        const int v = head_units_warp(a, load_seq(a.c, a.cu, a.rows, s, nullptr, false), lane);
        if (lane == 0) pre[s] = v;
    }
    __syncthreads();
    if (warp == 0) {
        Start r;
        r.s = r.h = r.rg = r.item = 0;
        r.q.row0 = r.q.n = r.q.len = 0;
        int base = 0;
        bool over = false;
        for (int s0 = 0; s0 < S; s0 += 32) {
            const int per = s0 + lane < S ? pre[s0 + lane] : 0;
            over |= (float)per * (float)a.c.kv_heads > (float)(kMostUnits / 32);
            const int own = per * a.c.kv_heads;
            const int v = lane_scan(own, lane);
            if (s0 + lane < S) pre[s0 + lane] = base + v - own;
            base += __shfl_sync(0xffffffffu, v, 31);   // at most 2^30 + 32 * 2^25
            over |= (uint32_t)base > (uint32_t)kMostUnits;
            if (__any_sync(0xffffffffu, over)) break;
        }
        if (__any_sync(0xffffffffu, over)) {
            if (lane == 0) record_error(a.status, BSA_ERR_UNSUPPORTED);
            base = 0;
        }
        if (lane == 0) pre[S] = base;
        __syncwarp();
        r.deal(a, base);
        const int u0 = team < r.teams ? r.first_unit(team) : base;
        if (u0 < base) {
            int lo = 0, hi = S;                     // the last sequence with pre[s] <= u0
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (pre[mid] <= u0) lo = mid; else hi = mid;
            }
            r.s = lo;
            r.q = load_seq(a.c, a.cu, a.rows, lo, nullptr, false);
            find_item(a, pre[lo], (pre[lo + 1] - pre[lo]) / a.c.kv_heads, u0, lane, r);
        }
        if (lane == 0) *st = r;
    }
    __syncthreads();
    return *st;
}

// Walks the segments (item, run of its units) of one team. Every role of a block runs its own
// copy over the same tables.
struct Walk {
    const AttnArgs& a;
    int u, u1, item;           // next unit, end of the team's run, first unit of the item
    int s, h, rg, ng;
    Seq q;
    Span span;                 // of the whole row group
    int j0, j1;                // this segment's units within the item
    bool has_start, has_end;   // the segment holds the item's first, last unit
    __device__ __forceinline__ Walk(const AttnArgs& args, const Start& st, int team) : a(args) {
        u = team < st.teams ? st.first_unit(team) : st.total;
        u1 = team < st.teams ? st.first_unit(team + 1) : st.total;
        item = st.item;
        s = st.s;
        h = st.h;
        rg = st.rg;
        q = st.q;
        ng = u < u1 ? group_count(a, q) : 0;
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
        j0 = u - item;
        j1 = min(item + cnt, u1) - item;
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
};

// What the arithmetic of a block has to know of a segment.
struct Rec {
    int tiles;             // key tiles to come (0: nothing to see); negative: no further segment
    int nrows, r0;         // rows of the query tile, first one within the chunk
    int row0, pos0, len;   // packed row and position of the chunk's first token, cached tokens
    int h, whole, run;     // key/value head; the segment is the whole item; run of the partial result
    int lo_min, hi_max;    // positions outside the sink that some row sees
    int lo_max, hi_min;    // [lo_max, hi_min) is seen by every row
};

// Words of a key tile: a bit per 16 keys whose page exists, and these.
enum { kFull = 0x100, kFirst = 0x200, kLast = 0x400, kEnd = 0x800 };

// The producer's part of a block, run by one warp: walks the team's segments, hands out a record
// for each (put_record), announces those with key tiles (begin) and then hands out their tiles:
// put_tile(meta, t, boxes, rows, at) gets tile t's words and, in lanes at .. at + boxes - 1 of
// `rows`, the first pool rows of its boxes (up to 128 keys of a page each; negative: no page). Any
// of the three returns false to stop. True when all is handed out. What can be computed for 32
// boxes at once is: the warp shares its scheduler with the arithmetic.
template <class PutRecord, class Begin, class PutTile>
__device__ __forceinline__ bool produce(const AttnArgs& a, const Start& start, int team, int member, int lane,
                                        PutRecord put_record, Begin begin, PutTile put_tile) {
    const int box = min(1 << a.c.pshift, kUnit), shift = min(a.c.pshift, 7);
    Walk w(a, start, team);
    for (; w.next(); w.done()) {
        const int r0 = (w.rg * a.R + member) * a.mr;
        const int nrows = min(a.mr, w.q.n * a.group - r0);
        if (nrows <= 0) continue;
        const Span own = a.R == 1 ? w.span : rows_span(a, w.q, r0, r0 + a.mr);
        auto wanted = [&](int k0, int n) { return k0 < own.hi_max && (k0 + n > own.lo_min || k0 < a.sink); };
        // how many of the run's tiles this query tile needs: of the tiles [0, sinks) and
        // [lo, hi) those that the run's two stretches (unit_of) hold
        const int hi = (own.hi_max + kUnit - 1) / kUnit, lo = own.lo_min / kUnit;
        const int sinks = min(min((int)(((long long)a.sink + kUnit - 1) / kUnit), lo), hi);
        auto held = [&](int p, int q) { return max(0, min(q, sinks) - p) + max(0, min(q, hi) - max(p, lo)); };
        const int skip = w.span.t_lo - w.span.n_sink;
        const int tiles = held(w.j0, min(w.j1, w.span.n_sink)) + held(max(w.j0, w.span.n_sink) + skip, w.j1 + skip);
        Rec rec;
        rec.tiles = tiles;
        rec.nrows = nrows;
        rec.r0 = r0;
        rec.row0 = w.q.row0;
        rec.pos0 = w.q.len - w.q.n;
        rec.len = w.q.len;
        rec.h = w.h;
        rec.whole = w.has_start && w.has_end;
        rec.run = w.has_start ? 1 : 0;
        rec.lo_min = own.lo_min;
        rec.hi_max = own.hi_max;
        rec.lo_max = own.lo_max;
        rec.hi_min = own.hi_min;
        // lane i: box i % boxes of the run's tile jb + i / boxes; the next batch's page ids are on
        // their way while this one's tiles are handed out
        const int bshift = 7 - shift, boxes = 1 << bshift, per = 32 >> bshift;
        const int sub = (lane & (boxes - 1)) * box;
        const int32_t* pages = a.c.table + (long long)w.s * a.c.max_pages;
        auto fetch = [&](int jb) {
            const int j = jb + (lane >> bshift), k0 = unit_of(w.span, j) * kUnit + sub;
            return j < w.j1 && wanted(k0, box) ? pages[k0 >> a.c.pshift] : -1;
        };
        int ahead = fetch(w.j0), left = tiles;
        if (!put_record(rec)) return false;
        if (tiles > 0 && !begin(w, r0)) return false;
        for (int jb = w.j0; left > 0 && jb < w.j1; jb += per) {
            int page = ahead;
            ahead = fetch(jb + per);
            const int j = jb + (lane >> bshift), mine = unit_of(w.span, j), key = mine * kUnit;
            if (page >= a.c.pages) {
                record_error(a.status, BSA_ERR_DEVICE_BOUNDS);
                page = -1;
            }
            const int rows = page < 0 ? -1
                : ((page * a.c.kv_heads + w.h) << a.c.pshift) + ((key + sub) & ((1 << a.c.pshift) - 1));
            const unsigned have = __ballot_sync(0xffffffffu, page >= 0);
            const unsigned want = __ballot_sync(0xffffffffu, j < w.j1 && wanted(key, kUnit));
            const unsigned whole = __ballot_sync(0xffffffffu, key + kUnit <= own.hi_min &&
                                                                  (key >= own.lo_max || key + kUnit <= min(a.sink, own.lo_min)));
            for (int at = 0; at < 32 && left > 0; at += boxes) {
                if (!((want >> at) & 1u)) continue;
                const unsigned got = (have >> at) & ((1u << boxes) - 1u);
                int meta = 0xff;
                if (got != (1u << boxes) - 1u) {
                    meta = 0;
                    for (int i = 0; i < 8; ++i) meta |= ((got >> ((i * 16) >> shift)) & 1u) << i;
                } else if ((whole >> at) & 1u) {
                    meta |= kFull;
                }
                meta |= (left == tiles ? kFirst : 0) | (left == 1 ? kLast : 0);
                --left;
                if (!put_tile(meta, __shfl_sync(0xffffffffu, mine, at), boxes, rows, at)) return false;
            }
        }
        if (lane == 0 && member == 0 && !rec.whole && w.has_start) {   // the merge kernel's record of this item
            int* d = a.desc + team * kDesc;
            d[1] = w.q.row0;
            d[2] = w.q.n;
            d[3] = w.h;
            d[4] = w.rg;
            d[5] = start.team_of(w.item + max(1, w.span.count) - 1);
            d[0] = 1;
        }
    }
    return true;
}

// Where a block keeps the partial result of a segment: run 0 of a team for the item that
// began in an earlier team, run 1 for the item that it leaves unfinished.
template <int M>
__device__ __forceinline__ float* part_at(const AttnArgs& a, int team, int run, int member) {
    return a.part + ((long long)(team * 2 + run) * a.R + member) * (M * 65);
}

// Every kernel here is launched so that it may start while the one before it in the stream ends,
// and waits for that one's results first.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Allows a kernel its dynamic shared memory, once per device (`done`: a bit each, of the first 64).
inline cudaError_t allow_smem(const void* kernel, size_t bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <class... P, class... A>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// two e4m3 codes (the lower or upper half of w) to f16, exact
__device__ __forceinline__ uint32_t half2_of(uint32_t w, bool upper) {
    uint32_t r;
    if (upper)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// 2^(byte - 127), the scale that a scale byte stands for; 255 stands for NaN (a row that held
// infinite or NaN elements)
__device__ __forceinline__ float pow2_of(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7fc00000u) : pow2_of(byte);
}

}  // namespace kv
}  // namespace bsa
