// Attention of new tokens over a paged key/value cache: the form for many query rows per
// key/value head (chunks and frames), on tcgen05. The mathematics is kv_attn.cu's; the bound here
// is the exponentials (16 a clock and SM: 128 x 128 scores take 1,024 clocks against 650 of
// matrix instructions), then the tensor pipe.
//
// A block is that of the global layer's attention (attn_tc.cu): a TMA producer warp, one MMA
// thread (S = Q K^T into TMEM columns [0,128), O += P V with P (bf16) in [128,192) and O in
// [192,256)), four softmax warps with one query row per thread, two blocks per SM; persistent,
// the barriers running on across items as in frame_attn.cu. What differs:
//   - a query tile is the `group` heads of 128 / group tokens (mr rows), one 3D TMA box;
//   - a 128-key tile is gathered from its pages by up to eight TMA boxes of whole pages; pages
//     that do not exist are not loaded, and the tile's page mask (a bit per 16 keys) goes to the
//     softmax with the stage;
//   - tiles that not every row of the tile sees whole are taken key by key from a 128-bit mask
//     per row. Their rows of V that no row sees are zeroed before the product, and NaN or
//     infinite values that only some rows see are taken out of V and marked in the rows that do;
//   - an e4m3 cache is copied raw into a ring of half tiles (K, V, K, ...) and two further warps
//     turn it into the bf16 tiles that the MMA reads (exact: power-of-two scales);
//   - the R blocks of a team walk the same keys for R neighbouring query tiles, so that a
//     key/value tile comes from HBM once for all of them; the runs of teams are as in kv_cache.cuh.
// Every wait is bounded; a timeout is reported through the status word.
#include <cuda.h>

#include "kv_cache.cuh"
#include "sm100.cuh"
#include "tma_map.cuh"

namespace bsa {
namespace {

using namespace sm100;
using namespace kv;

constexpr uint32_t kTmemCols = 256, kColS = 0, kColP = 128, kColO = 192;
constexpr float kScaleLog2 = 0.18033688011112042f;   // log2(e) / sqrt(64)
constexpr float kRescale = 8.0f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr uint32_t kTile = 128 * 128;                // 128 rows of 64 bf16
constexpr uint32_t kRawHalf = 128 * 64 + 128;        // 128 e4m3 rows of K or V and their scales
constexpr int kRaw = 3;                              // raw half tiles in flight
constexpr uint64_t kDrainNs = 50000000ull;

template <bool FP8>
struct Cfg {
    static constexpr int NS = FP8 ? 2 : 3;           // K/V stages
    static constexpr int kThreads = FP8 ? 256 : 192;
    static constexpr int kSoftmaxWarp = FP8 ? 4 : 2; // first of the four softmax warps
    static constexpr uint32_t kOffQ = 0;
    static constexpr uint32_t kOffK = kTile;
    static constexpr uint32_t kOffV = kOffK + NS * kTile;
    static constexpr uint32_t kOffRaw = kOffV + NS * kTile;
    static constexpr uint32_t kOffCtl = kOffRaw + (FP8 ? kRaw * kRawHalf : 0);
};

struct Ctl {
    uint64_t q_full, q_empty;
    uint64_t k_full[3], kv_empty[3], v_full[3];      // v_full: e4m3 only (bf16: with k_full)
    uint64_t raw_full[kRaw], raw_empty[kRaw];
    uint64_t s_full, s_free, p_full, o_done, o_final, drain;
    int meta[3];                                     // page mask of the stage's tile
    int raw_meta[kRaw];
    uint32_t tmem_base;
    int abort;
    Start start;
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

// This block's query tile within a segment, and the tiles of the segment's run that it needs.
struct Mine {
    const AttnArgs& a;
    const Walk& w;
    int r0, nrows;         // first row within the chunk; rows (0: nothing to do)
    Span own;
    int j;
    __device__ __forceinline__ Mine(const AttnArgs& args, const Walk& walk, int member) : a(args), w(walk) {
        r0 = (w.rg * a.R + member) * a.mr;
        nrows = min(a.mr, w.q.n * a.group - r0);
        if (nrows > 0) own = rows_span(a, w.q, r0, r0 + a.mr);
        j = w.j0;
    }
    // next key tile; false at the end of the run
    __device__ __forceinline__ bool next(int& t) {
        while (j < w.j1) {
            t = unit_of(w.span, j++);
            const int k0 = t * kUnit;
            if (k0 < own.hi_max && (k0 + kUnit > own.lo_min || k0 < a.sink)) return true;
        }
        return false;
    }
};

// low n bits, any n
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

__device__ __forceinline__ uint32_t half2_of(uint32_t w, bool upper) {   // two e4m3 codes, exact
    uint32_t r;
    if (upper)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
// two e4m3 codes times a power of two, exact: f16, its exponent field moved into a bf16 as it is
// (2^-112 times the value), one product with 2^(112 + e)
__device__ __forceinline__ uint32_t bf16_of(uint32_t w, bool upper, __nv_bfloat162 f) {
    const uint32_t h = half2_of(w, upper);
    const uint32_t b = ((h >> 3) & 0x0fff0fffu) | (h & 0x80008000u);
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b), f);
    return *reinterpret_cast<const uint32_t*>(&r);
}

template <bool FP8>
__global__ void __launch_bounds__(Cfg<FP8>::kThreads, 2)
kv_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const AttnArgs a) {
    using C = Cfg<FP8>;
    constexpr int NS = C::NS;
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctl& ctl = *reinterpret_cast<Ctl*>(smem + C::kOffCtl);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int team = blockIdx.x / a.R, member = blockIdx.x - team * a.R;
    volatile int* abort = &ctl.abort;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x == 0 && member == 0) a.desc[team * kDesc] = 0;
    // tile swizzles assume a 1024-byte aligned base; refuse to run otherwise
    if ((smem_u32(smem) & 1023u) != 0u) {
        if (threadIdx.x == 0) record_error(a.status, BSA_ERR_DEVICE_BOUNDS);
        return;
    }
    plan(a, team, reinterpret_cast<long long*>(smem),
         reinterpret_cast<int*>(smem + sizeof(long long) * (BSA_KV_MAX_SEQS + 1)), &ctl.start);
    const Start start = ctl.start;
    if (team >= start.teams) return;
    if (threadIdx.x == 0) {
        mbar_init(&ctl.q_full, 1);
        mbar_init(&ctl.q_empty, 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&ctl.k_full[s], FP8 ? 2 : 1);
            mbar_init(&ctl.v_full[s], 2);
            mbar_init(&ctl.kv_empty[s], 1);
        }
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(&ctl.raw_full[s], 1);
            mbar_init(&ctl.raw_empty[s], 2);
        }
        mbar_init(&ctl.s_full, 1);
        mbar_init(&ctl.s_free, 4);
        mbar_init(&ctl.p_full, 4);
        mbar_init(&ctl.o_done, 1);
        mbar_init(&ctl.o_final, 1);
        mbar_init(&ctl.drain, 1);
        ctl.abort = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch(&tm_q);
        if (!FP8) {
            tma_prefetch(&tm_k);
            tma_prefetch(&tm_v);
        }
    }
    if (warp == 1) {
        tmem_alloc(&ctl.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    fence_async_shared();   // the plan's tables lay where TMA writes next
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;
    int issued = 0;         // K/V tiles (e4m3: half tiles) whose loads the producer issued
    int q_loads = 0;        // Q tiles the producer issued

    if (warp < C::kSoftmaxWarp) {
        if (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == 0) {
            // ======================================================== producer
            const int box = min(1 << a.c.pshift, 128), shift = min(a.c.pshift, 7);   // keys of a TMA box
            int U = 0, I = 0;
            bool ok = true;
            Walk w(a, start, team);
            while (ok && w.next()) {
                Mine mine(a, w, member);
                int t;
                if (mine.nrows <= 0 || !mine.next(t)) {
                    w.done();
                    continue;
                }
                if (I > 0 && !warp_wait(&ctl.q_empty, (I - 1) & 1, abort, a.status)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&ctl.q_full, a.mr * 128);
                    tma_load_3d(smem + C::kOffQ, &tm_q, &ctl.q_full, 0, w.h * a.group, w.q.row0 + mine.r0 / a.group);
                }
                q_loads = ++I;
                do {
                    // the pages of the tile, one box per lane
                    const int k0 = t * kUnit + lane * box;
                    int page = -1;
                    if (lane < (128 >> shift) && k0 < mine.own.hi_max &&
                        (k0 + box > mine.own.lo_min || k0 < a.sink))
                        page = a.c.table[(long long)w.s * a.c.max_pages + (k0 >> a.c.pshift)];
                    if (page >= a.c.pages) {
                        record_error(a.status, BSA_ERR_DEVICE_BOUNDS);
                        page = -1;
                    }
                    const unsigned have = __ballot_sync(0xffffffffu, page >= 0);
                    int meta = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) meta |= ((have >> ((i * 16) >> shift)) & 1u) << i;
                    const long long row = page < 0 ? 0
                        : (((long long)page * a.c.kv_heads + w.h) << a.c.pshift) + (k0 & ((1 << a.c.pshift) - 1));
                    const uint32_t at = lane * box;
                    if (!FP8) {
                        const int st = U % NS;
                        if (U >= NS && !warp_wait(&ctl.kv_empty[st], ((U / NS) - 1) & 1, abort, a.status)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) {
                            ctl.meta[st] = meta;
                            mbar_arrive_expect_tx(&ctl.k_full[st], __popc(have) * box * 256);
                        }
                        __syncwarp();
                        if (page >= 0) {
                            tma_load_2d(smem + C::kOffK + st * kTile + at * 128, &tm_k, &ctl.k_full[st], 0, (int)row);
                            tma_load_2d(smem + C::kOffV + st * kTile + at * 128, &tm_v, &ctl.k_full[st], 0, (int)row);
                        }
                        issued = U + 1;
                    } else {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int x = 2 * U + half, slot = x % kRaw;
                            if (x >= kRaw && !warp_wait(&ctl.raw_empty[slot], ((x / kRaw) - 1) & 1, abort, a.status)) {
                                ok = false;
                                break;
                            }
                            uint8_t* dst = smem + C::kOffRaw + slot * kRawHalf;
                            if (lane == 0) {
                                ctl.raw_meta[slot] = meta;
                                mbar_arrive_expect_tx(&ctl.raw_full[slot], __popc(have) * box * 65);
                            }
                            __syncwarp();
                            if (page >= 0) {
                                bulk_load(dst + at * 64, static_cast<const uint8_t*>(half ? a.v : a.k) + row * 64, box * 64,
                                          &ctl.raw_full[slot]);
                                bulk_load(dst + 8192 + at, (half ? a.vs : a.ks) + row, box, &ctl.raw_full[slot]);
                            }
                            issued = x + 1;
                        }
                        if (!ok) break;
                    }
                    ++U;
                } while (mine.next(t));
                w.done();
            }
        } else if (warp == 1) {
            // ======================================================== MMA issuer
            if (lane == 0) {
                constexpr uint32_t idesc_qk = idesc_f16(128, 128, 1u, false);
                constexpr uint32_t idesc_pv = idesc_f16(128, 64, 1u, true);
                const uint32_t q_base = smem_u32(smem + C::kOffQ);
                auto issue_qk = [&](int U) -> bool {
                    const int st = U % NS;
                    if (!mbar_wait(&ctl.k_full[st], (U / NS) & 1, abort, a.status)) return false;
                    tc_fence_after();
                    const uint32_t k_base = smem_u32(smem + C::kOffK + st * kTile);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_ss(tmem + kColS, sdesc_sw128(q_base + 32 * ks, 16, 1024),
                               sdesc_sw128(k_base + 32 * ks, 16, 1024), idesc_qk, ks > 0 ? 1u : 0u);
                    mma_commit(&ctl.s_full);
                    return true;
                };
                int U = 0, I = 0;
                bool ok = true;
                Walk w(a, start, team);
                while (ok && w.next()) {
                    Mine mine(a, w, member);
                    int t;
                    if (mine.nrows <= 0 || !mine.next(t)) {
                        w.done();
                        continue;
                    }
                    if (!mbar_wait(&ctl.q_full, I & 1, abort, a.status)) break;
                    // the previous item's last S has been read by the softmax
                    if (U > 0 && !mbar_wait(&ctl.s_free, (U - 1) & 1, abort, a.status)) break;
                    if (!issue_qk(U)) break;
                    for (bool first = true, more = true; more; first = false, ++U) {
                        more = mine.next(t);
                        if (more) {
                            if (!mbar_wait(&ctl.s_free, U & 1, abort, a.status) || !issue_qk(U + 1)) {
                                ok = false;
                                break;
                            }
                        } else {
                            mma_commit(&ctl.q_empty);   // the item's last Q K^T is issued
                        }
                        const int st = U % NS;
                        if (FP8 && !mbar_wait(&ctl.v_full[st], (U / NS) & 1, abort, a.status)) {
                            ok = false;
                            break;
                        }
                        if (!mbar_wait(&ctl.p_full, U & 1, abort, a.status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t v_base = smem_u32(smem + C::kOffV + st * kTile);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_ts(tmem + kColO, tmem + kColP + 8 * ks, sdesc_sw128(v_base + 2048 * ks, 0, 1024), idesc_pv,
                                   (!first || ks > 0) ? 1u : 0u);
                        mma_commit(&ctl.kv_empty[st]);
                        mma_commit(&ctl.o_done);
                        if (!more) mma_commit(&ctl.o_final);
                    }
                    ++I;
                    w.done();
                }
            }
        } else if (FP8) {
            // ======================================================== e4m3 -> bf16
            // four lanes share a row of 64 codes; each writes two 16-byte chunks of the swizzled
            // bf16 row. Rows of pages that do not exist are left as they are.
            const int cw = warp - 2;
            int U = 0;
            bool ok = true;
            Walk w(a, start, team);
            while (ok && w.next()) {
                Mine mine(a, w, member);
                int t;
                if (mine.nrows <= 0) {
                    w.done();
                    continue;
                }
                while (mine.next(t)) {
                    const int st = U % NS;
                    if (U >= NS && !warp_wait(&ctl.kv_empty[st], ((U / NS) - 1) & 1, abort, a.status)) {
                        ok = false;
                        break;
                    }
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        const int x = 2 * U + half, slot = x % kRaw;
                        if (!warp_wait(&ctl.raw_full[slot], (x / kRaw) & 1, abort, a.status)) {
                            ok = false;
                            break;
                        }
                        const uint8_t* src = smem + C::kOffRaw + slot * kRawHalf;
                        uint8_t* dst = smem + (half ? C::kOffV : C::kOffK) + st * kTile;
                        const int meta = ctl.raw_meta[slot];
                        if (cw == 0 && lane == 0 && half == 0) ctl.meta[st] = meta;
#pragma unroll 4
                        for (int i = 0; i < 8; ++i) {
                            const int r = i * 16 + cw * 8 + (lane >> 2);
                            if ((meta >> i) & 1) {
                                const uint4 c = *reinterpret_cast<const uint4*>(src + r * 64 + (lane & 3) * 16);
                                const uint32_t b = src[8192 + r];
                                // 2^(b - 127 + 112); bytes above 142 (255, or never written): NaN
                                const uint32_t f1 = b > 142u ? 0x7fc0u : (b + 112u) << 7, f2 = f1 | (f1 << 16);
                                const __nv_bfloat162 f = *reinterpret_cast<const __nv_bfloat162*>(&f2);
                                const int c0 = 2 * (lane & 3);
                                *reinterpret_cast<uint4*>(dst + r * 128 + ((c0 ^ (r & 7)) * 16)) =
                                    make_uint4(bf16_of(c.x, false, f), bf16_of(c.x, true, f), bf16_of(c.y, false, f),
                                               bf16_of(c.y, true, f));
                                *reinterpret_cast<uint4*>(dst + r * 128 + (((c0 + 1) ^ (r & 7)) * 16)) =
                                    make_uint4(bf16_of(c.z, false, f), bf16_of(c.z, true, f), bf16_of(c.w, false, f),
                                               bf16_of(c.w, true, f));
                            }
                        }
                        fence_async_shared();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(half ? &ctl.v_full[st] : &ctl.k_full[st]);
                            mbar_arrive(&ctl.raw_empty[slot]);
                        }
                    }
                    if (!ok) break;
                    ++U;
                }
                w.done();
            }
        }
    } else {
        // ============================================================ softmax + epilogue
        if (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        const int quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        int U = 0, I = 0;
        bool ok = true;
        Walk w(a, start, team);
        while (ok && w.next()) {
            Mine mine(a, w, member);
            if (mine.nrows <= 0) {
                w.done();
                continue;
            }
            float m_ref = -INFINITY, l = 0.f;
            uint32_t poison0 = 0u, poison1 = 0u;   // columns that met a non-finite value of a key the row sees
            int lo = 0, hi = 0;
            if (row < mine.nrows) visible(a, w.q.len, w.q.len - w.q.n + (mine.r0 + row) / a.group, lo, hi);
            int t;
            bool first = true;
            while (mine.next(t)) {
                const int st = U % NS;
                if (!warp_wait(&ctl.s_full, U & 1, abort, a.status)) { ok = false; break; }
                tc_fence_after();
                uint32_t s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32(lane_base + kColS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c]));
                // done already (the product waited for it): orders the read of the page mask
                if (!warp_wait(&ctl.k_full[st], (U / NS) & 1, abort, a.status)) { ok = false; break; }
                const int meta = ctl.meta[st];
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.s_free);
                const int k0 = t * kUnit;
                const Span& own = mine.own;
                const bool full = meta == 0xff && k0 + kUnit <= own.hi_min &&
                                  (k0 >= own.lo_max || k0 + kUnit <= min(a.sink, own.lo_min));
                float mt = -INFINITY;
                uint32_t see[4];
                if (full) {
                    float acc[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] = __uint_as_float(s[i]);
#pragma unroll
                    for (int c = 8; c < 128; c += 2)
                        acc[(c / 2) & 7] = max3f(acc[(c / 2) & 7], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                    mt = max3f(max3f(acc[0], acc[1], acc[2]), max3f(acc[3], acc[4], acc[5]), fmaxf(acc[6], acc[7]));
                } else {
                    // columns of this row that count
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int b = k0 + 32 * k;
                        see[k] = low_bits(hi - b) & (~low_bits(lo - b) | low_bits(a.sink - b)) &
                                 (((meta >> (2 * k)) & 1 ? 0xffffu : 0u) | ((meta >> (2 * k + 1)) & 1 ? 0xffff0000u : 0u));
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            if (!((see[k] >> c) & 1u)) s[32 * k + c] = 0xff800000u;   // -infinity
                            mt = fmaxf(mt, __uint_as_float(s[32 * k + c]));
                        }
                    }
                    // V of key k0 + row: P = 0 does not silence what is not finite
                    if (FP8 && !warp_wait(&ctl.v_full[st], (U / NS) & 1, abort, a.status)) { ok = false; break; }
                    uint4* v = reinterpret_cast<uint4*>(smem + C::kOffV + st * kTile + row * 128);
                    const int key = k0 + row;
                    const bool any = ((meta >> (row >> 4)) & 1) && key < own.hi_max && (key >= own.lo_min || key < a.sink);
                    uint32_t bad0 = 0u, bad1 = 0u;
                    if (any) {
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            const uint4 x = v[c];
                            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
                            uint32_t bits = 0u, z[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const bool b0 = (y[i] & 0x7f80u) == 0x7f80u, b1 = (y[i] & 0x7f800000u) == 0x7f800000u;
                                z[i] = (b0 ? 0u : y[i] & 0xffffu) | (b1 ? 0u : y[i] & 0xffff0000u);
                                bits |= (b0 ? 1u : 0u) << (2 * i) | (b1 ? 2u : 0u) << (2 * i);
                            }
                            if (bits) {
                                v[c] = make_uint4(z[0], z[1], z[2], z[3]);
                                const int col = ((c ^ (row & 7)) & 7) * 8;   // the chunk's first column
                                if (col < 32) bad0 |= bits << col;
                                else bad1 |= bits << (col - 32);
                            }
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 8; ++c) v[c] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    // rare: K's tile is done with (S is read), so its memory passes the columns on
                    uint32_t found;
                    asm volatile(
                        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                        "barrier.cta.red.or.pred.aligned q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                        : "=r"(found) : "r"(bad0 | bad1) : "memory");
                    if (found) {
                        uint2* list = reinterpret_cast<uint2*>(smem + C::kOffK + st * kTile);
                        list[row] = make_uint2(bad0, bad1);
                        asm volatile("barrier.cta.sync.aligned 1, 128;" ::: "memory");
#pragma unroll 1
                        for (int k = 0; k < 4; ++k)
#pragma unroll 1
                            for (int c = 0; c < 32; ++c)
                                if ((see[k] >> c) & 1u) {
                                    const uint2 b = list[32 * k + c];
                                    poison0 |= b.x;
                                    poison1 |= b.y;
                                }
                        asm volatile("barrier.cta.sync.aligned 1, 128;" ::: "memory");
                    }
                    fence_async_shared();
                }
                const float mt2 = mt * kScaleLog2;
                const bool need = mt2 > m_ref + kRescale;
                const bool corr = need && m_ref != -INFINITY;
                const float new_ref = need ? mt2 : m_ref;
                const float factor = corr ? ex2_approx(m_ref - new_ref) : 1.f;
                m_ref = new_ref;
                const float ref = m_ref == -INFINITY ? 0.f : m_ref;   // nothing seen yet: every p is 0
                float2 r2[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) r2[i] = make_float2(0.f, 0.f);
                const float2 scale2 = make_float2(kScaleLog2, kScaleLog2);
                const float2 shift2 = make_float2(-ref, -ref);
#pragma unroll
                for (int c = 0; c < 128; c += 2) {
                    const int i = c / 2;
                    const float2 x =
                        __ffma2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, shift2);
                    const float2 pr = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                    r2[i & 3] = __fadd2_rn(r2[i & 3], pr);
                    s[i] = pack_bf16(pr.x, pr.y);
                }
                const float rs =
                    ((r2[0].x + r2[0].y) + (r2[1].x + r2[1].y)) + ((r2[2].x + r2[2].y) + (r2[3].x + r2[3].y));
                l = l * factor + rs;
                // P.V of the item's previous tile must be done before O is rescaled or P is
                // overwritten (for the first tile, the previous item's o_final wait covered it)
                if (!first && !warp_wait(&ctl.o_done, (U - 1) & 1, abort, a.status)) { ok = false; break; }
                tc_fence_after();
                if (__any_sync(0xffffffffu, corr)) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t o[32];
                        tmem_ld32(lane_base + kColO + 32 * k, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * factor);
                        tmem_st32(lane_base + kColO + 32 * k, o);
                    }
                }
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    tmem_st32(lane_base + kColP + 32 * c, *reinterpret_cast<const uint32_t(*)[32]>(&s[32 * c]));
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_full);
                first = false;
                ++U;
            }
            if (!ok) break;
            // -------------------------------------------------------- epilogue of the segment
            const bool some = !first;
            if (some) {
                if (!warp_wait(&ctl.o_final, I & 1, abort, a.status)) { ok = false; break; }
                tc_fence_after();
                ++I;
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;   // l = 0: nothing seen. NaN stays.
            const float lse = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
            const bool whole = w.has_start && w.has_end;
            const int i = (mine.r0 + row) / a.group;
            const int head = w.h * a.group + (mine.r0 + row - i * a.group);
            float* part = part_at<128>(a, team, w.has_start ? 1 : 0, member);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float o[32];
                if (some) {
                    uint32_t v[32];
                    tmem_ld32(lane_base + kColO + 32 * k, v);
                    tmem_wait_ld();
                    const uint32_t bad = k ? poison1 : poison0;
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        o[c] = __uint_as_float(v[c]) * inv;
                        if ((bad >> c) & 1u) o[c] = __uint_as_float(0x7fc00000u);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = 0.f;
                }
                if (row < mine.nrows) {
                    if (whole) {
                        __nv_bfloat16* dst = a.out + (long long)(w.q.row0 + i) * a.out_stride + head * 64 + 32 * k;
#pragma unroll
                        for (int c = 0; c < 32; c += 8) Vec16<__nv_bfloat16>::store(dst + c, o + c);
                    } else {
                        float* dst = part + row * 64 + 32 * k;
#pragma unroll
                        for (int c = 0; c < 32; c += 4) Vec16<float>::store(dst + c, o + c);
                    }
                }
            }
            if (row < mine.nrows) {
                if (!whole) part[128 * 64 + row] = lse;
                else if (a.lse != nullptr) a.lse[(long long)head * a.rows + w.q.row0 + i] = lse;
            }
            tc_fence_before();
            if (row == 0 && member == 0 && !whole && w.has_start) {   // the merge kernel's record of this item
                int* d = a.desc + team * kDesc;
                d[1] = w.q.row0;
                d[2] = w.q.n;
                d[3] = w.h;
                d[4] = w.rg;
                d[5] = w.last_team(w.item + max(1, w.span.count), start.total);
                d[0] = 1;
            }
            w.done();
        }
    }

    // ------------------------------------------------------------------ teardown
    __syncthreads();
    if (ctl.abort) {
        volatile int never = 0;
        if (warp == 0 && lane == 0) {
            if (q_loads > 0) mbar_wait(&ctl.q_full, (q_loads - 1) & 1, &never, a.status, kDrainNs);
            constexpr int ring = FP8 ? kRaw : NS;
            for (int u = max(0, issued - ring); u < issued; ++u)
                mbar_wait(FP8 ? &ctl.raw_full[u % ring] : &ctl.k_full[u % ring], (u / ring) & 1, &never, a.status, kDrainNs);
        }
        if (warp == 1 && lane == 0) {
            mma_commit(&ctl.drain);
            mbar_wait(&ctl.drain, 0, &never, a.status, kDrainNs);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <bool FP8>
cudaError_t launch(AttnArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
    using C = Cfg<FP8>;
    const size_t smem = C::kOffCtl + (sizeof(Ctl) + 15) / 16 * 16;
    auto kern = kv_tc_kernel<FP8>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<a.max_teams * a.R, C::kThreads, smem, st>>>(q, k, v, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_merge128(const AttnArgs& a, cudaStream_t st);

cudaError_t launch_kv_tc(AttnArgs& a, bool fp8, cudaStream_t st) {
    const uint32_t tokens = 128 / a.group;
    a.mr = (int)tokens * a.group;
    a.min_run = 2;
    const uint64_t rows = ((uint64_t)a.c.pages * a.c.kv_heads) << a.c.pshift;
    const uint32_t box = a.c.pshift < 7 ? 1u << a.c.pshift : 128u;
    CUtensorMap q, k, v;
    if (!make_rows_map(&q, a.q, a.rows, a.c.heads, a.q_stride, a.group, tokens)) return cudaErrorInvalidValue;
    if (fp8) {
        k = v = q;
    } else if (!make_tile_map(&k, a.k, rows, 64, box, false) || !make_tile_map(&v, a.v, rows, 64, box, false)) {
        return cudaErrorInvalidValue;
    }
    const cudaError_t e = fp8 ? launch<true>(a, q, k, v, st) : launch<false>(a, q, k, v, st);
    return e != cudaSuccess ? e : launch_kv_merge128(a, st);
}

}  // namespace bsa
