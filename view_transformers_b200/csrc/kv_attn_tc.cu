// Attention of new tokens over a paged key/value cache: the form for many query rows per
// key/value head (chunks and frames), on tcgen05. The mathematics is kv_attn.cu's; the bound here
// is the softmax: a 128 x 128 tile's exponentials (16 a clock and SM) take 1,024 clocks against
// 650 of matrix instructions, and its other instructions share the four schedulers with them.
// Measured on a B200, 16 heads, call by call with other inputs every pass: a frame of 782 new tokens
// over 78,200 cached ones in bf16: 418 us, 599 TFLOP/s (368 us, 681 TFLOP/s in a chain of graph nodes
// over three sets of inputs; the last of its seven tiles has 14 rows); a frame of 1,374 tokens over 33
// such frames in e4m3: 448 us, 569 TFLOP/s. Neither is at a pipe's limit (exponentials 43 to 48%, issue
// 47 to 55%, tensor 27%): a tile's chain (read S, maximum, exponentials, write P, products) is serial
// in a thread, and two such chains a scheduler do not hide its latency. With the exponentials left
// out the frame took 288 us in a chain, of 388 then. The steps' times below are of such chains.
//
// A block is that of the global layer's attention (attn_tc.cu): a TMA producer warp, an MMA warp
// per query tile (S = Q K^T into TMEM columns [0,128), O += P V with P (bf16) in [128,192) and O
// in [192,256)), four softmax warps per query tile with one query row per thread; persistent, the
// barriers running on across items as in frame_attn.cu. What differs:
//   - a query tile is the `group` heads of 128 / group tokens, one 3D TMA box;
//   - a 128-key tile is gathered from its pages by up to eight TMA boxes of whole pages; pages
//     that do not exist are not loaded, and the tile's page mask (a bit per 16 keys) goes to the
//     softmax with the stage;
//   - tiles that not every row of the block sees whole are taken key by key from a 128-bit mask
//     per row. Their rows of V that no row sees are zeroed before the product, and NaN or
//     infinite values that only some rows see are taken out of V and marked in the rows that do;
//   - bf16: one query tile a block, two blocks per SM. e4m3: two query tiles a block, one block per
//     SM. Its codes are copied raw into a ring of half tiles (K, V, K, ...) and four further warps turn
//     them into the bf16 tiles that both products read (exact: power-of-two scales). They convert a
//     tile once for 256 rows, and leave the registers for whole rows of scores (two blocks of one
//     tile each measured 494 against 458 us, but 85 against 94 us on 15 chunks of 1 to 199 rows,
//     most with rows for one tile alone). The schedulers fetch all roles' code, so the conversion's
//     loop is kept short: the frame of 1,374 tokens took 546 us with it unrolled four times and 488
//     with it not unrolled; later, beside the present softmax, 455 not unrolled and 450 twice;
//   - the R blocks of a team walk the same keys for R neighbouring pieces of a chunk, so that a
//     key/value tile comes from HBM once for all of them; the runs of teams are as in kv_cache.cuh.
// Every wait is bounded; a timeout is reported through the status word.
#include <cuda.h>

#include <type_traits>

#include "kv_cache.cuh"
#include "sm100.cuh"
#include "tma_map.cuh"

namespace bsa {
namespace {

using namespace sm100;
using namespace kv;

constexpr uint32_t kTmemCols = 256, kColS = 0, kColP = 128, kColO = 192;   // of a query tile
constexpr float kScaleLog2 = 0.18033688011112042f;   // log2(e) / sqrt(64)
constexpr float kRescale = 8.0f;
constexpr float kNone = -1e38f;                      // the reference before anything is seen, below every finite score
constexpr float kLn2 = 0.69314718055994531f;
constexpr uint32_t kTile = 128 * 128;                // 128 rows of 64 bf16
constexpr uint32_t kRawHalf = 128 * 64 + 128;        // 128 e4m3 rows of K or V and their scales
constexpr int kRaw = 6;                              // raw half tiles in flight
constexpr int kAlone = 0x1000;                       // word of a key tile: the second query tile has no rows
constexpr uint64_t kDrainNs = 50000000ull;

template <bool FP8>
struct Cfg {
    static constexpr int T = FP8 ? 2 : 1;            // query tiles of a block
    static constexpr int NS = 3;                     // K/V stages
    // Every kPoly-th pair of a whole tile's weights is taken by exp2_poly. The frame chunk above: 388 us
    // without, 386 with every third, 374 with every fourth, 383 with every sixth; the window in e4m3, whose
    // schedulers also convert: 475 us without, 472 with every sixth, 465 with every eighth
    static constexpr int kPoly = FP8 ? 8 : 4;
    // warps 0 .. 3: producer, products; 4 T softmax warps; in e4m3 four for the conversion
    static constexpr int kThreads = FP8 ? 512 : 256;
    static constexpr uint32_t kOffQ = 0;
    static constexpr uint32_t kOffK = kOffQ + T * kTile;
    static constexpr uint32_t kOffV = kOffK + NS * kTile;
    static constexpr uint32_t kOffRaw = kOffV + NS * kTile;
    static constexpr uint32_t kOffList = kOffRaw + (FP8 ? kRaw * kRawHalf : 0);   // [NS][128] uint2
    static constexpr uint32_t kOffCtl = kOffList + (FP8 ? NS * 1024 : 0);
};

struct Ctl {
    uint64_t q_full, q_empty;
    uint64_t k_full[3], kv_empty[3], v_full[3];      // v_full: e4m3 only (bf16: with k_full)
    uint64_t clean[3];                               // of a stage's V, by the first query tile's warps (two tiles)
    uint64_t raw_full[kRaw], raw_empty[kRaw];
    uint64_t rec_full[2], rec_empty[2], meet;
    struct {
        uint64_t s_full, s_free, p_full, o_done, o_final;
    } q[2];                                          // of the query tiles
    uint64_t drain;
    Rec rec[2];
    int meta[3], tile[3];                            // of the stages
    int found[3];                                    // of the stages: the last tile with values taken out, plus 1
    int raw_meta[kRaw], raw_tile[kRaw];
    uint32_t tmem_base;
    int abort;
    Start start;
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* tm, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}
// untiled copy: both addresses 16-byte aligned, bytes a multiple of 16
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// orders this thread's shared-memory accesses before later accesses by TMA and tcgen05
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// one lane of a converged warp, the same one each time
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

// low n bits, any n
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// two e4m3 codes times a power of two, exact, through f16 and f32: half of the instructions go to
// the floating-point pipes (moving the bits with integer instructions alone measured slower)
__device__ __forceinline__ uint32_t bf16_of(uint32_t w, bool upper, float f) {
    const uint32_t h = half2_of(w, upper);
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const float2 r = __fmul2_rn(v, make_float2(f, f));
    return pack_bf16(r.x, r.y);
}

// 2^y for y <= 127 on the floating-point pipe: y = n + f with n its nearest integer (by adding and
// taking away 1.5 2^23, whose low bits then hold n + 127), a fourth-degree polynomial for 2^f on
// [-1/2, 1/2] (relative minimax by Remez' exchange, error 2.7e-6), times 2^n. Below 2^-126: 2^-126.
// NaN stays NaN.
__device__ __forceinline__ float2 exp2_poly(float2 y) {
    asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(y.x));   // -126
    asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(y.y));
    const float2 magic = make_float2(12583039.f, 12583039.f);   // 1.5 2^23 + 127
    const float2 t = __fadd2_rn(y, magic);
    const float2 n = __fadd2_rn(t, make_float2(-12583039.f, -12583039.f));
    const float2 f = __ffma2_rn(n, make_float2(-1.f, -1.f), y);
    float2 p = make_float2(0.009570102207362652f, 0.009570102207362652f);
    p = __ffma2_rn(p, f, make_float2(0.05591785907745361f, 0.05591785907745361f));
    p = __ffma2_rn(p, f, make_float2(0.240247443318367f, 0.240247443318367f));
    p = __ffma2_rn(p, f, make_float2(0.6931217908859253f, 0.6931217908859253f));
    p = __ffma2_rn(p, f, make_float2(0.9999992847442627f, 0.9999992847442627f));
    return __fmul2_rn(p, make_float2(__uint_as_float(__float_as_uint(t.x) << 23), __uint_as_float(__float_as_uint(t.y) << 23)));
}

template <bool FP8>
__global__ void __launch_bounds__(Cfg<FP8>::kThreads, FP8 ? 1 : 2)
kv_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ AttnArgs a) {
    using C = Cfg<FP8>;
    constexpr int NS = C::NS, T = C::T;
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctl& ctl = *reinterpret_cast<Ctl*>(smem + C::kOffCtl);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int team = blockIdx.x / a.R, member = blockIdx.x - team * a.R;
    volatile int* abort = &ctl.abort;
    let_next_start();
    wait_for_previous();

    if (threadIdx.x == 0 && member == 0) a.desc[team * kDesc] = 0;
    // tile swizzles assume a 1024-byte aligned base; refuse to run otherwise
    if ((smem_u32(smem) & 1023u) != 0u) {
        if (threadIdx.x == 0) record_error(a.status, BSA_ERR_DEVICE_BOUNDS);
        return;
    }
    int* tables = reinterpret_cast<int*>(smem);
    const Start start = plan(a, team, tables, tables + BSA_KV_MAX_SEQS + 1, &ctl.start);
    if (team >= start.teams || start.total == 0) return;
    if (threadIdx.x == 0) {
        mbar_init(&ctl.q_full, 1);
        mbar_init(&ctl.q_empty, T);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&ctl.k_full[s], FP8 ? 4 : 1);
            mbar_init(&ctl.v_full[s], 4);
            mbar_init(&ctl.kv_empty[s], T);
            mbar_init(&ctl.clean[s], 4);
            ctl.found[s] = 0;
        }
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(&ctl.raw_full[s], 1);
            mbar_init(&ctl.raw_empty[s], 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ctl.rec_full[s], 1);
            mbar_init(&ctl.rec_empty[s], 4 * T);
        }
        for (int s = 0; s < T; ++s) {
            mbar_init(&ctl.q[s].s_full, 1);
            mbar_init(&ctl.q[s].s_free, 4);
            mbar_init(&ctl.q[s].p_full, 4);
            mbar_init(&ctl.q[s].o_done, 1);
            mbar_init(&ctl.q[s].o_final, 1);
        }
        mbar_init(&ctl.drain, T);
        mbar_init(&ctl.meet, 4);
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
        tmem_alloc(&ctl.tmem_base, T * kTmemCols);
        tmem_relinquish();
    }
    fence_async_shared();   // the plan's tables lay where TMA writes next
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;
    int issued = 0;         // K/V tiles (e4m3: half tiles) whose loads the producer issued
    int q_loads = 0;        // Q tiles the producer issued

    // Roles 0 (producer), 1 and 2 (products of the first and second query tile) of warps 0 .. 3, 4:
    // softmax, 5: conversion. A warp's scheduler is its number modulo 4, for the softmax's too, so two
    // blocks of an SM (told apart by where their tensor memory lies) take the roles in opposite
    // halves: no row quarter of a tile then trails the others.
    const int role = warp >= 4 + 4 * T ? 5 : warp >= 4 ? 4 : T == 1 && (tmem & 0xffffu) ? warp ^ 2 : warp;
    const int tile_rows = a.mr / T;   // a query tile's

    // registers a thread: together what the block is launched with (128 a thread). bf16 80 and 176: 375
    // instead of 371 us; e4m3 72 and 184: 477 instead of 472
    if (role < 4) {
        if (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (role == 0) {
            // ======================================================== producer
            int U = 0, I = 0, X = 0;     // tiles, Q loads, segments so far
            int alone = 0;               // kAlone if the segment has no rows for the second query tile
            auto put_record = [&](const Rec& r) -> bool {
                const int slot = X & 1;
                alone = r.nrows <= tile_rows ? kAlone : 0;
                if (X >= 2 && !warp_wait(&ctl.rec_empty[slot], ((X >> 1) - 1) & 1, abort, a.status)) return false;
                if (lane == 0) {
                    ctl.rec[slot] = r;
                    mbar_arrive(&ctl.rec_full[slot]);
                }
                ++X;
                return true;
            };
            auto begin = [&](const Walk& w, int r0) -> bool {
                if (I > 0 && !warp_wait(&ctl.q_empty, (I - 1) & 1, abort, a.status)) return false;
                if (lane == 0) {
                    const int loads = T == 1 || alone ? 1 : 2;
                    mbar_arrive_expect_tx(&ctl.q_full, loads * tile_rows * 128);
                    for (int i = 0; i < loads; ++i)
                        tma_load_3d(smem + C::kOffQ + i * kTile, &tm_q, &ctl.q_full, 0, w.h * a.group,
                                    w.q.row0 + (r0 + i * tile_rows) / a.group);
                }
                q_loads = ++I;
                return true;
            };
            auto put_tile = [&](int words, int t, int boxes, int rows, int at) -> bool {
                const int meta = words | alone;
                const int box = kUnit / boxes, i = lane - at;   // this lane's box
                const int row = i >= 0 && i < boxes ? rows : -1, k = i * box;
                const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
                if (!FP8) {
                    const int st = U % NS;
                    if (U >= NS && !warp_wait(&ctl.kv_empty[st], ((U / NS) - 1) & 1, abort, a.status)) return false;
                    if (lane == 0) {
                        ctl.meta[st] = meta;
                        ctl.tile[st] = t;
                        mbar_arrive_expect_tx(&ctl.k_full[st], __popc(have) * box * 256);
                    }
                    __syncwarp();
                    if (row >= 0) {
                        tma_load_2d(smem + C::kOffK + st * kTile + k * 128, &tm_k, &ctl.k_full[st], 0, row);
                        tma_load_2d(smem + C::kOffV + st * kTile + k * 128, &tm_v, &ctl.k_full[st], 0, row);
                    }
                    issued = U + 1;
                } else {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int x = 2 * U + half, slot = x % kRaw;
                        if (x >= kRaw && !warp_wait(&ctl.raw_empty[slot], ((x / kRaw) - 1) & 1, abort, a.status))
                            return false;
                        uint8_t* dst = smem + C::kOffRaw + slot * kRawHalf;
                        if (lane == 0) {
                            ctl.raw_meta[slot] = meta;
                            ctl.raw_tile[slot] = t;
                            mbar_arrive_expect_tx(&ctl.raw_full[slot], __popc(have) * box * 65);
                        }
                        __syncwarp();
                        if (row >= 0) {
                            bulk_load(dst + k * 64, static_cast<const uint8_t*>(half ? a.v : a.k) + (long long)row * 64,
                                      box * 64, &ctl.raw_full[slot]);
                            bulk_load(dst + 8192 + k, (half ? a.vs : a.ks) + row, box, &ctl.raw_full[slot]);
                        }
                        issued = x + 1;
                    }
                }
                ++U;
                return true;
            };
            const bool ok = produce(a, start, team, member, lane, put_record, begin, put_tile);
            // no further tile, no further segment
            if (ok) {
                const int st = U % NS, x = 2 * U, slot = x % kRaw;
                if (!FP8 ? U < NS || warp_wait(&ctl.kv_empty[st], ((U / NS) - 1) & 1, abort, a.status)
                         : x < kRaw || warp_wait(&ctl.raw_empty[slot], ((x / kRaw) - 1) & 1, abort, a.status)) {
                    if (lane == 0) {
                        if (FP8) {
                            ctl.raw_meta[slot] = kEnd;
                            mbar_arrive(&ctl.raw_full[slot]);
                        } else {
                            ctl.meta[st] = kEnd;
                            mbar_arrive(&ctl.k_full[st]);
                        }
                    }
                    Rec rec = {};
                    rec.tiles = -1;
                    put_record(rec);
                }
            }
        } else if (role <= T) {
            // ======================================================== MMA issuer of query tile g
            // The whole warp runs the loop, so that addresses and descriptors are uniform values, and one
            // lane issues. (With one lane in the loop, issuing a tile's ten products and commits took
            // 1,100 clocks, and this thread, not the exponentials, set the pace.)
            const bool leader = elect_one();
            const int g = T == 1 ? 0 : role - 1;
            const uint32_t tm = tmem + g * kTmemCols;
            constexpr uint32_t idesc_qk = idesc_f16(128, 128, 1u, false);
            constexpr uint32_t idesc_pv = idesc_f16(128, 64, 1u, true);
            const uint64_t q_desc = sdesc_sw128(smem_u32(smem + C::kOffQ + g * kTile), 16, 1024);
            const uint64_t k_desc = sdesc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
            const uint64_t v_desc = sdesc_sw128(smem_u32(smem + C::kOffV), 0, 1024);
            auto issue_qk = [&](int st) {
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)   // 32 bytes a step, in 16-byte units
                        mma_ss(tm + kColS, q_desc + 2 * ks, k_desc + (uint64_t)(st * (kTile >> 4)) + 2 * ks, idesc_qk,
                               ks > 0 ? 1u : 0u);
                    mma_commit(&ctl.q[g].s_full);
                }
                __syncwarp();
            };
            int I = 0, U = 0, meta = 0, st = 0;   // segments, tiles of this query tile
            uint32_t turn = 0u;            // parity of the stage's use
            bool fresh = true;             // the next tile starts a segment
            for (;;) {
                if (fresh) {               // within a segment its QK^T is issued already
                    if (!warp_wait(&ctl.k_full[st], turn, abort, a.status)) break;
                    meta = *(volatile int*)&ctl.meta[st];
                    if (meta & kEnd) break;
                    if (g == 1 && (meta & kAlone)) {
                        __syncwarp();
                        if (leader) {
                            mbar_arrive(&ctl.kv_empty[st]);
                            if (meta & kLast) mbar_arrive(&ctl.q_empty);
                        }
                        if (meta & kLast) ++I;
                        turn ^= st + 1 == NS ? 1u : 0u;
                        st = st + 1 == NS ? 0 : st + 1;
                        continue;
                    }
                    if (!warp_wait(&ctl.q_full, I & 1, abort, a.status)) break;
                    ++I;
                    // the previous segment's last S has been read by the softmax
                    if (U > 0 && !warp_wait(&ctl.q[g].s_free, (U - 1) & 1, abort, a.status)) break;
                    tc_fence_after();
                    issue_qk(st);
                }
                const int cur = meta;
                const int sn = st + 1 == NS ? 0 : st + 1;
                const uint32_t tn = st + 1 == NS ? turn ^ 1u : turn;
                fresh = (cur & kLast) != 0;
                if (!fresh) {
                    if (!warp_wait(&ctl.k_full[sn], tn, abort, a.status) ||
                        !warp_wait(&ctl.q[g].s_free, U & 1, abort, a.status))
                        break;
                    tc_fence_after();
                    issue_qk(sn);
                    meta = *(volatile int*)&ctl.meta[sn];
                } else if (leader) {
                    mma_commit(&ctl.q_empty);   // the segment's last Q K^T is issued
                }
                if (FP8 && !warp_wait(&ctl.v_full[st], turn, abort, a.status)) break;
                if (!warp_wait(&ctl.q[g].p_full, U & 1, abort, a.status)) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)   // 16 rows of 128 bytes a step
                        mma_ts(tm + kColO, tm + kColP + 8 * ks, v_desc + (uint64_t)(st * (kTile >> 4)) + 128 * ks, idesc_pv,
                               (!(cur & kFirst) || ks > 0) ? 1u : 0u);
                    mma_commit(&ctl.kv_empty[st]);
                    mma_commit(&ctl.q[g].o_done);
                    if (fresh) mma_commit(&ctl.q[g].o_final);
                }
                __syncwarp();
                ++U;
                st = sn;
                turn = tn;
            }
        }
    } else if (FP8 && role == 5) {
        // ============================================================ e4m3 -> bf16
        // four lanes share a row of 64 codes; each writes two 16-byte chunks of the swizzled
        // bf16 row. Rows of pages that do not exist are left as they are.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const int cw = warp - 4 - 4 * T;
        bool ok = true;
        for (int U = 0; ok; ++U) {
            const int st = U % NS;
            if (U >= NS && !warp_wait(&ctl.kv_empty[st], ((U / NS) - 1) & 1, abort, a.status)) break;
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
                if (cw == 0 && lane == 0 && half == 0) {
                    ctl.meta[st] = meta;
                    ctl.tile[st] = ctl.raw_tile[slot];
                }
                if (meta & kEnd) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.k_full[st]);
                    ok = false;
                    break;
                }
#pragma unroll 2      // a short loop: see above
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 32 + cw * 8 + (lane >> 2);
                    if ((meta >> (r >> 4)) & 1) {
                        const uint4 c = *reinterpret_cast<const uint4*>(src + r * 64 + (lane & 3) * 16);
                        const uint32_t b = src[8192 + r];
                        const float f = scale_of(b);
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
        }
    } else {
        // ============================================================ softmax + epilogue
        if (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int quad = warp & 3, g = T == 1 ? 0 : (warp >> 2) - 1;   // g: the query tile
        const int row = quad * 32 + lane;
        const uint32_t lane_base = tmem + g * kTmemCols + ((uint32_t)(quad * 32) << 16);
        int U = 0, N = 0, I = 0, met = 0;                    // N: tiles of the block, U, I: of this query tile
        auto meet = [&]() -> bool {   // the first query tile's four warps; bounded like every wait
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.meet);
            return warp_wait(&ctl.meet, met++ & 1, abort, a.status);
        };
        for (int X = 0;; ++X) {
            if (!warp_wait(&ctl.rec_full[X & 1], (X >> 1) & 1, abort, a.status)) break;
            const Rec& rec = ctl.rec[X & 1];
            const int tiles = rec.tiles;
            if (tiles < 0) break;
            const int nrows = min(tile_rows, rec.nrows - g * tile_rows), r0 = rec.r0 + g * tile_rows;
            if (nrows <= 0) {         // the products skip these tiles too
                N += tiles;
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.rec_empty[X & 1]);
                continue;
            }
            float m_ref = kNone, l = 0.f;
            uint32_t poison0 = 0u, poison1 = 0u;   // columns that met a non-finite value of a key the row sees
            int lo = 0, hi = 0;
            if (row < nrows) visible(a, rec.len, rec.pos0 + a.by_group.of(r0 + row), lo, hi);
            bool ok = true;
            for (int u = 0; u < tiles; ++u, ++U, ++N) {
                const int st = N % NS;
                if (!warp_wait(&ctl.q[g].s_full, U & 1, abort, a.status)) { ok = false; break; }
                tc_fence_after();
                uint32_t s[128];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tmem_ld32(lane_base + kColS + 32 * k, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * k]));
                // the tile's words: written before k_full, for which the product's thread waited
                const int meta = *(volatile int*)&ctl.meta[st];
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.q[g].s_free);
                if (!(meta & kFull)) {
                    // columns of this row that count
                    const int k0 = ctl.tile[st] * kUnit;
                    uint32_t see[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int b = k0 + 32 * k;
                        see[k] = low_bits(hi - b) & (~low_bits(lo - b) | low_bits(a.sink - b)) &
                                 (((meta >> (2 * k)) & 1 ? 0xffffu : 0u) | ((meta >> (2 * k + 1)) & 1 ? 0xffff0000u : 0u));
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (__all_sync(0xffffffffu, see[k] == 0xffffffffu)) continue;
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!((see[k] >> c) & 1u)) s[32 * k + c] = 0xff800000u;   // -infinity
                    }
                    // What was taken out of each row of V. One query tile: rare, and K's tile is done with (S
                    // is there), so its memory passes it on.
                    uint2* list = reinterpret_cast<uint2*>(T == 2 ? smem + C::kOffList + st * 1024
                                                                  : smem + C::kOffK + st * kTile);
                    if (g == 0) {
                        // V of key k0 + row: P = 0 does not silence what is not finite
                        if (FP8 && !warp_wait(&ctl.v_full[st], (N / NS) & 1, abort, a.status)) { ok = false; break; }
                        uint4* v = reinterpret_cast<uint4*>(smem + C::kOffV + st * kTile + row * 128);
                        const int key = k0 + row;
                        const bool any =
                            ((meta >> (row >> 4)) & 1) && key < rec.hi_max && (key >= rec.lo_min || key < a.sink);
                        // Keys that some rows see and others do not, if any: the rest a NaN spoils for all, or none
                        const bool mixed = (rec.hi_min < rec.hi_max && rec.hi_min < k0 + kUnit && rec.hi_max > k0) ||
                                           (rec.lo_min < rec.lo_max && rec.lo_min < k0 + kUnit && rec.lo_max > k0);
                        if (!any) {
#pragma unroll
                            for (int c = 0; c < 8; ++c) v[c ^ (row & 7)] = make_uint4(0u, 0u, 0u, 0u);
                        }
                        if (mixed) {
                            uint32_t bad0 = 0u, bad1 = 0u;
#pragma unroll 2
                            for (int c = 0; c < (any ? 8 : 0); ++c) {   // columns 8 c .. 8 c + 7, swizzled
                                uint4* at = v + (c ^ (row & 7));
                                const uint4 x = *at;
                                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
                                uint32_t full = 0u;         // an exponent of all ones carries into the sign's place
#pragma unroll
                                for (int i = 0; i < 4; ++i) full |= (y[i] & 0x7f807f80u) + 0x00800080u;
                                if (full & 0x80008000u) {
                                    uint32_t bits = 0u, z[4];
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const bool b0 = (y[i] & 0x7f80u) == 0x7f80u, b1 = (y[i] & 0x7f800000u) == 0x7f800000u;
                                        z[i] = (b0 ? 0u : y[i] & 0xffffu) | (b1 ? 0u : y[i] & 0xffff0000u);
                                        bits |= (b0 ? 1u : 0u) << (2 * i) | (b1 ? 2u : 0u) << (2 * i);
                                    }
                                    *at = make_uint4(z[0], z[1], z[2], z[3]);
                                    if (c < 4) bad0 |= bits << (8 * c);
                                    else bad1 |= bits << (8 * c - 32);
                                }
                            }
                            if (bad0 | bad1) ctl.found[st] = N + 1;
                            if (!meet()) { ok = false; break; }
                            if (*(volatile int*)&ctl.found[st] == N + 1) {
                                list[row] = make_uint2(bad0, bad1);
                                if (!meet()) { ok = false; break; }
                            }
                        }
                        fence_async_shared();
                    } else if (!warp_wait(&ctl.clean[st], (N / NS) & 1, abort, a.status)) {
                        ok = false;
                        break;
                    }
                    if (*(volatile int*)&ctl.found[st] == N + 1) {
#pragma unroll 1
                        for (int k = 0; k < 4; ++k)
#pragma unroll 1
                            for (int c = 0; c < 32; ++c)
                                if ((see[k] >> c) & 1u) {
                                    const uint2 b = list[32 * k + c];
                                    poison0 |= b.x;
                                    poison1 |= b.y;
                                }
                        if (T == 1) fence_async_shared();
                    }
                }
                if (T == 2 && g == 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.clean[st]);
                }
                float mt;
                {
                    float acc[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] = __uint_as_float(s[i]);
#pragma unroll
                    for (int c = 4; c < 128; c += 2)
                        acc[(c / 2) & 3] = max3f(acc[(c / 2) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                    mt = fmaxf(fmaxf(acc[0], acc[1]), fmaxf(acc[2], acc[3]));
                }
                const float mt2 = mt * kScaleLog2;
                const bool need = mt2 > m_ref + kRescale;
                const bool corr = need && m_ref != kNone;
                const float new_ref = need ? mt2 : m_ref;
                const float factor = corr ? ex2_approx(m_ref - new_ref) : 1.f;
                m_ref = new_ref;
                float2 r2[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) r2[i] = make_float2(0.f, 0.f);
                const float2 scale2 = make_float2(kScaleLog2, kScaleLog2);
                const float2 shift2 = make_float2(-m_ref, -m_ref);
                // 128 scores to 64 pairs of weights, in place
                auto weigh = [&](auto whole_tile) {
#pragma unroll
                    for (int c = 0; c < 128; c += 2) {
                        const int i = c / 2;
                        const float2 y =
                            __ffma2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, shift2);
                        const float2 pr = decltype(whole_tile)::value && i % C::kPoly == C::kPoly - 1
                                              ? exp2_poly(y)
                                              : make_float2(ex2_approx(y.x), ex2_approx(y.y));
                        r2[i & 3] = __fadd2_rn(r2[i & 3], pr);
                        s[i] = pack_bf16(pr.x, pr.y);
                    }
                };
                if (meta & kFull) weigh(std::true_type{});
                else weigh(std::false_type{});
                // P.V of the item's previous tile must be done before O is rescaled or P is
                // overwritten (for the first tile, the previous item's o_final wait covered it)
                if (u > 0 && !warp_wait(&ctl.q[g].o_done, (U - 1) & 1, abort, a.status)) { ok = false; break; }
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
                for (int k = 0; k < 2; ++k)
                    tmem_st32(lane_base + kColP + 32 * k, *reinterpret_cast<const uint32_t(*)[32]>(&s[32 * k]));
                l = l * factor + (((r2[0].x + r2[0].y) + (r2[1].x + r2[1].y)) + ((r2[2].x + r2[2].y) + (r2[3].x + r2[3].y)));
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.q[g].p_full);
            }
            if (!ok) break;
            // -------------------------------------------------------- epilogue of the segment
            const bool some = tiles > 0;
            if (some) {
                if (!warp_wait(&ctl.q[g].o_final, I & 1, abort, a.status)) break;
                tc_fence_after();
                ++I;
            }
            // nothing seen, or scores of -infinity alone (exp2_poly gives those 2^-126). NaN stays.
            const bool none = l == 0.f || (m_ref == kNone && l == l);
            const float inv = none ? 0.f : 1.f / l;
            const float lse = none ? -INFINITY : (m_ref + log2f(l)) * kLn2;
            const bool whole = rec.whole;
            const int i = a.by_group.of(r0 + row);
            const int head = rec.h * a.group + (r0 + row - i * a.group);
            float* part = part_at<128 * T>(a, team, rec.run, member);
            const int at = g * tile_rows + row;
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
                if (row < nrows) {
                    if (whole) {
                        __nv_bfloat16* dst = a.out + (long long)(rec.row0 + i) * a.out_stride + head * 64 + 32 * k;
#pragma unroll
                        for (int c = 0; c < 32; c += 8) Vec16<__nv_bfloat16>::store(dst + c, o + c);
                    } else {
                        float* dst = part + at * 64 + 32 * k;
#pragma unroll
                        for (int c = 0; c < 32; c += 4) Vec16<float>::store(dst + c, o + c);
                    }
                }
            }
            if (row < nrows) {
                if (!whole) part[T * 128 * 64 + at] = lse;
                else if (a.lse != nullptr) a.lse[(long long)head * a.rows + rec.row0 + i] = lse;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.rec_empty[X & 1]);
        }
    }

    // ------------------------------------------------------------------ teardown
    __syncthreads();
    if (ctl.abort) {
        volatile int never = 0;
        if (role == 0 && lane == 0) {
            if (q_loads > 0) mbar_wait(&ctl.q_full, (q_loads - 1) & 1, &never, a.status, kDrainNs);
            constexpr int ring = FP8 ? kRaw : NS;
            for (int u = max(0, issued - ring); u < issued; ++u)
                mbar_wait(FP8 ? &ctl.raw_full[u % ring] : &ctl.k_full[u % ring], (u / ring) & 1, &never, a.status, kDrainNs);
        }
        if (role >= 1 && role <= T && elect_one()) {   // the threads that issued the products
            mma_commit(&ctl.drain);
            mbar_wait(&ctl.drain, 0, &never, a.status, kDrainNs);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, T * kTmemCols);
    }
}

template <bool FP8>
cudaError_t launch(AttnArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
    using C = Cfg<FP8>;
    const size_t smem = C::kOffCtl + (sizeof(Ctl) + 15) / 16 * 16;
    auto kern = kv_tc_kernel<FP8>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed);
    if (e != cudaSuccess) return e;
    return launch_early(kern, dim3(a.max_teams * a.R), C::kThreads, smem, st, q, k, v, a);
}

}  // namespace

cudaError_t launch_kv_merge(const AttnArgs& a, bool wide, cudaStream_t st);

// Blocks per team. The R blocks of a team read the same keys at about the same time, so with
// tiles query tiles per chunk the cache comes from HBM tiles / R times instead of tiles times;
// against that stand the members without a tile in a chunk's last row group and the blocks left
// over when R does not divide their number. The largest R within 4% of the best use of the
// blocks; 1 for chunks of unequal lengths (max_new well above the mean), whose short ones would
// leave members idle. The frame chunk above: R = 7 388 us, R = 1 432 us (of 388 then).
static int team_size(const AttnArgs& a, int blocks, int max_new) {
    const int tiles = (int)(((long long)max_new * a.group + a.mr - 1) / a.mr);
    if (tiles < 2 || (long long)a.rows * 100 < (long long)a.c.seqs * max_new * 85) return 1;
    int best = 1;
    for (int r = 2; r <= 16 && r <= tiles; ++r) {
        const double use = (double)tiles / ((tiles + r - 1) / r * r) * (blocks / r * r) / blocks;
        if (use >= 0.96) best = r;   // R = 1 uses all of them
    }
    return best;
}

cudaError_t launch_kv_tc(AttnArgs& a, bool fp8, int max_new, cudaStream_t st) {
    const uint32_t tokens = 128 / a.group;
    const int per_block = fp8 ? Cfg<true>::T : Cfg<false>::T;
    a.mr = (int)tokens * a.group * per_block;
    a.max_teams /= per_block;            // as many blocks per SM as keep its tensor memory full
    a.R = team_size(a, a.max_teams, max_new);
    a.max_teams /= a.R;
    a.set_divisors();
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
    return e != cudaSuccess ? e : launch_kv_merge(a, fp8, st);
}

}  // namespace bsa
