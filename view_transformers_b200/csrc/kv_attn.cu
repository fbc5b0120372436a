// Attention of new tokens over a paged key/value cache: the form for few query rows per
// key/value head (single tokens, camera and register tokens, grouped heads), and the merge of
// split rows that it shares with the form for many.
//
//   out = sum_j p_j v_j / l, p_j = 2^(x_j - m), x_j = q.k_j log2(e)/8, l = sum_j p_j, over the
//   keys a row sees, with a running reference m that is raised only when some x exceeds it by 8.
//
// With few rows the keys and values are read once and nothing else matters: the bound is HBM
// (128 bytes a row of K or V, 65 in e4m3). So the matrix instruction is the small one (mma.sync),
// with 8 rows of its 16 (the cache is read once per 8 rows). Measured on a B200, call by call with other
// inputs every pass, one token each: 32 streams of up to 32,768 keys, 32 heads over 8, e4m3: 149 us,
// 4.02 TB/s (0.61 of the copy rate; 132 us in a chain of graph nodes over three sets of inputs); 8
// streams of 16,000 keys, 16 heads, bf16: 113 us, 4.64 TB/s; one token over 7,820 keys: 17.0 us, of
// which the split of the work, the first loads' latency and the merge are most. Other steps' times in
// this file are of such chains. No pipe is at its limit in e4m3 (issue 60%, integer 47%, HBM 54% in
// the chain): the latency of a group's loads and conversions is not hidden by two blocks an SM.
//   - a block is eight warps that work alone until an item ends: each takes every eighth group of
//     16 (bf16) or 32 (e4m3) keys, copies them asynchronously into a ring of its own (two groups
//     ahead, across items) and keeps its own m, l and O. Page ids are fetched 32 groups at a time, a
//     lane each, when the 32 before are used up or an item begins; that group's copy waits for them.
//     (One producer warp with TMA for all eight was measured: at 1,400 to 2,000 clocks a tile it
//     kept e4m3 at 61% of HBM.)
//   - a dot product does not care about the order of its terms, so the lane that must hold
//     neighbouring d of key g takes 16 neighbouring bytes of that key instead, and Q is loaded in
//     the same order; P.V's columns are dealt out so that a lane needs 8 neighbouring d of its
//     keys. All reads of a stage are 8 or 16 bytes wide and free of bank conflicts: bf16 rows are
//     swizzled as they are copied (16-byte chunk c of row r at c ^ (r & 7)); e4m3 rows are not, and
//     the keys are numbered so that the four rows that a lane quad needs lie next to each other.
// bf16: P is rounded to bf16.
// e4m3: the integer pipe (two clocks an instruction) is the busiest, so the codes become f16 by
// the one conversion there is and their scales go elsewhere: a K row's into the scores; a V
// row's, 2^e, into P: w_j = p_j 2^(e_j), rounded to f16 relative to the largest w of the group (full
// precision over 28 binades, whatever the scales), and the group's product is added to O in fp32
// at its own scale. Q is f16 too, scaled by a power of two per row, exact for elements within
// 2^-28 of the row's largest. (The e4m3 form of mma.sync, with Q and P in two parts each, measured
// slower: 184 against 165 us on 32 ragged streams.)
#include "kv_cache.cuh"
#include "sm100.cuh"

namespace bsa {
namespace {

using namespace kv;
using sm100::ex2_approx;

constexpr int kWarps = 8;
constexpr int M = 8;                                 // rows of a query tile
constexpr int kThreads = kWarps * 32;
constexpr float kScaleLog2 = 0.18033688011112042f;   // log2(e) / sqrt(64)
constexpr float kRescale = 8.0f;
constexpr float kLn2 = 0.69314718055994531f;

template <bool FP8>
struct Cfg {
    static constexpr int kKeys = FP8 ? 32 : 16;                       // keys of a group
    static constexpr int kPer = kUnit / kKeys;                        // groups of a unit
    static constexpr uint32_t kV = 2048;                              // a stage: K, V, K scales, V scales
    static constexpr uint32_t kStage = 4096 + (FP8 ? 64 : 0);
    static constexpr int kStages = 3;
    static constexpr uint32_t kMerge = kWarps * kStages * kStage;     // [4][row][64], [4][row][2]
    static constexpr uint32_t kSmem = kMerge + 4 * M * 66 * 4;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the scales whose bytes `pick` takes from two words of scale bytes
__device__ __forceinline__ float2 scales_of(uint32_t w0, uint32_t w1, uint32_t pick) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, lo;\n\t}" : "=r"(r) : "r"(__byte_perm(w0, w1, pick)));
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}

__device__ __forceinline__ bool has_nonfinite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 2)
kv_rows_kernel(const __grid_constant__ AttnArgs a) {
    using namespace sm100;
    using C = Cfg<FP8>;
    constexpr int GK = C::kKeys;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Start shared_start;
    // columns of a row that met a NaN or infinite value; two sets, of which the next item's is
    // written while the last one's is cleared
    __shared__ uint32_t poisons[2][M][2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int team = blockIdx.x;
    if (tid < M * 4) (&poisons[0][0][0])[tid] = 0u;
    let_next_start();
    wait_for_previous();
    int* tables = reinterpret_cast<int*>(smem);
    const Start st = plan(a, team, tables, tables + BSA_KV_MAX_SEQS + 1, &shared_start);
    if (tid == 0) a.desc[team * kDesc] = 0;
    if (team >= st.teams || st.total == 0) return;
    __syncthreads();

    const uint32_t ring = smem_u32(smem) + warp * (C::kStages * C::kStage);
    float* mo = reinterpret_cast<float*>(smem + C::kMerge);           // [4][row][64]
    float* mml = mo + 4 * M * 64;                                     // [4][row][2]
    const int g = lane >> 2, t = lane & 3;

    // first key of group x of a segment, and whether any row may see some of its keys
    auto first_key = [](const Span& sp, int x) { return unit_of(sp, x / C::kPer) * kUnit + x % C::kPer * GK; };
    auto wanted = [&](const Span& sp, int k0) { return k0 < sp.hi_max && (k0 + GK > sp.lo_min || k0 < a.sink); };
    // this warp's groups of a segment are first_group, first_group + 8, ...
    auto first_group = [&](const Walk& w) { return w.j0 * C::kPer + ((warp - w.j0 * C::kPer) & (kWarps - 1)); };

    Walk w(a, st, team);
    bool more = w.next();
    // ---------------------------------------------------------------- the loader
    // lane i holds the pool rows of the group base + 8 i (its two 16-key halves) of its segment, and
    // bit i of `full` tells whether every row sees every key of that group
    Walk lw = w;
    bool live = more;
    int lx = live ? first_group(lw) : 0, base = lx - 8 * 32, row0h = -1, row1h = -1;
    uint32_t full = 0u;
    uint32_t held = 0u;                     // 4 bits per stage: the halves that hold keys; full
    auto load_step = [&](int stage) {
        while (live && lx >= lw.j1 * C::kPer) {
            lw.done();
            live = lw.next();
            lx = live ? first_group(lw) : 0;
            base = lx - 8 * 32;
        }
        uint32_t got = 0u;
        if (live) {
            if (lx - base >= 8 * 32) {
                base = lx;
                const Span& sp = lw.span;
                const int x = lx + 8 * lane, k0 = first_key(sp, x);
                const bool in = x < lw.j1 * C::kPer && wanted(sp, k0);
                const int32_t* pages = a.c.table + (long long)lw.s * a.c.max_pages;
                auto row_of = [&](int k, bool use) {
                    const int page = use ? pages[k >> a.c.pshift] : -1;
                    if (page >= a.c.pages) record_error(a.status, BSA_ERR_DEVICE_BOUNDS);
                    return page < 0 || page >= a.c.pages
                               ? -1
                               : ((page * a.c.kv_heads + lw.h) << a.c.pshift) + (k & ((1 << a.c.pshift) - 1));
                };
                row0h = row_of(k0, in);
                // pages of 16 tokens end inside a group of 32; the second one may lie past the tables
                if (GK == 32)
                    row1h = a.c.pshift > 4 ? (row0h < 0 ? -1 : row0h + 16) : row_of(k0 + 16, in && k0 + 16 < sp.hi_max);
                full = __ballot_sync(0xffffffffu, row0h >= 0 && (GK == 16 || row1h >= 0) && k0 + GK <= sp.hi_min &&
                                                      (k0 >= sp.lo_max || k0 + GK <= min(a.sink, sp.lo_min)));
            }
            const int from = (lx - base) >> 3;
            const int r0h = __shfl_sync(0xffffffffu, row0h, from);
            const int r1h = GK == 32 ? __shfl_sync(0xffffffffu, row1h, from) : -1;
            got = (r0h >= 0 ? 1u : 0u) | (r1h >= 0 ? 2u : 0u) | ((full >> from) & 1u) << 2;
            const uint32_t dst = ring + stage * C::kStage + lane * 16;
            if (!FP8) {
                if (got) {
                    const long long at = (long long)r0h * 128 + lane * 16;
                    const uint8_t* kp = static_cast<const uint8_t*>(a.k) + at;
                    const uint8_t* vp = static_cast<const uint8_t*>(a.v) + at;
                    // rows 4 i + lane / 8: the swizzle has one of two values
                    const int c = lane & 7, r = lane >> 3;
                    const uint32_t even = dst + ((c ^ r) - c) * 16, odd = dst + ((c ^ (r + 4)) - c) * 16;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        cp16((i & 1 ? odd : even) + i * 512, kp + i * 512);
                        cp16((i & 1 ? odd : even) + i * 512 + C::kV, vp + i * 512);
                    }
                }
            } else {
                auto copy = [&](int row, uint32_t to, int n) {   // n times 8 rows of K and V
                    const long long at = (long long)row * 64 + lane * 16;
                    const uint8_t* kp = static_cast<const uint8_t*>(a.k) + at;
                    const uint8_t* vp = static_cast<const uint8_t*>(a.v) + at;
#pragma unroll
                    for (int i = 0; i < n; ++i) {
                        cp16(to + i * 512, kp + i * 512);
                        cp16(to + i * 512 + C::kV, vp + i * 512);
                    }
                };
                const uint8_t* sc = lane & 2 ? a.vs : a.ks;      // lanes 0, 1: K, 2, 3: V; the halves
                if ((got & 3u) == 3u && r1h == r0h + 16) {
                    copy(r0h, dst, 4);
                    if (lane < 4) cp16(dst + 4096, sc + r0h + (lane & 1) * 16);
                } else {
                    if (r0h >= 0) copy(r0h, dst, 2);
                    if (r1h >= 0) copy(r1h, dst + 1024, 2);
                    const int rs = lane & 1 ? r1h : r0h;
                    if (lane < 4 && rs >= 0) cp16(dst + 4096, sc + rs);
                }
            }
            lx += 8;
        }
        held = (held & ~(15u << (4 * stage))) | (got << (4 * stage));
        cp_commit();
    };
    // ---------------------------------------------------------------- arithmetic
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) load_step(i);
    int stage = 0, set = 0;
    for (; more; set ^= 1) {
        uint32_t(&poison)[M][2] = poisons[set];
        const int row0 = w.q.row0, pos0 = w.q.len - w.q.n, len = w.q.len;
        const int r0 = w.rg * M, nrows = min(M, w.q.n * a.group - r0);
        const Span& sp = w.span;
        // ---------------------------------------------------------------- Q
        // k-step ks takes the words qf[ks][0] and qf[ks][1] of row g
        uint32_t qf[4][2];
        float rowf = kScaleLog2;            // x = score * rowf (e4m3: times the key's scale)
        uint4 c0 = make_uint4(0u, 0u, 0u, 0u), c1 = c0;
        if (g < nrows) {
            const int i = a.by_group.of(r0 + g);
            const uint4* p = reinterpret_cast<const uint4*>(a.q + (long long)(row0 + i) * a.q_stride +
                                                            ((long long)w.h * a.group + (r0 + g - i * a.group)) * 64);
            c0 = p[2 * t];
            c1 = p[2 * t + 1];
        }
        uint32_t wds[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        if (FP8) {
            // to f16 with the largest element of the row at 2^14 .. 2^15
            uint32_t top = 0u;
#pragma unroll
            for (int k = 0; k < 8; ++k) top = max(top, max(wds[k] & 0x7fffu, (wds[k] >> 16) & 0x7fffu));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = max((int)(top >> 7) - 14, 1);          // biased exponent of the factor
            const float inv = pow2_of(254 - e);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                wds[k] = pack_half2(__uint_as_float(wds[k] << 16) * inv, __uint_as_float(wds[k] & 0xffff0000u) * inv);
            rowf = kScaleLog2 * pow2_of(e);
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            qf[ks][0] = wds[2 * ks];
            qf[ks][1] = wds[2 * ks + 1];
        }
        float o[8][4];                      // row g: o[j][0] and o[j][1]; the other eight rows stay 0
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[j][c] = 0.f;
        float m = -INFINITY, l = 0.f;

        if constexpr (!FP8) {
#pragma unroll 1
        for (int gx = first_group(w); gx < w.j1 * C::kPer; gx += 8) {
            cp_wait<C::kStages - 2>();
            __syncwarp();
            const uint32_t there = (held >> (4 * stage)) & 3u;
            const bool all = (held >> (4 * stage)) & 4u;
            const uint32_t src = ring + stage * C::kStage;
            const int next_stage = stage == 0 ? C::kStages - 1 : stage - 1;   // emptied by the step before
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
            load_step(next_stage);
            if (there == 0u) continue;
            const int kb = all ? 0 : first_key(sp, gx);
            // column x (0 .. 7) of the scores' half jj stands for key jj * 8 + x of the warp's 16
            // ------------------------------------------------------------ scores
            float x[2][4];
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
#pragma unroll
                for (int c = 0; c < 4; ++c) x[jj][c] = 0.f;
                const int r = jj * 8 + g;
                const uint4 k0 = lds16(src + r * 128 + (((2 * t) ^ (r & 7)) << 4));
                const uint4 k1 = lds16(src + r * 128 + (((2 * t + 1) ^ (r & 7)) << 4));
                const uint32_t kw[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16(x[jj], qf[ks][0], 0u, qf[ks][1], 0u, kw[2 * ks], kw[2 * ks + 1]);
#pragma unroll
                for (int c = 0; c < 2; ++c) x[jj][c] *= kScaleLog2;
            }
            // ------------------------------------------------------------ V, and what is seen
            uint32_t vw[4][4];              // 8 values of the lane's four keys
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = (i >> 1) * 8 + 2 * t + (i & 1);
                const uint4 v = lds16(src + C::kV + r * 128 + ((g ^ (r & 7)) << 4));
                vw[i][0] = v.x;
                vw[i][1] = v.y;
                vw[i][2] = v.z;
                vw[i][3] = v.w;
            }
            if (!all) {
                int lo = 0, hi = 0;
                if (g < nrows) visible(a, len, pos0 + a.by_group.of(r0 + g), lo, hi);
#pragma unroll
                for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int key = kb + jj * 8 + 2 * t + c;
                        if (!(key < hi && (key >= lo || key < a.sink))) x[jj][c] = -INFINITY;
                    }
                // P = 0 does not silence a NaN: non-finite values are taken out of V and marked
                // in the rows that see them (none, past the end)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = kb + (i >> 1) * 8 + 2 * t + (i & 1);
                    bool bad = false;
#pragma unroll
                    for (int k = 0; k < 4; ++k) bad |= has_nonfinite(vw[i][k]);
                    if (bad) {
                        uint32_t cols = 0u;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if ((vw[i][k] & 0x7f80u) == 0x7f80u) {
                                cols |= 1u << (2 * k);
                                vw[i][k] &= 0xffff0000u;
                            }
                            if ((vw[i][k] & 0x7f800000u) == 0x7f800000u) {
                                cols |= 2u << (2 * k);
                                vw[i][k] &= 0xffffu;
                            }
                        }
                        for (int r = 0; r < nrows; ++r) {
                            int rlo, rhi;
                            visible(a, len, pos0 + a.by_group.of(r0 + r), rlo, rhi);
                            if (key < rhi && (key >= rlo || key < a.sink))
                                atomicOr(&poison[r][g >> 2], cols << ((g & 3) * 8));
                        }
                    }
                }
            }
            // ------------------------------------------------------------ softmax
            const float top = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
            if (__any_sync(0xffffffffu, top > m + kRescale)) {
                float n = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                n = fmaxf(fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 2)), m);
                const float f = m == -INFINITY ? 0.f : ex2_approx(m - n);
                m = n;
                l *= f;
#pragma unroll
                for (int j8 = 0; j8 < 8; ++j8) {
                    o[j8][0] *= f;
                    o[j8][1] *= f;
                }
            }
            uint32_t pf[2];
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const float p0 = ex2_approx(x[jj][0] - ref), p1 = ex2_approx(x[jj][1] - ref);
                l += p0 + p1;
                pf[jj] = pack_bf16(p0, p1);
            }
            // ------------------------------------------------------------ O += P V
#pragma unroll
            for (int j8 = 0; j8 < 8; ++j8) {
                const uint32_t sel = j8 & 1 ? 0x7632u : 0x5410u;
                mma_bf16(o[j8], pf[0], 0u, pf[1], 0u, __byte_perm(vw[0][j8 >> 1], vw[1][j8 >> 1], sel),
                         __byte_perm(vw[2][j8 >> 1], vw[3][j8 >> 1], sel));
            }
        }
        } else {
#pragma unroll 1
        for (int gx = first_group(w); gx < w.j1 * C::kPer; gx += 8) {
            cp_wait<C::kStages - 2>();
            __syncwarp();
            const uint32_t there = (held >> (4 * stage)) & 3u;
            const bool all = (held >> (4 * stage)) & 4u;
            const uint32_t src = ring + stage * C::kStage;
            const int next_stage = stage == 0 ? C::kStages - 1 : stage - 1;   // emptied by the step before
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
            load_step(next_stage);
            if (there == 0u) continue;
            const int kb = all ? 0 : first_key(sp, gx);
            // column c of the scores' eighth n stands for key 8 n + c / 2 (c even), 8 n + 4 + (c / 2 ^ 1)
            // (odd): pairs of columns differ in parity and equal columns of a quad lie together
            const int kg = g & 1 ? 4 + ((g >> 1) ^ 1) : g >> 1;   // key of column g
            const int k1 = 4 + (t ^ 1);                           // key of column 2 t + 1; 2 t: t
            const uint32_t pick = t | k1 << 4;                    // their bytes of two words
            // ------------------------------------------------------------ scores
            float x[4][2];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint4 kw = lds16(src + (8 * n + kg) * 64 + t * 16);
                const uint32_t kc[4] = {kw.x, kw.y, kw.z, kw.w};
                float h[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16(h, qf[ks][0], 0u, qf[ks][1], 0u, half2_of(kc[ks], false), half2_of(kc[ks], true));
#pragma unroll
                for (int c = 0; c < 2; ++c) x[n][c] = h[c];
            }
            // the rows' scales (NaN for byte 255): a K row's goes into the scores, a V row's into P
            float vs[4][2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint4 kb4 = lds16(src + 4096 + half * 16);
                const uint4 vb4 = lds16(src + 4096 + 32 + half * 16);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int n = 2 * half + i;
                    const float2 ks = scales_of(i ? kb4.z : kb4.x, i ? kb4.w : kb4.y, pick);
                    const float2 v = scales_of(i ? vb4.z : vb4.x, i ? vb4.w : vb4.y, pick);
                    vs[n][0] = v.x;
                    vs[n][1] = v.y;
                    x[n][0] *= ks.x;
                    x[n][1] *= ks.y;
                }
            }
            // ------------------------------------------------------------ V
            uint2 vc[2][4];                   // codes of d 8 g .. 8 g + 7 for the lane's eight keys
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    vc[half][i] = lds8(src + C::kV + (half * 16 + (i >> 1) * 8 + (i & 1 ? k1 : t)) * 64 + g * 8);
            // ------------------------------------------------------------ what is seen
            if (!all) {
                int lo = 0, hi = 0;
                if (g < nrows) visible(a, len, pos0 + a.by_group.of(r0 + g), lo, hi);
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int key = kb + 8 * n + (c ? k1 : t);
                        if (!(key < hi && (key >= lo || key < a.sink) && ((there >> (n >> 1)) & 1))) x[n][c] = -INFINITY;
                    }
                // stale memory may hold NaN codes (a written row never does: NaN is in its scale)
                auto clean = [](uint32_t& w) {
                    w &= ~(((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 255u);
                };
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        clean(vc[half][i].x);
                        clean(vc[half][i].y);
                    }
            }
            // ------------------------------------------------------------ softmax
            float top = fmaxf(x[0][0], x[0][1]);
#pragma unroll
            for (int n = 1; n < 4; ++n) top = fmaxf(top, fmaxf(x[n][0], x[n][1]));
            top *= rowf;
            if (__any_sync(0xffffffffu, top > m + kRescale)) {
                float n = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                n = fmaxf(fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 2)), m);
                const float f = m == -INFINITY ? 0.f : ex2_approx(m - n);
                m = n;
                l *= f;
#pragma unroll
                for (int j8 = 0; j8 < 8; ++j8) {
                    o[j8][0] *= f;
                    o[j8][1] *= f;
                }
            }
            uint32_t pf[4];                   // w of the lane's two keys of each eighth
            const float ref = m == -INFINITY ? 0.f : m;
            float p[4][2], top_w = 0.f, sum = 0.f;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float e = ex2_approx(fmaf(x[n][c], rowf, -ref));
                    sum += e;
                    // a masked score stays -infinity and its w 0, whatever the scale byte holds
                    p[n][c] = all || x[n][c] != -INFINITY ? e * vs[n][c] : 0.f;
                    top_w = fmaxf(top_w, p[n][c]);
                }
            l += sum;
            top_w = fmaxf(top_w, __shfl_xor_sync(0xffffffffu, top_w, 1));
            top_w = fmaxf(top_w, __shfl_xor_sync(0xffffffffu, top_w, 2));
            // 2^k <= top_w < 2^(k + 1): scaled by 2^(14 - k), undone by back (k kept within -100 .. 100)
            const int k2 = min(max((int)(__float_as_uint(top_w) >> 23), 27), 227);
            const float up = pow2_of(268 - k2), back = pow2_of(k2 - 14);
#pragma unroll
            for (int n = 0; n < 4; ++n) pf[n] = pack_half2(p[n][0] * up, p[n][1] * up);
            // ------------------------------------------------------------ O += back (w up) V
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    uint32_t ab[2], cd[2];    // d 4 k + 2 z and one further, two keys each
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint2(&v)[4] = vc[half];
                        const uint32_t sel = z ? 0x7362u : 0x5140u;
                        ab[half] = k ? __byte_perm(v[0].y, v[1].y, sel) : __byte_perm(v[0].x, v[1].x, sel);
                        cd[half] = k ? __byte_perm(v[2].y, v[3].y, sel) : __byte_perm(v[2].x, v[3].x, sel);
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float h[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int half = 0; half < 2; ++half)
                            mma_f16(h, pf[2 * half], 0u, pf[2 * half + 1], 0u, half2_of(ab[half], y), half2_of(cd[half], y));
                        const int j8 = 4 * k + 2 * z + y;
#pragma unroll
                        for (int c = 0; c < 2; ++c) o[j8][c] = fmaf(h[c], back, o[j8][c]);
                    }
                }
        }
        }

        // -------------------------------------------------------------------- the block's warps
        // warps 4 .. 7 hand theirs to warps 0 .. 3, those the sums to the whole block. Lane (g, t)
        // holds columns 16 t .. 16 t + 15 of row g: o[j][0] is 16 t + j, o[j][1] 8 further
        auto place = [&](int c, int j8) {
            return reinterpret_cast<float4*>(mo + ((warp & 3) * M + g) * 64 + 16 * t + 8 * c + j8);
        };
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        auto put = [&] {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j8 = 0; j8 < 8; j8 += 4)
                    *place(c, j8) = make_float4(o[j8][c], o[j8 + 1][c], o[j8 + 2][c], o[j8 + 3][c]);
            if (t == 0) {
                mml[((warp & 3) * M + g) * 2] = m;
                mml[((warp & 3) * M + g) * 2 + 1] = l;
            }
        };
        if (warp >= 4) put();
        __syncthreads();
        if (warp < 4) {
            const float mk = mml[(warp * M + g) * 2], lk = mml[(warp * M + g) * 2 + 1];
            const float n = fmaxf(m, mk);
            const float f0 = m == -INFINITY ? 0.f : ex2_approx(m - n);
            const float f1 = mk == -INFINITY ? 0.f : ex2_approx(mk - n);
            m = n;
            l = l * f0 + lk * f1;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j8 = 0; j8 < 8; j8 += 4) {
                    const float4 v = *place(c, j8);
                    o[j8][c] = o[j8][c] * f0 + v.x * f1;
                    o[j8 + 1][c] = o[j8 + 1][c] * f0 + v.y * f1;
                    o[j8 + 2][c] = o[j8 + 2][c] * f0 + v.z * f1;
                    o[j8 + 3][c] = o[j8 + 3][c] * f0 + v.w * f1;
                }
            __syncwarp();
            put();
        }
        __syncthreads();
        const bool whole = w.has_start && w.has_end;
        float* part = part_at<M>(a, team, w.has_start ? 1 : 0, 0);
        if (tid < M * 16) {
            const int r = tid >> 4, c4 = (tid & 15) * 4;
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) mm = fmaxf(mm, mml[(k * M + r) * 2]);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float mk = mml[(k * M + r) * 2];
                const float f = mk == -INFINITY ? 0.f : ex2_approx(mk - mm);
                const float4 v = *reinterpret_cast<const float4*>(mo + (k * M + r) * 64 + c4);
                ll += f * mml[(k * M + r) * 2 + 1];
                acc[0] += f * v.x;
                acc[1] += f * v.y;
                acc[2] += f * v.z;
                acc[3] += f * v.w;
            }
            // l = 0: nothing seen. NaN stays.
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            const uint32_t bad = poison[r][c4 >> 5] >> (c4 & 31);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[k] *= inv;
                if ((bad >> k) & 1u) acc[k] = __uint_as_float(0x7fc00000u);
            }
            const float lse = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
            if (r < nrows) {
                if (whole) {
                    const int i = a.by_group.of(r0 + r);
                    const int head = w.h * a.group + (r0 + r - i * a.group);
                    *reinterpret_cast<uint2*>(a.out + (long long)(row0 + i) * a.out_stride + head * 64 + c4) =
                        make_uint2(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]));
                    if (c4 == 0 && a.lse != nullptr) a.lse[(long long)head * a.rows + row0 + i] = lse;
                } else {
                    *reinterpret_cast<float4*>(part + r * 64 + c4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    if (c4 == 0) part[M * 64 + r] = lse;
                }
            }
        }
        if (tid == 0 && !whole && w.has_start) {   // the merge kernel's record of this item
            int* d = a.desc + team * kDesc;
            d[1] = row0;
            d[2] = w.q.n;
            d[3] = w.h;
            d[4] = w.rg;
            d[5] = st.team_of(w.item + max(1, sp.count) - 1);
            d[0] = 1;
        }
        __syncthreads();
        if (tid < M * 2) (&poison[0][0])[tid] = 0u;
        w.done();
        more = w.next();
    }
    cp_wait<0>();
}

// Joins the partial results of an item that crosses team ends: the team that holds its first
// unit left it in run 1, the following ones in run 0. L = ln sum e^lse, out = sum e^(lse - L) o,
// in an order that only the split decides. The blocks of a (team, member) share its rows, at most 16
// each; 16 threads hold a row's columns, and with fewer rows several sets of 16 share a row's pieces.
// (Eight pieces' loads at a time instead of four: ragged chunks 100 -> 108 us, for the registers.)
constexpr int kMergeRows = 16;
template <int ROWS>
__global__ void __launch_bounds__(kMergeRows * 16)
kv_merge_kernel(const AttnArgs a) {
    __shared__ float4 sacc[kMergeRows][16];
    __shared__ float2 sml[kMergeRows][16];
    let_next_start();
    wait_for_previous();
    const int team = blockIdx.x / a.R, member = blockIdx.x - team * a.R;
    const int* d = a.desc + team * kDesc;
    if (d[0] == 0) return;
    const int row0 = d[1], h = d[3], last = d[5];
    const int r0 = (d[4] * a.R + member) * a.mr, rows = min(a.mr, d[2] * a.group - r0);
    if (rows <= 0) return;                       // a member without rows
    // rows a block takes: 16, or with many pieces to join as few as the blocks there are allow (16 and 24
    // rows of 55 and 93 pieces each: 33 -> 22 us a step)
    const int blocks = gridDim.y;
    const int per = ROWS <= kMergeRows || last - team < 16 ? kMergeRows : (rows + blocks - 1) / blocks;
    const int rb = (int)blockIdx.y * per;
    const int nrows = min(rows - rb, per);
    if (nrows <= 0) return;
    int sets = 1;                                // sets of 16 threads per row: a power of two
    while (nrows * sets * 2 <= kMergeRows) sets *= 2;
    const int c = threadIdx.x & 15, slot = threadIdx.x >> 4, r = slot / sets, set = slot - r * sets;
    float m = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < nrows) {
        constexpr int U = 4;
        for (int k = team + set; k <= last; k += U * sets) {
            float e[U];
            float4 v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int kk = min(k + i * sets, last);
                const float* p = part_at<ROWS>(a, kk, kk == team ? 1 : 0, member);
                v[i] = *reinterpret_cast<const float4*>(p + (rb + r) * 64 + 4 * c);
                e[i] = part_at<ROWS>(a, kk, kk == team ? 1 : 0, member)[ROWS * 64 + rb + r] * 1.4426950408889634f;
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (k + i * sets > last || e[i] == -INFINITY) continue;
                const float n = fmaxf(m, e[i]), f0 = ex2_approx(m - n), f1 = ex2_approx(e[i] - n);
                m = n;
                sum = sum * f0 + f1;
                acc.x = acc.x * f0 + v[i].x * f1;
                acc.y = acc.y * f0 + v[i].y * f1;
                acc.z = acc.z * f0 + v[i].z * f1;
                acc.w = acc.w * f0 + v[i].w * f1;
            }
        }
    }
    if (sets > 1) {
        sacc[slot][c] = acc;
        sml[slot][c] = make_float2(m, sum);
        __syncthreads();
        if (set != 0 || r >= nrows) return;
        for (int k = 1; k < sets; ++k) {
            const float2 o = sml[slot + k][c];
            const float4 v = sacc[slot + k][c];
            if (o.y == 0.f) continue;            // nothing seen (a NaN sum has no maximum either)
            const float n = fmaxf(m, o.x), f0 = ex2_approx(m - n), f1 = ex2_approx(o.x - n);
            m = n;
            sum = sum * f0 + o.y * f1;
            acc.x = acc.x * f0 + v.x * f1;
            acc.y = acc.y * f0 + v.y * f1;
            acc.z = acc.z * f0 + v.z * f1;
            acc.w = acc.w * f0 + v.w * f1;
        }
    }
    if (r >= nrows) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int i = a.by_group.of(r0 + rb + r);
    const int head = h * a.group + (r0 + rb + r - i * a.group);
    *reinterpret_cast<uint2*>(a.out + (long long)(row0 + i) * a.out_stride + head * 64 + 4 * c) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (c == 0 && a.lse != nullptr)
        a.lse[(long long)head * a.rows + row0 + i] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
}

template <bool FP8>
cudaError_t launch_rows(AttnArgs& a, cudaStream_t st) {
    using C = Cfg<FP8>;
    auto kern = kv_rows_kernel<FP8>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), C::kSmem, allowed);
    if (e != cudaSuccess) return e;
    return launch_early(kern, dim3(a.max_teams), kThreads, C::kSmem, st, a);
}

}  // namespace

template <int ROWS>
static cudaError_t launch_merge(const AttnArgs& a, cudaStream_t st) {
    return launch_early(kv_merge_kernel<ROWS>, dim3(a.max_teams * a.R, (a.mr + kMergeRows - 1) / kMergeRows), kMergeRows * 16, 0,
                        st, a);
}

cudaError_t launch_kv_merge(const AttnArgs& a, bool wide, cudaStream_t st) {
    return wide ? launch_merge<256>(a, st) : launch_merge<128>(a, st);
}

cudaError_t launch_kv_rows(AttnArgs& a, bool fp8, cudaStream_t st) {
    a.R = 1;
    a.mr = M;
    a.set_divisors();
    const cudaError_t e = fp8 ? launch_rows<true>(a, st) : launch_rows<false>(a, st);
    return e != cudaSuccess ? e : launch_merge<M>(a, st);
}

}  // namespace bsa
