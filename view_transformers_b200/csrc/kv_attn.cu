// Attention of new tokens over a paged key/value cache: the form for few query rows per
// key/value head (single tokens, camera and register tokens, grouped heads), and the merge of
// split rows that it shares with the form for many.
//
//   out = sum_j p_j v_j / l, p_j = 2^(x_j - m), x_j = q.k_j log2(e)/8, l = sum_j p_j, over the
//   keys a row sees, with a running reference m that is raised only when some x exceeds it by 8.
//
// With few rows the keys and values are read once and nothing else matters: the bound is HBM
// (128 bytes a row of K or V, 65 in e4m3). So the matrix instruction is the small one (mma.sync),
// with M rows (8 or 16 of its 16):
//   - one warp gathers tiles of 128 keys from their pages by TMA into a ring of stages, running
//     ahead across items; eight warps share the tiles, each with its own m, l and O, and meet at
//     the end of an item;
//   - a dot product does not care about the order of its terms, so the lane that must hold
//     neighbouring d of key g takes 16 neighbouring bytes of that key instead, and Q is loaded in
//     the same order; P.V's columns are dealt out so that a lane needs 8 neighbouring d of its
//     keys. All reads of a stage are 8 or 16 bytes wide and free of bank conflicts: bf16 tiles are
//     swizzled by TMA (16-byte chunk c of row r at c ^ (r & 7)); e4m3 tiles are not, and the keys
//     are numbered so that the four rows that a lane quad needs lie next to each other.
// bf16: a warp takes 16 keys of each tile, P is rounded to bf16.
// e4m3: a warp takes 32 keys of every second tile. The bound is then the integer pipe (two clocks an
// instruction), so the codes become f16 by the one conversion there is and their scales go
// elsewhere: a K row's into the scores; a V row's, 2^e, into P: w_j = p_j 2^(e_j), rounded to f16
// relative to the largest w of the warp's 32 keys (full precision over 28 binades, whatever the
// scales), and the step's product is added to O in fp32 at its own scale. Q is f16 too, scaled by a
// power of two per row, exact for elements within 2^-28 of the row's largest. (The e4m3 form of
// mma.sync, with Q and P in two parts each, measured slower: 184 against 165 us with bf16 operands on
// 32 ragged streams.)
#include "kv_cache.cuh"
#include "sm100.cuh"
#include "tma_map.cuh"

namespace bsa {
namespace {

using namespace kv;
using sm100::ex2_approx;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32 + 32;           // and the producer's warp
constexpr float kScaleLog2 = 0.18033688011112042f;   // log2(e) / sqrt(64)
constexpr float kRescale = 8.0f;
constexpr float kLn2 = 0.69314718055994531f;

template <bool FP8, int M>
struct Cfg {
    // e4m3: K, V, and their scales; bf16: K and V. Two blocks share an SM.
    static constexpr uint32_t kV = FP8 ? 8192 : 16384;
    static constexpr uint32_t kStage = FP8 ? 2 * 8192 + 2 * 128 : 2 * 16384;
    // e4m3: even, so that a stage always belongs to the same half of the warps
    static constexpr int NS = FP8 ? 4 : (M == 8 ? 3 : 2);
    static constexpr int kSharers = FP8 ? 4 : 8;                      // warps that read a tile
    static constexpr uint32_t kMerge = NS * kStage;                   // [warp][row][64 + 2]
    static constexpr uint32_t kCtl = kMerge + kWarps * M * 66 * 4;
};

template <int M>
struct Ctl {
    uint64_t full[4], empty[4];
    uint64_t rec_full[2], rec_empty[2], meet;
    Rec rec[2];
    int meta[4], tile[4];
    uint32_t poison[M][2];                  // columns of a row that met a NaN or infinite value
    int abort;
    Start start;
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status) {
    return __all_sync(0xffffffffu, sm100::mbar_wait(bar, parity, abort, status));
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

// two e4m3 codes (the lower or upper half of w) to f16, exact
__device__ __forceinline__ uint32_t half2_of(uint32_t w, bool upper) {
    uint32_t r;
    if (upper)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ bool has_nonfinite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <bool FP8, int M>
__global__ void __launch_bounds__(kThreads, 2)
kv_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ AttnArgs a) {
    using namespace sm100;
    using C = Cfg<FP8, M>;
    constexpr int NH = M / 8;               // 8-row halves in use
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctl<M>& ctl = *reinterpret_cast<Ctl<M>*>(smem + C::kCtl);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int team = blockIdx.x;
    volatile int* abort = &ctl.abort;

    if (tid == 0) {
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(&ctl.full[s], 1);
            mbar_init(&ctl.empty[s], C::kSharers);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ctl.rec_full[s], 1);
            mbar_init(&ctl.rec_empty[s], kWarps);
        }
        mbar_init(&ctl.meet, kWarps);
        ctl.abort = 0;
        fence_mbar_init();
    }
    if (tid < M * 2) (&ctl.poison[0][0])[tid] = 0u;
    let_next_start();
    wait_for_previous();
    // tile swizzles assume a 1024-byte aligned base; refuse to run otherwise
    if ((smem_u32(smem) & 1023u) != 0u) {
        if (tid == 0) {
            record_error(a.status, BSA_ERR_DEVICE_BOUNDS);
            a.desc[team * kDesc] = 0;
        }
        return;
    }
    int* tables = reinterpret_cast<int*>(smem);
    const Start st = plan(a, team, tables, tables + BSA_KV_MAX_SEQS + 1, &ctl.start);
    if (tid == 0) a.desc[team * kDesc] = 0;
    if (team >= st.teams || st.total == 0) return;
    fence_async_shared();                   // the plan's tables lay where TMA writes next
    __syncthreads();

    if (warp == kWarps) {
        // ============================================================ producer
        int U = 0, X = 0;
        auto put_record = [&](const Rec& r) -> bool {
            const int slot = X & 1;
            if (X >= 2 && !warp_wait(&ctl.rec_empty[slot], ((X >> 1) - 1) & 1, abort, a.status)) return false;
            if (lane == 0) {
                ctl.rec[slot] = r;
                mbar_arrive(&ctl.rec_full[slot]);
            }
            ++X;
            return true;
        };
        auto begin = [](const Walk&, int) { return true; };
        auto put_tile = [&](int meta, int t, int page, long long row, unsigned have, int at, int box) -> bool {
            const int s = U % C::NS;
            if (U >= C::NS && !warp_wait(&ctl.empty[s], ((U / C::NS) - 1) & 1, abort, a.status)) return false;
            uint8_t* dst = smem + s * C::kStage;
            if (lane == 0) {
                ctl.meta[s] = meta;
                ctl.tile[s] = t;
                mbar_arrive_expect_tx(&ctl.full[s], __popc(have) * box * (FP8 ? 130 : 256));
            }
            __syncwarp();
            if (page >= 0) {
                if (FP8) {
                    bulk_load(dst + at * 64, static_cast<const uint8_t*>(a.k) + row * 64, box * 64, &ctl.full[s]);
                    bulk_load(dst + C::kV + at * 64, static_cast<const uint8_t*>(a.v) + row * 64, box * 64, &ctl.full[s]);
                    bulk_load(dst + 16384 + at, a.ks + row, box, &ctl.full[s]);
                    bulk_load(dst + 16384 + 128 + at, a.vs + row, box, &ctl.full[s]);
                } else {
                    tma_load_2d(dst + at * 128, &tm_k, &ctl.full[s], 0, (int)row);
                    tma_load_2d(dst + C::kV + at * 128, &tm_v, &ctl.full[s], 0, (int)row);
                }
            }
            ++U;
            return true;
        };
        if (produce(a, st, team, 0, lane, put_record, begin, put_tile)) {
            Rec rec = {};
            rec.tiles = -1;
            put_record(rec);
        }
        // every copy has landed before the block's shared memory goes away
        volatile int never = 0;
        for (int u = max(0, U - C::NS); u < U; ++u)
            mbar_wait(&ctl.full[u % C::NS], (u / C::NS) & 1, &never, a.status, 50000000ull);
        return;
    }

    // ================================================================ arithmetic
    float* mo = reinterpret_cast<float*>(smem + C::kMerge);           // [warp][row][64]
    float* mml = mo + kWarps * M * 64;                                // [warp][row][2]
    const int g = lane >> 2, t = lane & 3;
    int U = 0, met = 0;
    auto meet = [&]() -> bool {             // the eight warps; bounded like every wait
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.meet);
        return warp_wait(&ctl.meet, met++ & 1, abort, a.status);
    };
    for (int X = 0;; ++X) {
        if (!warp_wait(&ctl.rec_full[X & 1], (X >> 1) & 1, abort, a.status)) break;
        const Rec& rec = ctl.rec[X & 1];
        const int tiles = rec.tiles;
        if (tiles < 0) break;
        const int nrows = rec.nrows, r0 = rec.r0, row0 = rec.row0, pos0 = rec.pos0, len = rec.len;
        // ---------------------------------------------------------------- Q
        // k-step ks takes the words qf[ks][hh] and qf[ks][NH + hh] of rows 8 hh + g
        uint32_t qf[4][2 * NH];
        float rowf[NH];                     // x = score * rowf (e4m3: times the key's scale)
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
            const int r = hh * 8 + g;
            uint4 c0 = make_uint4(0u, 0u, 0u, 0u), c1 = c0;
            if (r < nrows) {
                const int i = a.by_group.of(r0 + r);
                const __nv_bfloat16* p =
                    a.q + (long long)(row0 + i) * a.q_stride + ((long long)rec.h * a.group + (r0 + r - i * a.group)) * 64;
                const uint4* p4 = reinterpret_cast<const uint4*>(p);
                c0 = p4[2 * t];
                c1 = p4[2 * t + 1];
            }
            uint32_t wds[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            rowf[hh] = kScaleLog2;
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
                rowf[hh] = kScaleLog2 * pow2_of(e);
            }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                qf[ks][hh] = wds[2 * ks];
                qf[ks][NH + hh] = wds[2 * ks + 1];
            }
        }
        float o[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[j][c] = 0.f;
        float m[NH], l[NH];
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
            m[hh] = -INFINITY;
            l[hh] = 0.f;
        }

        if constexpr (!FP8) {
        for (int u = 0; u < tiles; ++u, ++U) {
            const int s = U % C::NS;
            if (!warp_wait(&ctl.full[s], (U / C::NS) & 1, abort, a.status)) return;
            const int meta = ctl.meta[s], kb = ctl.tile[s] * kUnit + warp * 16;
            const bool want = ((meta >> warp) & 1) &&
                              ((meta & kFull) || (kb < rec.hi_max && (kb + 16 > rec.lo_min || kb < a.sink)));
            const bool all = (meta & kFull) || (kb + 16 <= rec.hi_min &&
                                                (kb >= rec.lo_max || kb + 16 <= min(a.sink, rec.lo_min)));
            if (!want) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.empty[s]);
                continue;
            }
            // column x (0 .. 7) of the scores' half jj stands for key jj * 8 + x of the warp's 16
            const uint32_t src = smem_u32(smem + s * C::kStage);
            // ------------------------------------------------------------ scores
            float x[2][4];
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
#pragma unroll
                for (int c = 0; c < 4; ++c) x[jj][c] = 0.f;
                const int r = warp * 16 + jj * 8 + g;
                const uint4 k0 = lds16(src + r * 128 + (((2 * t) ^ (r & 7)) << 4));
                const uint4 k1 = lds16(src + r * 128 + (((2 * t + 1) ^ (r & 7)) << 4));
                const uint32_t kw[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16(x[jj], qf[ks][0], NH == 2 ? qf[ks][NH - 1] : 0u, qf[ks][NH], NH == 2 ? qf[ks][2 * NH - 1] : 0u,
                             kw[2 * ks], kw[2 * ks + 1]);
#pragma unroll
                for (int c = 0; c < 2 * NH; ++c) x[jj][c] *= kScaleLog2;
            }
            // ------------------------------------------------------------ V, and what is seen
            uint32_t vw[4][4];              // 8 values of the lane's four keys
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = warp * 16 + (i >> 1) * 8 + 2 * t + (i & 1);
                const uint4 v = lds16(src + C::kV + r * 128 + ((g ^ (r & 7)) << 4));
                vw[i][0] = v.x;
                vw[i][1] = v.y;
                vw[i][2] = v.z;
                vw[i][3] = v.w;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.empty[s]);
            uint32_t seen = 0xffu;          // bit (jj * 4 + c): x[jj][c] counts
            if (!all) {
                seen = 0u;
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    const int r = hh * 8 + g;
                    int lo = 0, hi = 0;
                    if (r < nrows) visible(a, len, pos0 + a.by_group.of(r0 + r), lo, hi);
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int key = kb + jj * 8 + 2 * t + c;
                            if (key < hi && (key >= lo || key < a.sink)) seen |= 1u << (jj * 4 + 2 * hh + c);
                        }
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
                            int lo, hi;
                            visible(a, len, pos0 + a.by_group.of(r0 + r), lo, hi);
                            if (key < hi && (key >= lo || key < a.sink))
                                atomicOr(&ctl.poison[r][g >> 2], cols << ((g & 3) * 8));
                        }
                    }
                }
#pragma unroll
                for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                    for (int c = 0; c < 2 * NH; ++c)
                        if (!((seen >> (jj * 4 + c)) & 1u)) x[jj][c] = -INFINITY;
            }
            // ------------------------------------------------------------ softmax
            float top[NH];
            bool need = false;
#pragma unroll
            for (int hh = 0; hh < NH; ++hh) {
                top[hh] = fmaxf(fmaxf(x[0][2 * hh], x[0][2 * hh + 1]), fmaxf(x[1][2 * hh], x[1][2 * hh + 1]));
                need |= top[hh] > m[hh] + kRescale;
            }
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    float n = top[hh];
                    n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 1));
                    n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 2));
                    n = fmaxf(n, m[hh]);
                    const float f = m[hh] == -INFINITY ? 0.f : ex2_approx(m[hh] - n);
                    m[hh] = n;
                    l[hh] *= f;
#pragma unroll
                    for (int j8 = 0; j8 < 8; ++j8) {
                        o[j8][2 * hh] *= f;
                        o[j8][2 * hh + 1] *= f;
                    }
                }
            }
            uint32_t pf[2][NH];
#pragma unroll
            for (int hh = 0; hh < NH; ++hh) {
                const float ref = m[hh] == -INFINITY ? 0.f : m[hh];
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const float p0 = ex2_approx(x[jj][2 * hh] - ref), p1 = ex2_approx(x[jj][2 * hh + 1] - ref);
                    l[hh] += p0 + p1;
                    pf[jj][hh] = pack_bf16(p0, p1);
                }
            }
            // ------------------------------------------------------------ O += P V
            const uint32_t p1a = NH == 2 ? pf[0][NH - 1] : 0u, p1b = NH == 2 ? pf[1][NH - 1] : 0u;
#pragma unroll
            for (int j8 = 0; j8 < 8; ++j8) {
                const uint32_t sel = j8 & 1 ? 0x7632u : 0x5410u;
                mma_bf16(o[j8], pf[0][0], p1a, pf[1][0], p1b, __byte_perm(vw[0][j8 >> 1], vw[1][j8 >> 1], sel),
                         __byte_perm(vw[2][j8 >> 1], vw[3][j8 >> 1], sel));
            }
        }
        } else {
        for (int u = 0; u < tiles; ++u, ++U) {
            if ((U & 1) != warp >> 2) continue;   // the other half's tile
            const int s = U % C::NS, sub = warp & 3;
            if (!warp_wait(&ctl.full[s], (U / C::NS) & 1, abort, a.status)) return;
            const int meta = ctl.meta[s], kb = ctl.tile[s] * kUnit + sub * 32;
            const int there = (meta >> (2 * sub)) & 3;   // pages of the two 16-key halves
            const bool want = there != 0 &&
                              ((meta & kFull) || (kb < rec.hi_max && (kb + 32 > rec.lo_min || kb < a.sink)));
            const bool all = (meta & kFull) || (there == 3 && kb + 32 <= rec.hi_min &&
                                                (kb >= rec.lo_max || kb + 32 <= min(a.sink, rec.lo_min)));
            if (!want) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.empty[s]);
                continue;
            }
            // column c of the scores' eighth n stands for key 8 n + c / 2 (c even), 8 n + 4 + (c / 2 ^ 1)
            // (odd): pairs of columns differ in parity and equal columns of a quad lie together
            const uint32_t src = smem_u32(smem + s * C::kStage);
            const int kg = g & 1 ? 4 + ((g >> 1) ^ 1) : g >> 1;   // key of column g
            const int k1 = 4 + (t ^ 1);                           // key of column 2 t + 1; 2 t: t
            // ------------------------------------------------------------ scores
            float x[4][2 * NH];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint4 kw = lds16(src + (sub * 32 + 8 * n + kg) * 64 + t * 16);
                const uint32_t kc[4] = {kw.x, kw.y, kw.z, kw.w};
                float h[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16(h, qf[ks][0], NH == 2 ? qf[ks][NH - 1] : 0u, qf[ks][NH], NH == 2 ? qf[ks][2 * NH - 1] : 0u,
                            half2_of(kc[ks], false), half2_of(kc[ks], true));
#pragma unroll
                for (int c = 0; c < 2 * NH; ++c) x[n][c] = h[c];
            }
            // scales: x takes the K row's as a factor (byte 255 gives inf, and inf - inf makes the score
            // NaN), y = x + the V row's exponent
            float ve[4][2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint4 kb4 = lds16(src + 16384 + sub * 32 + half * 16);
                const uint4 vb4 = lds16(src + 16384 + 128 + sub * 32 + half * 16);
                const uint32_t kw[4] = {kb4.x, kb4.y, kb4.z, kb4.w}, vw[4] = {vb4.x, vb4.y, vb4.z, vb4.w};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int n = 2 * half + i;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t at = c ? t ^ 1 : t;
                        const float ks = __uint_as_float(__byte_perm(kw[2 * i + c], 0u, 0x0444u | at << 12) >> 1);
                        const float zero = ks - ks;
#pragma unroll
                        for (int hh = 0; hh < NH; ++hh) x[n][2 * hh + c] = fmaf(x[n][2 * hh + c], ks * rowf[hh], zero);
                        // 2^23 + byte, as a float
                        ve[n][c] = __uint_as_float(__byte_perm(vw[2 * i + c], 0x4b000000u, 0x7650u | at)) - 8388735.f;
                    }
                }
            }
            // ------------------------------------------------------------ V
            uint2 vc[2][4];                   // codes of d 8 g .. 8 g + 7 for the lane's eight keys
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    vc[half][i] = lds8(src + C::kV + (sub * 32 + half * 16 + (i >> 1) * 8 + (i & 1 ? k1 : t)) * 64 + g * 8);
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.empty[s]);
            // ------------------------------------------------------------ what is seen
            if (!all) {
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    const int r = hh * 8 + g;
                    int lo = 0, hi = 0;
                    if (r < nrows) visible(a, len, pos0 + a.by_group.of(r0 + r), lo, hi);
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int key = kb + 8 * n + (c ? k1 : t);
                            if (!(key < hi && (key >= lo || key < a.sink) && ((there >> (n >> 1)) & 1)))
                                x[n][2 * hh + c] = -INFINITY;
                        }
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
            float top[NH], high = ve[0][0];   // of x per row; of the V exponents
            bool need = false;
#pragma unroll
            for (int n = 0; n < 4; ++n) high = fmaxf(high, fmaxf(ve[n][0], ve[n][1]));
            if (high > 100.f) {               // a V row that stands for NaN (or stale memory that is masked)
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        if (ve[n][c] > 100.f) ve[n][c] = __uint_as_float(0x7fc00000u);
            }
#pragma unroll
            for (int hh = 0; hh < NH; ++hh) {
                top[hh] = fmaxf(x[0][2 * hh], x[0][2 * hh + 1]);
#pragma unroll
                for (int n = 1; n < 4; ++n) top[hh] = fmaxf(top[hh], fmaxf(x[n][2 * hh], x[n][2 * hh + 1]));
                need |= top[hh] > m[hh] + kRescale;
            }
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    float n = top[hh];
                    n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 1));
                    n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 2));
                    n = fmaxf(n, m[hh]);
                    const float f = m[hh] == -INFINITY ? 0.f : ex2_approx(m[hh] - n);
                    m[hh] = n;
                    l[hh] *= f;
#pragma unroll
                    for (int j8 = 0; j8 < 8; ++j8) {
                        o[j8][2 * hh] *= f;
                        o[j8][2 * hh + 1] *= f;
                    }
                }
            }
            uint32_t pf[4][NH];               // w of the lane's two keys of each eighth
            float back[NH];
#pragma unroll
            for (int hh = 0; hh < NH; ++hh) {
                const float ref = m[hh] == -INFINITY ? 0.f : m[hh];
                float y[4][2], yt = -INFINITY, sum = 0.f;
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float xv = x[n][2 * hh + c];
                        sum += ex2_approx(xv - ref);
                        // a masked score stays -infinity, whatever the scale byte holds
                        y[n][c] = all || xv != -INFINITY ? xv + ve[n][c] : -INFINITY;
                        yt = fmaxf(yt, y[n][c]);
                    }
                l[hh] += sum;
                yt = fmaxf(yt, __shfl_xor_sync(0xffffffffu, yt, 1));
                yt = fmaxf(yt, __shfl_xor_sync(0xffffffffu, yt, 2));
                const float base = yt == -INFINITY ? 0.f : yt - 14.f;   // the largest w is 2^14
                back[hh] = ex2_approx(base - ref);
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    pf[n][hh] = pack_half2(ex2_approx(y[n][0] - base), ex2_approx(y[n][1] - base));
            }
            // ------------------------------------------------------------ O += 2^(base - m) w V
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
                            mma_f16(h, pf[2 * half][0], NH == 2 ? pf[2 * half][NH - 1] : 0u, pf[2 * half + 1][0],
                                    NH == 2 ? pf[2 * half + 1][NH - 1] : 0u, half2_of(ab[half], y), half2_of(cd[half], y));
                        const int j8 = 4 * k + 2 * z + y;
#pragma unroll
                        for (int c = 0; c < 2 * NH; ++c) o[j8][c] = fmaf(h[c], back[c >> 1], o[j8][c]);
                    }
                }
        }
        }

        // -------------------------------------------------------------------- the block's warps
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
            l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
            l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
            const int r = warp * M + hh * 8 + g;
            // lane (g, t) holds columns 16 t .. 16 t + 15 of row g: o[j][0] is 16 t + j, o[j][1] 8 further
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j8 = 0; j8 < 8; j8 += 4)
                    *reinterpret_cast<float4*>(mo + r * 64 + 16 * t + 8 * c + j8) =
                        make_float4(o[j8][2 * hh + c], o[j8 + 1][2 * hh + c], o[j8 + 2][2 * hh + c], o[j8 + 3][2 * hh + c]);
            if (t == 0) {
                mml[r * 2] = m[hh];
                mml[r * 2 + 1] = l[hh];
            }
        }
        if (!meet()) return;
        const bool whole = rec.whole;
        float* part = part_at<M>(a, team, rec.run, 0);
        if (tid < M * 16) {
            const int r = tid >> 4, c4 = (tid & 15) * 4;
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, mml[(k * M + r) * 2]);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
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
            const uint32_t bad = ctl.poison[r][c4 >> 5] >> (c4 & 31);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[k] *= inv;
                if ((bad >> k) & 1u) acc[k] = __uint_as_float(0x7fc00000u);
            }
            const float lse = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
            if (r < nrows) {
                if (whole) {
                    const int i = a.by_group.of(r0 + r);
                    const int head = rec.h * a.group + (r0 + r - i * a.group);
                    *reinterpret_cast<uint2*>(a.out + (long long)(row0 + i) * a.out_stride + head * 64 + c4) =
                        make_uint2(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]));
                    if (c4 == 0 && a.lse != nullptr) a.lse[(long long)head * a.rows + row0 + i] = lse;
                } else {
                    *reinterpret_cast<float4*>(part + r * 64 + c4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    if (c4 == 0) part[M * 64 + r] = lse;
                }
            }
        }
        if (!meet()) return;
        if (tid < M * 2) (&ctl.poison[0][0])[tid] = 0u;
        if (lane == 0) mbar_arrive(&ctl.rec_empty[X & 1]);
    }
}

// Joins the partial results of an item that crosses team ends: the team that holds its first
// unit left it in run 1, the following ones in run 0. L = ln sum e^lse, out = sum e^(lse - L) o,
// in an order that only the split decides. One block per 16 rows of a (team, member); 16 threads
// hold a row's columns, and with fewer rows several sets of 16 share a row's pieces.
constexpr int kMergeRows = 16;
template <int M>
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
    const int r0 = (d[4] * a.R + member) * a.mr, rb = blockIdx.y * kMergeRows;
    const int nrows = min(min(a.mr, d[2] * a.group - r0) - rb, kMergeRows);
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
                const float* p = part_at<M>(a, kk, kk == team ? 1 : 0, member) + (rb + r) * 64;
                v[i] = *reinterpret_cast<const float4*>(p + 4 * c);
                e[i] = part_at<M>(a, kk, kk == team ? 1 : 0, member)[M * 64 + rb + r] * 1.4426950408889634f;
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
            if (o.x == -INFINITY) continue;
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

template <bool FP8, int M>
cudaError_t launch_rows(AttnArgs& a, cudaStream_t st) {
    using C = Cfg<FP8, M>;
    auto kern = kv_rows_kernel<FP8, M>;
    const size_t smem = C::kCtl + sizeof(Ctl<M>);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    CUtensorMap k = {}, v = {};
    const uint64_t rows = ((uint64_t)a.c.pages * a.c.kv_heads) << a.c.pshift;
    const uint32_t box = a.c.pshift < 7 ? 1u << a.c.pshift : 128u;
    if (!FP8 && (!make_tile_map(&k, a.k, rows, 64, box, false) || !make_tile_map(&v, a.v, rows, 64, box, false)))
        return cudaErrorInvalidValue;
    return launch_early(kern, dim3(a.max_teams), kThreads, smem, st, k, v, a);
}

}  // namespace

template <int M>
static cudaError_t launch_merge(const AttnArgs& a, cudaStream_t st) {
    return launch_early(kv_merge_kernel<M>, dim3(a.max_teams * a.R, (a.mr + kMergeRows - 1) / kMergeRows), kMergeRows * 16,
                        0, st, a);
}

cudaError_t launch_kv_merge128(const AttnArgs& a, cudaStream_t st) { return launch_merge<128>(a, st); }

cudaError_t launch_kv_rows(AttnArgs& a, bool fp8, bool eight, cudaStream_t st) {
    cudaError_t e;
    a.R = 1;
    a.mr = eight ? 8 : 16;
    a.min_run = 1;
    a.set_divisors();
    if (eight) {
        e = fp8 ? launch_rows<true, 8>(a, st) : launch_rows<false, 8>(a, st);
        return e != cudaSuccess ? e : launch_merge<8>(a, st);
    }
    e = fp8 ? launch_rows<true, 16>(a, st) : launch_rows<false, 16>(a, st);
    return e != cudaSuccess ? e : launch_merge<16>(a, st);
}

}  // namespace bsa
