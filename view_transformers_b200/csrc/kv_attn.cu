// Attention of new tokens over a paged key/value cache: the form for few query rows per
// key/value head (single tokens, camera and register tokens, grouped heads), and the merge of
// split rows that it shares with the form for many.
//
//   out = sum_j p_j v_j / l, p_j = 2^(x_j - m), x_j = q.k_j log2(e)/8, l = sum_j p_j, over the
//   keys a row sees, with a running reference m that is raised only when some x exceeds it by 8.
//
// With few rows the keys and values are read once and nothing else matters: the bound is HBM
// (128 bytes a row of K or V, 65 in e4m3). So the matrix instruction is the small one, with
// M rows (8 or 16 of its 16), and its operands go from HBM through a ring of asynchronous copies
// straight into the registers that need them:
//   - each warp takes 16 of the 128 keys of a unit and keeps its own m, l and O; the eight warps
//     of a block meet at the end of an item;
//   - a dot product does not care about the order of its terms, so the lane that must hold two
//     neighbouring d of key g takes 16 neighbouring bytes of that key instead, and Q is loaded in
//     the same order; P.V's columns are likewise dealt out so that a lane needs 8 neighbouring d
//     of four keys. Every lane then reads back only what it copied itself: no barrier, no bank
//     conflict, and every copy covers whole 32-byte sectors;
//   - e4m3 codes become f16 by one conversion for Q.K (Q is scaled to f16 per row, exact for
//     elements within 2^-28 of the row's largest) and bf16 by shifting that for P.V, as powers of
//     two away; the rows' scales go into the scores and into P, which bf16 holds without loss.
#include <cfloat>

#include "kv_cache.cuh"
#include "sm100.cuh"

namespace bsa {
namespace {

using namespace kv;
using sm100::ex2_approx;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kScaleLog2 = 0.18033688011112042f;   // log2(e) / sqrt(64)
constexpr float kRescale = 8.0f;
constexpr float kLn2 = 0.69314718055994531f;

template <bool FP8, int M>
struct Cfg {
    static constexpr int kStepBytes = FP8 ? 2048 + 512 : 4096;   // 16 keys of K and V (and scales)
    static constexpr int kStages = FP8 ? (M == 8 ? 4 : 4) : (M == 8 ? 3 : 2);
    static constexpr size_t kRing = (size_t)kWarps * kStages * kStepBytes;
    static constexpr size_t kMerge = (size_t)kWarps * M * 66 * 4;
    static constexpr size_t kSmem = kRing + kMerge;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
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
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
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
// f16 with at most 7 mantissa bits to the bf16 2^-112 times as large: the exponent fields, 15 and
// 127 off, are not converted
__device__ __forceinline__ uint32_t bf16_of(uint32_t h) {
    return ((h >> 3) & 0x0fff0fffu) | (h & 0x80008000u);
}
constexpr uint32_t kVExp = 100;             // P carries 2^100 ...
constexpr float kVBack = 4096.f;            // ... and O 2^(112 - 100) in the end

__device__ __forceinline__ bool has_nonfinite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <bool FP8, int M>
__global__ void __launch_bounds__(kThreads, 2)
kv_rows_kernel(const AttnArgs a) {
    using C = Cfg<FP8, M>;
    constexpr int NH = M / 8;               // 8-row halves in use
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Start start;
    __shared__ uint32_t poison[M][2];       // columns of a row that met a NaN or infinite value
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int team = blockIdx.x;

    if (tid < M * 2) (&poison[0][0])[tid] = 0u;
    let_next_start();
    wait_for_previous();
    int* tables = reinterpret_cast<int*>(smem);
    const Start st = plan(a, team, tables, tables + BSA_KV_MAX_SEQS + 1, &start);
    if (tid == 0) a.desc[team * kDesc] = 0;
    if (team >= st.teams || st.total == 0) return;
    __syncthreads();

    const uint32_t ring = sm100::smem_u32(smem) + warp * (C::kStages * C::kStepBytes);
    float* mo = reinterpret_cast<float*>(smem + C::kRing);            // [warp][row][64]
    float* mml = mo + kWarps * M * 64;                                // [warp][row][2]

    // the loader runs kStages - 1 steps ahead of the arithmetic, across items; lane i holds the
    // page of the unit lbase + i of the loader's segment
    Walk lw(a, st, team);
    bool live = lw.next();
    int lj = live ? lw.j0 : 0, lbase = lj - 32, lpage = -1;
    uint32_t held = 0u;                     // bit s: stage s holds keys
    auto load_step = [&](int stage) {
        bool ok = false;
        if (live) {
            if (lj - lbase >= 32) {
                lbase = lj;
                lpage = -1;
                const int k = unit_of(lw.span, lj + lane) * kUnit + warp * 16;
                if (lj + lane < lw.j1 && k < lw.span.hi_max && (k + 16 > lw.span.lo_min || k < a.sink))
                    lpage = a.c.table[(long long)lw.s * a.c.max_pages + (k >> a.c.pshift)];
                if (lpage >= a.c.pages) {
                    record_error(a.status, BSA_ERR_DEVICE_BOUNDS);
                    lpage = -1;
                }
            }
            const int page = __shfl_sync(0xffffffffu, lpage, lj - lbase);
            ok = page >= 0;
            {
                const int kb = unit_of(lw.span, lj) * kUnit + warp * 16;
                if (ok) {
                    const long long row =
                        (((long long)page * a.c.kv_heads + lw.h) << a.c.pshift) + (kb & ((1 << a.c.pshift) - 1));
                    const uint32_t dst = ring + stage * C::kStepBytes;
                    if (!FP8) {
                        const uint8_t* kp = static_cast<const uint8_t*>(a.k) + row * 128;
                        const uint8_t* vp = static_cast<const uint8_t*>(a.v) + row * 128;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                cp16(dst + (j * 2 + c) * 512 + lane * 16, kp + (j * 8 + g) * 128 + c * 64 + t * 16);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            cp16(dst + 2048 + i * 512 + lane * 16, vp + (2 * t + (i & 1) + (i >> 1) * 8) * 128 + g * 16);
                    } else {
                        const uint8_t* kp = static_cast<const uint8_t*>(a.k) + row * 64;
                        const uint8_t* vp = static_cast<const uint8_t*>(a.v) + row * 64;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            cp16(dst + j * 512 + lane * 16, kp + (j * 8 + g) * 64 + t * 16);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            cp8(dst + 1024 + i * 256 + lane * 8, vp + (2 * t + (i & 1) + (i >> 1) * 8) * 64 + g * 8);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            cp4(dst + 2048 + i * 128 + lane * 4, a.ks + row + i * 8 + (t >> 1) * 4);
                            cp4(dst + 2304 + i * 128 + lane * 4, a.vs + row + i * 8 + (t >> 1) * 4);
                        }
                    }
                }
            }
            if (++lj >= lw.j1) {
                lw.done();
                live = lw.next();
                lj = live ? lw.j0 : 0;
                lbase = lj - 32;
            }
        }
        held = (held & ~(1u << stage)) | ((ok ? 1u : 0u) << stage);
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) load_step(i);

    Walk w(a, st, team);
    int stage = 0;
    while (w.next()) {
        const Seq q = w.q;
        const int nrows = q.n * a.group;
        const int r0 = w.rg * M;            // R = 1, mr = M: a row group is one query tile
        // ---------------------------------------------------------------- Q
        uint32_t qf[4][2 * NH];
        float rowf[NH];                     // x = score * rowf
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
            const int r = r0 + hh * 8 + g;
            uint4 c0 = make_uint4(0u, 0u, 0u, 0u), c1 = c0;
            if (r < nrows) {
                const int i = r / a.group;
                const __nv_bfloat16* p =
                    a.q + (long long)(q.row0 + i) * a.q_stride + ((long long)w.h * a.group + (r - i * a.group)) * 64;
                const uint4* p4 = reinterpret_cast<const uint4*>(p);
                c0 = p4[FP8 ? 2 * t : t];
                c1 = p4[FP8 ? 2 * t + 1 : 4 + t];
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
                    wds[k] = sm100::pack_half2(__uint_as_float(wds[k] << 16) * inv,
                                               __uint_as_float(wds[k] & 0xffff0000u) * inv);
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

        for (int j = w.j0; j < w.j1; ++j) {
            cp_wait<C::kStages - 2>();
            const bool ok = (held >> stage) & 1u;
            const uint32_t src = ring + stage * C::kStepBytes;
            const int kb = unit_of(w.span, j) * kUnit + warp * 16;
            // the stage that the previous step emptied
            load_step(stage == 0 ? C::kStages - 1 : stage - 1);
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
            if (!ok) continue;
            // ------------------------------------------------------------ scores
            float x[2][4];
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
#pragma unroll
                for (int c = 0; c < 4; ++c) x[jj][c] = 0.f;
                if (!FP8) {
                    const uint4 k0 = lds16(src + (jj * 2) * 512 + lane * 16);
                    const uint4 k1 = lds16(src + (jj * 2 + 1) * 512 + lane * 16);
                    const uint32_t kw[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16(x[jj], qf[ks][0], NH == 2 ? qf[ks][NH - 1] : 0u, qf[ks][NH], NH == 2 ? qf[ks][2 * NH - 1] : 0u,
                                 kw[2 * ks], kw[2 * ks + 1]);
                } else {
                    const uint4 k0 = lds16(src + jj * 512 + lane * 16);
                    const uint32_t kw[4] = {k0.x, k0.y, k0.z, k0.w};
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16(x[jj], qf[ks][0], NH == 2 ? qf[ks][NH - 1] : 0u, qf[ks][NH], NH == 2 ? qf[ks][2 * NH - 1] : 0u,
                                half2_of(kw[ks], false), half2_of(kw[ks], true));
                }
            }
            float vsc[2][2];
            if (FP8) {
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const uint32_t kw = lds4(src + 2048 + jj * 128 + lane * 4) >> ((t & 1) * 16);
                    const uint32_t vw = lds4(src + 2304 + jj * 128 + lane * 4) >> ((t & 1) * 16);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float kf = scale_of((kw >> (8 * c)) & 255u);
                        const uint32_t vb = (vw >> (8 * c)) & 255u;
                        vsc[jj][c] = vb >= 155u ? __uint_as_float(0x7fc00000u) : pow2_of(vb + kVExp);
#pragma unroll
                        for (int hh = 0; hh < NH; ++hh) x[jj][2 * hh + c] *= kf * rowf[hh];
                    }
                }
            } else {
#pragma unroll
                for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                    for (int c = 0; c < 2 * NH; ++c) x[jj][c] *= kScaleLog2;
            }
            // ------------------------------------------------------------ V, and what is seen
            uint32_t vw[4][4];              // key i of the lane's four: 8 values (bf16) or codes
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!FP8) {
                    const uint4 v = lds16(src + 2048 + i * 512 + lane * 16);
                    vw[i][0] = v.x;
                    vw[i][1] = v.y;
                    vw[i][2] = v.z;
                    vw[i][3] = v.w;
                } else {
                    const uint2 v = lds8(src + 1024 + i * 256 + lane * 8);
                    vw[i][0] = v.x;
                    vw[i][1] = v.y;
                }
            }
            const Span& sp = w.span;
            const bool all = kb + 16 <= sp.hi_min && (kb >= sp.lo_max || kb + 16 <= min(a.sink, sp.lo_min));
            uint32_t seen = 0xffu;          // bit (jj * 4 + c): x[jj][c] counts
            if (!all) {
                seen = 0u;
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    const int r = r0 + hh * 8 + g;
                    int lo = 0, hi = 0;
                    if (r < nrows) visible(a, q.len, q.len - q.n + r / a.group, lo, hi);
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int key = kb + jj * 8 + 2 * t + c;
                            if (key < hi && (key >= lo || key < a.sink)) seen |= 1u << (jj * 4 + 2 * hh + c);
                        }
                }
                if (!FP8) {
                    // P = 0 does not silence a NaN: rows of V past the end are dropped, and a
                    // non-finite value that only some rows see is kept apart
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = kb + 2 * t + (i & 1) + (i >> 1) * 8;
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
                            for (int r = r0; r < min(r0 + M, nrows); ++r) {
                                int lo, hi;
                                visible(a, q.len, q.len - q.n + r / a.group, lo, hi);
                                if (key < hi && (key >= lo || key < a.sink))
                                    atomicOr(&poison[r - r0][g >> 2], cols << ((g & 3) * 8));
                            }
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
                    float p0 = ex2_approx(x[jj][2 * hh] - ref), p1 = ex2_approx(x[jj][2 * hh + 1] - ref);
                    l[hh] += p0 + p1;
                    if (FP8) {
                        p0 *= vsc[jj][0];
                        p1 *= vsc[jj][1];
                        if (!all) {         // a masked P is 0, whatever the scale byte holds
                            if (!((seen >> (jj * 4 + 2 * hh)) & 1u)) p0 = 0.f;
                            if (!((seen >> (jj * 4 + 2 * hh + 1)) & 1u)) p1 = 0.f;
                        }
                    }
                    pf[jj][hh] = pack_bf16(p0, p1);
                }
            }
            // ------------------------------------------------------------ O += P V
            const uint32_t p1a = NH == 2 ? pf[0][NH - 1] : 0u, p1b = NH == 2 ? pf[1][NH - 1] : 0u;
            if (!FP8) {
#pragma unroll
                for (int j8 = 0; j8 < 8; ++j8) {
                    const uint32_t sel = j8 & 1 ? 0x7632u : 0x5410u;
                    mma_bf16(o[j8], pf[0][0], p1a, pf[1][0], p1b, __byte_perm(vw[0][j8 >> 1], vw[1][j8 >> 1], sel),
                             __byte_perm(vw[2][j8 >> 1], vw[3][j8 >> 1], sel));
                }
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint32_t sel = z ? 0x7362u : 0x5140u;
                        const uint32_t ab = __byte_perm(vw[0][k], vw[1][k], sel);
                        const uint32_t cd = __byte_perm(vw[2][k], vw[3][k], sel);
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            mma_bf16(o[4 * k + 2 * z + y], pf[0][0], p1a, pf[1][0], p1b, bf16_of(half2_of(ab, y)),
                                     bf16_of(half2_of(cd, y)));
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
        __syncthreads();
        const bool whole = w.has_start && w.has_end;
        float* part = part_at<M>(a, team, w.has_start ? 1 : 0, 0);
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
            const float inv = (ll == 0.f ? 0.f : 1.f / ll) * (FP8 ? kVBack : 1.f);
            const uint32_t bad = poison[r][c4 >> 5] >> (c4 & 31);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[k] *= inv;
                if ((bad >> k) & 1u) acc[k] = __uint_as_float(0x7fc00000u);
            }
            const float lse = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
            if (r0 + r < nrows) {
                if (whole) {
                    const int i = (r0 + r) / a.group;
                    const int head = w.h * a.group + (r0 + r - i * a.group);
                    *reinterpret_cast<uint2*>(a.out + (long long)(q.row0 + i) * a.out_stride + head * 64 + c4) =
                        make_uint2(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]));
                    if (c4 == 0 && a.lse != nullptr) a.lse[(long long)head * a.rows + q.row0 + i] = lse;
                } else {
                    *reinterpret_cast<float4*>(part + r * 64 + c4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    if (c4 == 0) part[M * 64 + r] = lse;
                }
            }
        }
        if (tid == 0 && !whole && w.has_start) {   // the merge kernel's record of this item
            int* d = a.desc + team * kDesc;
            d[1] = q.row0;
            d[2] = q.n;
            d[3] = w.h;
            d[4] = w.rg;
            d[5] = st.team_of(w.item + max(1, w.span.count) - 1);
            d[0] = 1;
        }
        __syncthreads();
        if (tid < M * 2) (&poison[0][0])[tid] = 0u;
        w.done();
    }
    cp_wait<0>();
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
    const int i = (r0 + rb + r) / a.group;
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
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_early(kern, dim3(a.max_teams), kThreads, C::kSmem, st, a);
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
    if (eight) {
        e = fp8 ? launch_rows<true, 8>(a, st) : launch_rows<false, 8>(a, st);
        return e != cudaSuccess ? e : launch_merge<8>(a, st);
    }
    e = fp8 ? launch_rows<true, 16>(a, st) : launch_rows<false, 16>(a, st);
    return e != cudaSuccess ? e : launch_merge<16>(a, st);
}

}  // namespace bsa
