// Appending new tokens to the paged key/value cache (bf16 copy, or e4m3 with a power-of-two
// scale per row) and reading cached tokens back. Both move rows of 64 values between packed
// token-major tensors and head-major pages and are bound by HBM: an appended row of K or V costs
// 128 bytes read and 128 (bf16) or 65 (e4m3) written, a row read back the mirror of that.
//
// Eight threads share a row (16 bytes of bf16 each), so a warp reads four rows of 128
// contiguous bytes and writes four of 128 or 64; the maximum of a row is three shuffles. A thread
// works on kRows rows at once: their loads are issued before the first is used.
#include <cuda_fp8.h>

#include "kv_cache.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;

struct CopyArgs {
    kv::CacheArgs c;
    int rows;
    const int32_t* cu;
    const int32_t* first;      // reading only
    const void* src[2];        // K and V: the packed tensors (append) or the pools (read)
    void* dst[2];
    uint8_t* scale[2];
    long long stride;          // elements between packed rows
    int32_t* status;
};

// Sequence of packed row r: cu (shared memory) ascending; -1 when no sequence holds it.
__device__ __forceinline__ int seq_of(const int* cu, int S, int r) {
    int lo = 0, hi = S;        // cu[lo] <= r < cu[hi] if cu is what it should be
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= r) lo = mid; else hi = mid;
    }
    return cu[lo] <= r && r < cu[lo + 1] ? lo : -1;
}

__device__ __forceinline__ void load_cu(const CopyArgs& a, int* cu) {
    for (int s = threadIdx.x; s <= a.c.seqs; s += kThreads) cu[s] = a.cu[s];
    __syncthreads();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int s = threadIdx.x; s < a.c.seqs; s += kThreads)
            if (cu[s] < 0 || cu[s + 1] < cu[s] || cu[s + 1] > a.rows) record_error(a.status, BSA_ERR_DEVICE_BOUNDS);
}

// Row of the pools that holds position pos of sequence s and head h; -1: no page, -2: out of range.
__device__ __forceinline__ long long pool_row(const kv::CacheArgs& c, int s, int pos, int h) {
    if (pos < 0 || (pos >> c.pshift) >= c.max_pages) return -2;
    const int page = c.table[(long long)s * c.max_pages + (pos >> c.pshift)];
    if (page < 0) return -1;
    if (page >= c.pages) return -2;
    return (((long long)page * c.kv_heads + h) << c.pshift) + (pos & ((1 << c.pshift) - 1));
}

// e4m3 pair (lower half of w) to f16x2, exact
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads)
kv_append_kernel(const CopyArgs a) {
    __shared__ int cu[BSA_KV_MAX_SEQS + 1];
    load_cu(a, cu);
    const int Hk = a.c.kv_heads, which = blockIdx.y;
    const int sub = threadIdx.x & 7;
    const long long total = (long long)a.rows * Hk;
    const uint4* src = static_cast<const uint4*>(a.src[which]);
    for (long long base = (long long)blockIdx.x * (kThreads / 8 * kRows); base < total;
         base += (long long)gridDim.x * (kThreads / 8 * kRows)) {
        uint4 x[kRows];
        int r[kRows], h[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const long long at = base + i * (kThreads / 8) + (threadIdx.x >> 3);
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            r[i] = -1;
            h[i] = 0;
            if (at < total) {
                r[i] = (int)((unsigned)at / (unsigned)Hk);
                h[i] = (int)at - r[i] * Hk;
                x[i] = __ldg(src + ((long long)r[i] * a.stride + h[i] * 64) / 8 + sub);
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int s = r[i] < 0 ? -1 : seq_of(cu, a.c.seqs, r[i]);
            long long row = -1;
            if (s >= 0) {
                const int pos = a.c.kv_len[s] - (cu[s + 1] - cu[s]) + (r[i] - cu[s]);
                row = pool_row(a.c, s, pos, h[i]);
                if (row < 0 && sub == 0) record_error(a.status, BSA_ERR_DEVICE_BOUNDS);
            }
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            bool bad = false;
            if (!FP8) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    bad |= (w[k] & 0x7f80u) == 0x7f80u || (w[k] & 0x7f800000u) == 0x7f800000u;
                if (row >= 0) static_cast<uint4*>(a.dst[which])[row * 8 + sub] = x[i];
            } else {
                float f[8], top = 0.f;
                bool naan = false;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[2 * k] = __uint_as_float(w[k] << 16);
                    f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float m = fabsf(f[k]);
                    naan |= !(m <= 3.4e38f);            // infinite or NaN
                    top = fmaxf(top, m);
                }
                if (naan) top = __uint_as_float(0x7f800000u);
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                naan = top > 3.4e38f;                   // anywhere in the row
                bad = top > 14680064.f;
                // top = m 2^x with 0.5 <= m < 1 and 448 = 0.875 2^9: e = x - 9, or one more
                // when m > 0.875 (mantissa field above 0x600000)
                const uint32_t bits = __float_as_uint(top);
                int e = (int)(bits >> 23) - 126 - 9 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
                e = min(max(e, BSA_KV_EXP_MIN), BSA_KV_EXP_MAX);
                const float inv = kv::pow2_of(127 - e);
                uint32_t code[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // the conversion saturates to 448
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * k] * inv, f[4 * k + 1] * inv),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * k + 2] * inv, f[4 * k + 3] * inv),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    code[k] = naan ? 0u : lo | (hi << 16);
                }
                if (row >= 0) {
                    static_cast<uint2*>(a.dst[which])[row * 8 + sub] = make_uint2(code[0], code[1]);
                    if (sub == 0) a.scale[which][row] = (uint8_t)(naan ? 255 : e + 127);
                }
            }
            if (bad && row >= 0) record_error(a.status, BSA_ERR_RANGE);
        }
    }
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(const CopyArgs a) {
    __shared__ int cu[BSA_KV_MAX_SEQS + 1];
    load_cu(a, cu);
    const int Hk = a.c.kv_heads, which = blockIdx.y;
    const int sub = threadIdx.x & 7;
    const long long total = (long long)a.rows * Hk;
    for (long long base = (long long)blockIdx.x * (kThreads / 8 * kRows); base < total;
         base += (long long)gridDim.x * (kThreads / 8 * kRows)) {
        long long row[kRows];
        int r[kRows], h[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const long long at = base + i * (kThreads / 8) + (threadIdx.x >> 3);
            r[i] = -1;
            row[i] = -1;
            if (at < total) {
                const int t = (int)((unsigned)at / (unsigned)Hk);
                h[i] = (int)at - t * Hk;
                const int s = seq_of(cu, a.c.seqs, t);
                if (s >= 0) {
                    r[i] = t;
                    const int pos = a.first[s] + (t - cu[s]);
                    row[i] = pos < a.c.kv_len[s] ? pool_row(a.c, s, pos, h[i]) : -2;
                    if (row[i] == -2 && sub == 0) record_error(a.status, BSA_ERR_DEVICE_BOUNDS);
                }
            }
        }
        uint4 x[kRows];
        uint32_t e[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            e[i] = 127u;
            if (row[i] >= 0) {
                if (FP8) {
                    const uint2 c = __ldg(static_cast<const uint2*>(a.src[which]) + row[i] * 8 + sub);
                    x[i].x = c.x;
                    x[i].y = c.y;
                    e[i] = a.scale[which][row[i]];
                } else {
                    x[i] = __ldg(static_cast<const uint4*>(a.src[which]) + row[i] * 8 + sub);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (r[i] < 0) continue;
            if (FP8) {
                const float f = kv::scale_of(e[i]);
                const uint32_t c[2] = {x[i].x, x[i].y};
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t p = e4m3_to_half2(k & 1 ? c[k >> 1] >> 16 : c[k >> 1]);
                    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&p));
                    o[k] = kv::pack_bf16(v.x * f, v.y * f);   // exact: 4 significant bits times a power of two
                }
                x[i] = make_uint4(o[0], o[1], o[2], o[3]);
            }
            static_cast<uint4*>(a.dst[which])[((long long)r[i] * a.stride + h[i] * 64) / 8 + sub] = x[i];
        }
    }
}

}  // namespace

cudaError_t launch_kv_copy(const kv::CacheArgs& c, bool fp8, bool read, int rows, const int32_t* cu,
                           const int32_t* first, const void* const src[2], void* const dst[2],
                           uint8_t* const scale[2], long long stride, int32_t* status, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    CopyArgs a;
    a.c = c;
    a.rows = rows;
    a.cu = cu;
    a.first = first;
    for (int i = 0; i < 2; ++i) {
        a.src[i] = src[i];
        a.dst[i] = dst[i];
        a.scale[i] = scale[i];
    }
    a.stride = stride;
    a.status = status;
    const long long blocks = ((long long)rows * c.kv_heads + kThreads / 8 * kRows - 1) / (kThreads / 8 * kRows);
    const dim3 grid((unsigned)(blocks < num_sms() * 16 ? blocks : num_sms() * 16), 2);
    if (read) {
        if (fp8) kv_read_kernel<true><<<grid, kThreads, 0, st>>>(a);
        else kv_read_kernel<false><<<grid, kThreads, 0, st>>>(a);
    } else {
        if (fp8) kv_append_kernel<true><<<grid, kThreads, 0, st>>>(a);
        else kv_append_kernel<false><<<grid, kThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace bsa
