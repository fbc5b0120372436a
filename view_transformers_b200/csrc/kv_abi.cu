// C ABI of the paged key/value cache: host-side validation and launches.
#include <cstdint>

#include "kv_cache.cuh"

namespace bsa {

cudaError_t launch_kv_copy(const kv::CacheArgs& c, bool fp8, bool read, int rows, const int32_t* cu,
                           const int32_t* first, const void* const src[2], void* const dst[2],
                           uint8_t* const scale[2], long long stride, int32_t* status, cudaStream_t st);
cudaError_t launch_kv_rows(kv::AttnArgs& a, bool fp8, cudaStream_t st);
cudaError_t launch_kv_tc(kv::AttnArgs& a, bool fp8, int max_new, cudaStream_t st);

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int64_t kMost = INT32_MAX;

bsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA; }

// Sizes only; the pointers are checked by the calls that use them.
bsa_status check_sizes(const bsa_kv_cache* c) {
    if (c == nullptr) return BSA_ERR_INVALID_ARG;
    if (c->seqs < 1 || c->heads < 1 || c->kv_heads < 1 || c->heads % c->kv_heads != 0 || c->head_dim < 1 ||
        c->page_tokens < 1 || c->pages < 1 || c->max_pages < 1 ||
        (c->format != BSA_KV_BF16 && c->format != BSA_KV_E4M3))
        return BSA_ERR_INVALID_ARG;
    if (c->head_dim != BSA_HEAD_DIM || c->heads > BSA_MAX_HEADS || c->seqs > BSA_KV_MAX_SEQS || c->page_tokens < 16 ||
        c->page_tokens > 256 || (c->page_tokens & (c->page_tokens - 1)) != 0)
        return BSA_ERR_UNSUPPORTED;
    // pages * kv_heads < 2^38, so the products below stay inside 64 bits. Positions stay below 2^30 (kernels
    // look some thousands ahead of them)
    if ((int64_t)c->pages * c->kv_heads * c->page_tokens > kMost ||
        (int64_t)c->max_pages * c->page_tokens > (int64_t)1 << 30)
        return BSA_ERR_UNSUPPORTED;
    return BSA_OK;
}

bsa_status check_cache(const bsa_kv_cache* c, int32_t rows, kv::CacheArgs* a) {
    const bsa_status s = check_sizes(c);
    if (s != BSA_OK) return s;
    if (rows < 0) return BSA_ERR_INVALID_ARG;
    if ((int64_t)rows * c->heads > kMost / 2) return BSA_ERR_UNSUPPORTED;
    if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v) || !c->page_table || !aligned4(c->page_table) ||
        !c->kv_len || !aligned4(c->kv_len))
        return BSA_ERR_INVALID_ARG;
    if (c->format == BSA_KV_E4M3 &&
        (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale)))
        return BSA_ERR_INVALID_ARG;
    a->seqs = c->seqs;
    a->heads = c->heads;
    a->kv_heads = c->kv_heads;
    a->pshift = __builtin_ctz((unsigned)c->page_tokens);
    a->pages = c->pages;
    a->max_pages = c->max_pages;
    a->table = c->page_table;
    a->kv_len = c->kv_len;
    return BSA_OK;
}

bool bad_stride(int64_t stride, int64_t heads) {
    return stride < heads * BSA_HEAD_DIM || stride % 8 != 0 || stride > (int64_t)1 << 38;
}

// Blocks of the attention kernels: two per SM.
int max_blocks() { return 2 * num_sms(); }
constexpr int kMaxRowsPerBlock = 128;

size_t desc_bytes() { return ((size_t)max_blocks() * kv::kDesc * 4 + 255) / 256 * 256; }

size_t workspace_bytes_needed() {
    return desc_bytes() + (size_t)max_blocks() * 2 * kMaxRowsPerBlock * 65 * 4;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" {

bsa_status bsa_kv_append(const bsa_kv_cache* cache, int32_t rows, const int32_t* cu_new, const void* k,
                         const void* v, int64_t row_stride, int32_t* status_dev, bsa_stream_t stream) {
    kv::CacheArgs c;
    const bsa_status s = check_cache(cache, rows, &c);
    if (s != BSA_OK) return s;
    if (!cu_new || !aligned4(cu_new) || !aligned4(status_dev)) return BSA_ERR_INVALID_ARG;
    if (rows == 0) return BSA_OK;
    if (!k || !v || !aligned16(k) || !aligned16(v) || bad_stride(row_stride, cache->kv_heads))
        return BSA_ERR_INVALID_ARG;
    const void* const src[2] = {k, v};
    void* const dst[2] = {cache->k, cache->v};
    uint8_t* const scale[2] = {cache->k_scale, cache->v_scale};
    return from_cuda(launch_kv_copy(c, cache->format == BSA_KV_E4M3, false, rows, cu_new, nullptr, src, dst, scale,
                                    row_stride, status_dev, reinterpret_cast<cudaStream_t>(stream)));
}

bsa_status bsa_kv_read(const bsa_kv_cache* cache, int32_t rows, const int32_t* cu_rows, const int32_t* first,
                       void* k, void* v, int64_t row_stride, int32_t* status_dev, bsa_stream_t stream) {
    kv::CacheArgs c;
    const bsa_status s = check_cache(cache, rows, &c);
    if (s != BSA_OK) return s;
    if (!cu_rows || !aligned4(cu_rows) || !first || !aligned4(first) || !aligned4(status_dev))
        return BSA_ERR_INVALID_ARG;
    if (rows == 0) return BSA_OK;
    if (!k || !v || !aligned16(k) || !aligned16(v) || bad_stride(row_stride, cache->kv_heads))
        return BSA_ERR_INVALID_ARG;
    const void* const src[2] = {cache->k, cache->v};
    void* const dst[2] = {k, v};
    uint8_t* const scale[2] = {cache->k_scale, cache->v_scale};
    return from_cuda(launch_kv_copy(c, cache->format == BSA_KV_E4M3, true, rows, cu_rows, first, src, dst, scale,
                                    row_stride, status_dev, reinterpret_cast<cudaStream_t>(stream)));
}

bsa_status bsa_kv_workspace_size(const bsa_kv_cache* cache, size_t* bytes) {
    if (bytes == nullptr) return BSA_ERR_INVALID_ARG;
    const bsa_status s = check_sizes(cache);
    if (s != BSA_OK) return s;
    *bytes = workspace_bytes_needed();
    return BSA_OK;
}

bsa_status bsa_kv_attention(const bsa_kv_cache* cache, int32_t rows, int32_t max_new, int32_t unit,
                            int32_t window, int32_t sink, const int32_t* cu_new, const void* q,
                            int64_t q_stride, void* out, int64_t out_stride, float* lse, void* workspace,
                            size_t workspace_bytes, int32_t* status_dev, bsa_stream_t stream) {
    kv::AttnArgs a;
    const bsa_status s = check_cache(cache, rows, &a.c);
    if (s != BSA_OK) return s;
    if (max_new < 0 || unit < 0 || window < 0 || sink < 0 || (window > 0 && unit == 0) || (sink > 0 && window == 0) ||
        !cu_new || !aligned4(cu_new) || !aligned4(status_dev) || !aligned4(lse))
        return BSA_ERR_INVALID_ARG;
    if (rows == 0) return BSA_OK;
    if (!q || !out || !aligned16(q) || !aligned16(out) || bad_stride(q_stride, cache->heads) ||
        bad_stride(out_stride, cache->heads))
        return BSA_ERR_INVALID_ARG;
    if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < workspace_bytes_needed())
        return BSA_ERR_INVALID_ARG;
    a.group = cache->heads / cache->kv_heads;
    a.rows = rows;
    a.unit = unit;
    a.window = window;
    a.sink = sink;
    a.cu = cu_new;
    a.k = cache->k;
    a.v = cache->v;
    a.ks = cache->k_scale;
    a.vs = cache->v_scale;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = q_stride;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.out_stride = out_stride;
    a.lse = lse;
    a.desc = static_cast<int*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + desc_bytes());
    a.status = status_dev;
    a.max_teams = max_blocks();
    // Query rows of a key/value head, at most, choose the kernel: up to 8 (e4m3: 24) the form for few
    // rows, which reads the cache once per 8 of them, else the form for many. Measured (us in
    // a chain of graph nodes; few, many):
    //   bf16  1 stream of 78,200 keys, 16 heads,  8 rows: 73.5, 65.6; 12 rows:  126, 67.6; 24 rows:  180, 67.5
    //         8 streams of 1,000 keys,            8 rows: 15.8, 20.7; 12 rows: 22.1, 20.7; 24 rows: 28.3, 20.9
    //         6 of 95 keys, 4 heads,              8 rows:  6.2, 12.1; 12 rows:  7.3, 12.1; 24 rows:  7.8, 12.1
    //   e4m3  1 stream of 78,200 keys, 16 heads,  8 rows: 48.8,  111; 24 rows:  105,  112; 32 rows:  134,  110
    //         32 streams of 9,000 keys,           8 rows:  133,  392; 24 rows:  366,  393; 32 rows:  481,  389
    //         8 streams of 1,000 keys,            8 rows: 16.4, 28.1; 24 rows: 28.1, 28.3
    // (The lengths are on the device. 16 rows in one of the few rows' instructions, e4m3: 217 us instead of
    // 250 for 16 rows on the 32 streams, 25.6 instead of 21.9 on the 8.)
    const bool fp8 = cache->format == BSA_KV_E4M3;
    const long long per_head = (long long)max_new * a.group;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(per_head > (fp8 ? 24 : 8) ? launch_kv_tc(a, fp8, max_new, st) : launch_kv_rows(a, fp8, st));
}

}  // extern "C"
