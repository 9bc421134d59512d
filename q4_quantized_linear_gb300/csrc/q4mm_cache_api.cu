// q4mm_cache_api.cu -- the C entry points of the paged cache, the attention over
// it, the probabilities and the verification of drafted tokens (declared in
// include/q4mm.h): argument checks, and which kernel takes a call.
#include <algorithm>
#include <cmath>

#include "../../include/q4mm.h"
#include "q4mm_cache.h"

namespace q4 {
namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;     // rows x heads
constexpr int64_t kMaxPageTokens = 1024;
constexpr int64_t kMaxTokens = int64_t(1) << 30;   // of a sequence
constexpr int64_t kMaxVocab = int64_t(1) << 24;
constexpr float kLog2e = 1.4426950408889634f;
constexpr size_t kMetaBytes = 2 * sizeof(int4) * kAttnMaxCtas;

cudaStream_t as_stream(q4mm_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

bool valid_page(int64_t page_tokens, int64_t kv_heads, int64_t d, int ctype)
{
    return page_tokens >= 16 && page_tokens <= kMaxPageTokens && (page_tokens & (page_tokens - 1)) == 0 && kv_heads >= 1 &&
           kv_heads <= 4096 && d >= 8 && d <= kMaxHeadDim && d % 8 == 0 &&
           (ctype == Q4_TYPE_F16 || ctype == Q4_TYPE_BF16 || ctype == Q4_TYPE_I8);
}
// A matrix of `cols` columns on its elements' boundaries.
int check_matrix(const void *p, int64_t ld, int64_t cols, int type)
{
    if (!p || ld < cols || ld > (int64_t(1) << 40)) return Q4_ERR_INVALID_ARG;
    return aligned_to(p, static_cast<uintptr_t>(type_size(type))) ? Q4_OK : Q4_ERR_ALIGNMENT;
}
int check_array(const void *p, uintptr_t align, bool optional = false)
{
    if (!p) return optional ? Q4_OK : Q4_ERR_INVALID_ARG;
    return aligned_to(p, align) ? Q4_OK : Q4_ERR_ALIGNMENT;
}
int first_fault(std::initializer_list<int> codes)
{
    for (int c : codes)
        if (c != Q4_OK) return c;
    return Q4_OK;
}

int make_cache(KvCache *c, const void *pages, int64_t n_pages, int64_t page_tokens, int64_t kv_heads, int64_t d, int ctype,
               const int32_t *table, int64_t ldt)
{
    if (!valid_page(page_tokens, kv_heads, d, ctype) || n_pages < 1 || n_pages > 0x7FFFFFFF || ldt < 1 || ldt > kMaxTokens)
        return Q4_ERR_INVALID_ARG;
    const int rc = first_fault({check_array(pages, 16), check_array(table, 4)});
    if (rc != Q4_OK) return rc;
    c->pages = static_cast<uint8_t *>(const_cast<void *>(pages));
    c->head_bytes = kv_head_bytes(page_tokens, d, ctype);
    c->page_bytes = static_cast<int64_t>(c->head_bytes) * kv_heads;
    c->n_pages = static_cast<int>(n_pages);
    c->page_tokens = static_cast<int>(page_tokens);
    c->log_page = log2_of(page_tokens);
    c->heads = static_cast<int>(kv_heads);
    c->d = static_cast<int>(d);
    c->chunks = static_cast<int>(ceil_div(d, kChunk));
    c->type = ctype;
    c->table = table;
    c->ldt = ldt;
    c->capacity = static_cast<int>(std::min(ldt * page_tokens, kMaxTokens));
    return Q4_OK;
}

bool valid_batch(int64_t n_seq, int64_t rows, int64_t heads)
{
    return n_seq >= 0 && n_seq <= kMaxSeqs && rows >= 0 && heads >= 1 && rows <= kMaxRows / heads;
}

int kv_rows(bool write, const void *K, int64_t ldk, const void *V, int64_t ldv, int type, const void *pages, int64_t n_pages,
            int64_t page_tokens, int64_t kv_heads, int64_t d, int ctype, const int32_t *table, int64_t ldt, const int32_t *at,
            const int32_t *starts, int64_t n_seq, int64_t rows, cudaStream_t s)
{
    if (!is_float_type(type) || !valid_page(page_tokens, kv_heads, d, ctype) || !valid_batch(n_seq, rows, kv_heads))
        return Q4_ERR_INVALID_ARG;
    if (n_seq == 0 || rows == 0) return Q4_OK;
    KvRowsArgs a{};
    int rc = make_cache(&a.c, pages, n_pages, page_tokens, kv_heads, d, ctype, table, ldt);
    if (rc == Q4_OK)
        rc = first_fault({check_array(at, 4, !write), check_array(starts, 4), check_matrix(K, ldk, kv_heads * d, type),
                          check_matrix(V, ldv, kv_heads * d, type)});
    if (rc != Q4_OK) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    const int size = type_size(type);
    RowAlign al;
    al.add(K, ldk * size);
    al.add(V, ldv * size);
    a.K = const_cast<void *>(K), a.V = const_cast<void *>(V);
    a.ldk = ldk, a.ldv = ldv;
    a.at = at, a.starts = starts;
    a.n_seq = static_cast<int>(n_seq), a.rows = rows;
    a.status = dev.status;
    const bool vec = al.bytes() == 16;   // a head's values then start on 16 bytes too: d is a multiple of 8
    return guarded([&] {
        return cuda_status(write ? launch_kv_write(a, type, vec, dev.sm_count, s) : launch_kv_read(a, type, vec, dev.sm_count, s));
    });
}

// Whether the tcgen05 kernel has a part in a call with up to so many query rows of
// a sequence and head: with its two halves tensor memory holds the sums of heads of up to
// 128 dims.
bool tensor_takes(int64_t rows, int chunks) { return rows > kWarpRows && chunks <= 2; }

int block_of(int64_t rows)
{
    return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

} // namespace
} // namespace q4

using namespace q4;

extern "C" {

Q4MM_API size_t q4_kv_page_size(int64_t page_tokens, int64_t kv_heads, int64_t d, int ctype)
{
    if (!valid_page(page_tokens, kv_heads, d, ctype)) return 0;
    return static_cast<size_t>(kv_head_bytes(page_tokens, d, ctype)) * static_cast<size_t>(kv_heads);
}

Q4MM_API int q4_kv_write(void *pages, int64_t n_pages, int64_t page_tokens, int64_t kv_heads, int64_t d, int ctype,
                         const int32_t *table, int64_t ldt, const int32_t *lens, const int32_t *starts, int64_t n_seq,
                         const void *K, int64_t ldk, const void *V, int64_t ldv, int type, int64_t rows,
                         q4mm_stream_t stream)
{
    return kv_rows(true, K, ldk, V, ldv, type, pages, n_pages, page_tokens, kv_heads, d, ctype, table, ldt, lens, starts, n_seq,
                   rows, as_stream(stream));
}

Q4MM_API int q4_kv_read(void *K, int64_t ldk, void *V, int64_t ldv, int type, const void *pages, int64_t n_pages,
                        int64_t page_tokens, int64_t kv_heads, int64_t d, int ctype, const int32_t *table, int64_t ldt,
                        const int32_t *first, const int32_t *starts, int64_t n_seq, int64_t rows, q4mm_stream_t stream)
{
    return kv_rows(false, K, ldk, V, ldv, type, pages, n_pages, page_tokens, kv_heads, d, ctype, table, ldt, first, starts, n_seq,
                   rows, as_stream(stream));
}

Q4MM_API size_t q4_attention_workspace_size(int64_t rows, int64_t n_seq, int64_t heads, int64_t kv_heads, int64_t d)
{
    if (kv_heads < 1 || heads < 1 || heads % kv_heads != 0 || d < 8 || d > kMaxHeadDim || d % 8 != 0 ||
        !valid_batch(n_seq, rows, heads) || rows == 0 || n_seq == 0)
        return 0;
    const int64_t group = heads / kv_heads;
    const int chunks = static_cast<int>(ceil_div(d, kChunk));
    int64_t parts = 2 * kAttnMaxCtas * attn_part_floats(block_of(rows * group), chunks);
    if (tensor_takes(rows * group, chunks)) parts = std::max(parts, 2 * kTensorMaxCtas * attn_part_floats(kTensorRows, chunks));
    return kMetaBytes + sizeof(float) * static_cast<size_t>(parts);
}

Q4MM_API int q4_attention(void *O, int64_t ldo, const void *Q, int64_t ldq, int type, int64_t heads, float scale,
                          int64_t window, const void *pages, int64_t n_pages, int64_t page_tokens, int64_t kv_heads,
                          int64_t d, int ctype, const int32_t *table, int64_t ldt, const int32_t *lens,
                          const int32_t *starts, int64_t n_seq, int64_t rows, int64_t max_new, void *workspace,
                          size_t workspace_bytes, q4mm_stream_t stream)
{
    if (!is_float_type(type) || !valid_page(page_tokens, kv_heads, d, ctype) || heads < 1 || heads % kv_heads != 0 ||
        !valid_batch(n_seq, rows, heads) || window < 0 || max_new < 0 || !(scale > 0.0f) || !std::isfinite(scale * kLog2e))
        return Q4_ERR_INVALID_ARG;
    // the tensor cores multiply numbers of one type
    if ((ctype == Q4_TYPE_BF16 && type != Q4_TYPE_BF16) || (ctype == Q4_TYPE_F16 && type == Q4_TYPE_BF16)) return Q4_ERR_INVALID_ARG;
    if (n_seq == 0 || rows == 0) return Q4_OK;
    AttnArgs a{};
    int rc = make_cache(&a.c, pages, n_pages, page_tokens, kv_heads, d, ctype, table, ldt);
    if (rc == Q4_OK)
        rc = first_fault({check_array(lens, 4), check_array(starts, 4), check_matrix(O, ldo, heads * d, type),
                          check_matrix(Q, ldq, heads * d, type), check_array(workspace, 256, true)});
    if (rc != Q4_OK) return rc;
    if (!workspace || workspace_bytes < q4_attention_workspace_size(rows, n_seq, heads, kv_heads, d)) return Q4_ERR_WORKSPACE;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    const int size = type_size(type);
    RowAlign al;
    al.add(O, ldo * size);
    al.add(Q, ldq * size);
    a.O = O, a.Q = Q;
    a.ldo = ldo, a.ldq = ldq;
    a.type = type, a.vec = al.bytes() == 16;
    a.group = static_cast<int>(heads / kv_heads);
    a.scale_log2 = scale * kLog2e;   // (scores in powers of two)
    a.window = window < 0x7FFFFFFF ? static_cast<int>(window) : 0;   // (a len is below 2^31)
    a.lens = lens, a.starts = starts;
    a.n_seq = static_cast<int>(n_seq), a.rows = static_cast<int>(rows);
    a.meta = static_cast<int4 *>(workspace);
    a.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kMetaBytes);
    a.status = dev.status, a.wait_ns = wait_limit();
    const int64_t most = (max_new > 0 ? std::min(max_new, rows) : rows) * a.group;   // query rows of a sequence and head
    a.rows_above = 0, a.rows_upto = 0x7FFFFFFF;
    a.block = block_of(most);
    cudaStream_t s = as_stream(stream);
    return guarded([&] {
        if (type != Q4_TYPE_F32 && tensor_takes(most, a.c.chunks)) {
            // sequences with many new tokens; all of them where those are the rule by the size of
            // the buffers. Without this the second pair of launches took 8 of 84 us of four prompts
            // that had no use for it. What it costs where a batch has both (32 heads on 8 of 128,
            // single tokens over 8192; the two parts in calls of their own): 4 prompts of 2000 and 4
            // tokens, bf16 cache, 240 us (211 + 32), int8 543 (472 + 27); 8 prompts of 540 and 24
            // tokens 282 (79 + 125) and 682 (173 + 84).
            const bool alone = rows * a.group >= n_seq * 8 * kWarpRows || n_seq == 1;
            AttnArgs many = a;
            many.rows_above = alone ? 0 : kWarpRows;
            const cudaError_t e = launch_attn_tensor(many, dev.sm_count, s);
            if (e != cudaSuccess || alone) return cuda_status(e);
            a.rows_upto = kWarpRows;
        }
        return cuda_status(launch_attn_warp(a, dev.sm_count, s));
    });
}

Q4MM_API int q4_token_probs(float *P, int64_t ldp, const void *logits, int64_t ldl, int type, const float *temperature,
                            int64_t rows, int64_t n, q4mm_stream_t stream)
{
    if (!is_float_type(type) || rows < 0 || rows > (int64_t(1) << 27) || n < 1 || n > kMaxVocab) return Q4_ERR_INVALID_ARG;
    if (rows == 0) return Q4_OK;
    int rc = first_fault({check_matrix(P, ldp, n, Q4_TYPE_F32), check_matrix(logits, ldl, n, type), check_array(temperature, 4, true)});
    if (rc != Q4_OK) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    const ProbsArgs a{P, logits, ldp, ldl, temperature, rows, n, dev.status, wait_limit()};
    return guarded([&] { return cuda_status(launch_token_probs(a, type, dev.sm_count, as_stream(stream))); });
}

Q4MM_API int q4_draft_verify(int32_t *tokens, int64_t ldt, int32_t *kept, const float *P, int64_t ldp, const float *Q,
                             int64_t ldq, const int32_t *drafted, int64_t ldd, const int32_t *counts, const float *accept,
                             int64_t lda, const float *sample, int64_t n_seq, int64_t max_draft, int64_t n,
                             q4mm_stream_t stream)
{
    if (n_seq < 0 || n_seq > (int64_t(1) << 24) || max_draft < 0 || max_draft > 1024 || n < 1 || n > kMaxVerifyVocab)
        return Q4_ERR_INVALID_ARG;
    if (n_seq == 0) return Q4_OK;
    int rc = first_fault({check_matrix(tokens, ldt, max_draft + 1, Q4_TYPE_F32), check_array(kept, 4), check_matrix(P, ldp, n, Q4_TYPE_F32),
                          check_array(sample, 4), check_array(counts, 4, true)});
    if (rc == Q4_OK && max_draft > 0)
        rc = first_fault({check_matrix(drafted, ldd, max_draft, Q4_TYPE_F32), check_matrix(accept, lda, max_draft, Q4_TYPE_F32),
                          Q ? check_matrix(Q, ldq, n, Q4_TYPE_F32) : Q4_OK});
    if (rc != Q4_OK) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    VerifyArgs a{};
    a.tokens = tokens, a.kept = kept;
    a.P = P, a.Q = max_draft > 0 ? Q : nullptr;
    a.ldt = ldt, a.ldp = ldp, a.ldq = ldq;
    a.drafted = drafted, a.counts = counts, a.ldd = ldd;
    a.accept = accept, a.sample = sample, a.lda = lda;
    a.n_seq = n_seq, a.n = n, a.max_draft = static_cast<int>(max_draft);
    return guarded([&] { return cuda_status(launch_draft_verify(a, dev.sm_count, as_stream(stream))); });
}

} // extern "C"
