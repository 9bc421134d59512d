// q4mm_block_api.cu -- the C entry points of what stands around the linear
// layers (declared in include/q4mm.h): argument checks, the access width that
// a call's addresses allow, and the launches of the norms and of the expert
// sort. (The int8 product's are in q4mm_w8a8.cu.)
#include <algorithm>
#include <cmath>

#include "../../include/q4mm.h"
#include "q4mm_internal.h"
#include "q4mm_moe.h"
#include "q4mm_norm.h"

namespace q4 {
namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxCols = int64_t(1) << 24;
constexpr int64_t kMaxPairs = int64_t(1) << 24;

cudaStream_t as_stream(q4mm_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// A matrix argument: a pointer, rows at least `cols` apart, on its elements'
// boundaries. rc keeps the first fault. Of a call without rows, what holds
// something for each row may have no address: an empty tensor has none.
struct Checker {
    bool rows;
    int rc = Q4_OK;
    explicit Checker(int64_t m) : rows(m > 0) {}
    void fail(int code)
    {
        if (rc == Q4_OK) rc = code;
    }
    void matrix(const void *p, int64_t ld, int64_t cols, int type, bool optional = false)
    {
        if (!p) {
            if (!optional && rows) fail(Q4_ERR_INVALID_ARG);
            return;
        }
        if (ld < cols || ld > (int64_t(1) << 40)) fail(Q4_ERR_INVALID_ARG);
        else if (!aligned_to(p, static_cast<uintptr_t>(type_size(type)))) fail(Q4_ERR_ALIGNMENT);
    }
    void vector(const void *p, uintptr_t align, bool optional = false)
    {
        if (!p) {
            if (!optional) fail(Q4_ERR_INVALID_ARG);
        } else if (!aligned_to(p, align)) {
            fail(Q4_ERR_ALIGNMENT);
        }
    }
    // one element or more for each row
    void per_row(const void *p, uintptr_t align) { vector(p, align, !rows); }
};

// Elements of one access of combine and its gradient: 16 bytes where every row
// starts on them, else one (16-bit rows then go by shifted words).
int vec_of(const RowAlign &a, int type) { return a.bytes() == 16 ? 16 / type_size(type) : 1; }

// 16 bytes where the rows of every float matrix (a), the codes (one byte an
// element) and the fp32 parameters beside them start at a vector of theirs, or
// where the float rows all start alike, as rows of one length and stride do; else
// an element (join 4000 x 4097 bf16: 90 us by elements, 36 by the words inside).
RowAccess access_of(const RowAlign &a, int type, const RowAlign *codes = nullptr, const RowAlign *params = nullptr)
{
    const int V = 16 / type_size(type);
    if (a.bytes() == 16 && (!codes || codes->bytes() >= V) && (!params || params->bytes() == 16)) return {V, false};
    return a.alike ? RowAccess{V, true} : RowAccess{1, false};
}

bool valid_gate(int kind) { return kind >= Q4_GATE_NONE && kind <= Q4_GATE_FULL; }
bool positive(float eps) { return eps > 0.0f && std::isfinite(eps); }

void check_gate(Checker &c, const void *gate, int64_t ldg, int kind, int64_t d, int type)
{
    if (!valid_gate(kind)) c.fail(Q4_ERR_INVALID_ARG);
    else if (kind == Q4_GATE_FULL) c.matrix(gate, ldg, d, type);
    else if (kind == Q4_GATE_TOKEN) c.per_row(gate, 4);
    else if (kind == Q4_GATE_CHANNEL) c.vector(gate, 4);
}

int norm_after_impl(void *Y, int64_t ldy, void *H, int64_t ldh, int htype, float *h_scale, bool next, const void *R,
                    int64_t ldr, const void *B, int64_t ldb, int type, const float *w, float w_offset,
                    const void *gate, int64_t ldg, int gate_kind, float scale, const float *w_next,
                    float w_offset_next, float eps, int64_t m, int64_t d, cudaStream_t s)
{
    if (!is_float_type(type) || m < 0 || m > kMaxRows || d < 1 || d > kMaxCols || !positive(eps)) return Q4_ERR_INVALID_ARG;
    if (next && htype != type && htype != Q4_TYPE_I8) return Q4_ERR_INVALID_ARG;
    const bool codes = next && htype == Q4_TYPE_I8;
    Checker c(m);
    c.matrix(Y, ldy, d, type);
    c.matrix(R, ldr, d, type);
    c.matrix(B, ldb, d, type);
    c.vector(w, 4, true);
    check_gate(c, gate, ldg, gate_kind, d, type);
    if (next) {
        c.matrix(H, ldh, d, htype);
        c.vector(w_next, 4, true);
        if (codes) c.per_row(h_scale, 4);
    }
    if (c.rc != Q4_OK) return c.rc;
    if (m == 0) return Q4_OK;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    const int size = type_size(type);
    RowAlign al, ca, pa;
    al.add(Y, ldy * size);
    al.add(R, ldr * size);
    al.add(B, ldb * size);
    if (gate_kind == Q4_GATE_FULL) al.add(gate, ldg * size);
    if (next && !codes) al.add(H, ldh * size);
    if (codes) ca.add(H, ldh);
    pa.add(w, 0);
    pa.add(next ? w_next : nullptr, 0);
    if (gate_kind == Q4_GATE_CHANNEL) pa.add(gate, 0);
    NormAfterArgs a{};
    a.Y = Y, a.R = R, a.B = B;
    a.ldy = ldy, a.ldr = ldr, a.ldb = ldb;
    a.w = w, a.w_off = w_offset;
    a.gate = gate, a.ldg = ldg, a.gate_kind = gate_kind;
    a.scale = scale, a.eps = eps, a.out_eps = eps;
    a.m = m, a.d = d;
    a.status = dev.status, a.wait_ns = wait_limit();
    if (next) a.out = NormOut{H, ldh, codes ? 1 : 0, h_scale, w_next, w_offset_next};
    return guarded([&] { return cuda_status(launch_norm_after(a, type, access_of(al, type, codes ? &ca : nullptr, &pa), dev.sm_count, s)); });
}

} // namespace

// The coding of tokens alone is the norm's kernel without the norm.
int quantize_rows(int8_t *Xq, int64_t ldq, float *sx, const void *X, int64_t ldx, int type, int64_t m, int64_t k,
                  int sm_count, cudaStream_t s)
{
    RowAlign al, ca;
    al.add(X, ldx * type_size(type));
    ca.add(Xq, ldq);
    NormBeforeArgs a{};
    a.out = NormOut{Xq, ldq, 1, sx, nullptr, 0.0f};
    a.X = X, a.ldx = ldx, a.plain = 1;
    a.m = m, a.d = k;
    return guarded([&] { return cuda_status(launch_norm_before(a, type, access_of(al, type, &ca), sm_count, s)); });
}

} // namespace q4

using namespace q4;

extern "C" {

Q4MM_API int q4_a8_quantize(int8_t *Xq, float *sx, const void *X, int64_t ldx, int type, int64_t m, int64_t k,
                            q4mm_stream_t stream)
{
    if (!is_float_type(type) || m < 0 || m > kMaxRows || k < 1 || k > kMaxCols) return Q4_ERR_INVALID_ARG;
    Checker c(m);
    c.per_row(Xq, 1);
    c.per_row(sx, 4);
    c.matrix(X, ldx, k, type);
    if (c.rc != Q4_OK) return c.rc;
    if (m == 0) return Q4_OK;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    return quantize_rows(Xq, k, sx, X, ldx, type, m, k, dev.sm_count, as_stream(stream));
}

Q4MM_API int q4_norm_before(void *H, int64_t ldh, int htype, float *h_scale, const void *X, int64_t ldx, int type,
                            const float *w, float w_offset, float eps, int64_t m, int64_t d, q4mm_stream_t stream)
{
    if (!is_float_type(type) || (htype != type && htype != Q4_TYPE_I8) || m < 0 || m > kMaxRows || d < 1 ||
        d > kMaxCols || !positive(eps))
        return Q4_ERR_INVALID_ARG;
    const bool codes = htype == Q4_TYPE_I8;
    Checker c(m);
    c.matrix(H, ldh, d, htype);
    c.matrix(X, ldx, d, type);
    c.vector(w, 4, true);
    if (codes) c.per_row(h_scale, 4);
    if (c.rc != Q4_OK) return c.rc;
    if (m == 0) return Q4_OK;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    const int size = type_size(type);
    RowAlign al, ca, pa;
    al.add(X, ldx * size);
    if (codes) ca.add(H, ldh);
    else al.add(H, ldh * size);
    pa.add(w, 0);
    NormBeforeArgs a{};
    a.out = NormOut{H, ldh, codes ? 1 : 0, h_scale, w, w_offset};
    a.X = X, a.ldx = ldx, a.eps = eps;
    a.m = m, a.d = d;
    return guarded([&] { return cuda_status(launch_norm_before(a, type, access_of(al, type, codes ? &ca : nullptr, &pa), dev.sm_count,
                                          as_stream(stream))); });
}

Q4MM_API int q4_norm_after(void *Y, int64_t ldy, const void *R, int64_t ldr, const void *B, int64_t ldb, int type,
                           const float *w, float w_offset, const void *gate, int64_t ldg, int gate_kind, float scale,
                           float eps, int64_t m, int64_t d, q4mm_stream_t stream)
{
    return norm_after_impl(Y, ldy, nullptr, 0, type, nullptr, false, R, ldr, B, ldb, type, w, w_offset, gate, ldg,
                           gate_kind, scale, nullptr, 0.0f, eps, m, d, as_stream(stream));
}

Q4MM_API int q4_norm_after_before(void *Y, int64_t ldy, void *H, int64_t ldh, int htype, float *h_scale,
                                  const void *R, int64_t ldr, const void *B, int64_t ldb, int type, const float *w,
                                  float w_offset, const void *gate, int64_t ldg, int gate_kind, float scale,
                                  const float *w_next, float w_offset_next, float eps, int64_t m, int64_t d,
                                  q4mm_stream_t stream)
{
    return norm_after_impl(Y, ldy, H, ldh, htype, h_scale, true, R, ldr, B, ldb, type, w, w_offset, gate, ldg,
                           gate_kind, scale, w_next, w_offset_next, eps, m, d, as_stream(stream));
}

Q4MM_API size_t q4_norm_workspace_size(int64_t m, int64_t d)
{
    if (m < 0 || m > kMaxRows || d < 1 || d > kMaxCols) return 0;
    return sizeof(float) * static_cast<size_t>(std::min<int64_t>(m, kNormPartials)) * static_cast<size_t>(d);
}

Q4MM_API int q4_norm_before_backward(void *dX, int64_t lddx, float *dw, const void *dH, int64_t lddh, const void *dR,
                                     int64_t lddr, const void *X, int64_t ldx, int type, const float *w,
                                     float w_offset, float eps, int64_t m, int64_t d, void *workspace,
                                     size_t workspace_bytes, q4mm_stream_t stream)
{
    if (!is_float_type(type) || m < 0 || m > kMaxRows || d < 1 || d > kMaxCols || !positive(eps)) return Q4_ERR_INVALID_ARG;
    Checker c(m);
    c.matrix(dX, lddx, d, type);
    c.matrix(dH, lddh, d, type);
    c.matrix(dR, lddr, d, type, true);
    c.matrix(X, ldx, d, type);
    c.vector(w, 4, true);
    c.vector(dw, 4, true);
    c.vector(workspace, 16, true);
    if (c.rc != Q4_OK) return c.rc;
    if (dw && m > 0 && (!workspace || workspace_bytes < q4_norm_workspace_size(m, d))) return Q4_ERR_WORKSPACE;
    if (m == 0 && !dw) return Q4_OK;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    cudaStream_t s = as_stream(stream);
    if (m == 0) return cuda_status(cudaMemsetAsync(dw, 0, sizeof(float) * static_cast<size_t>(d), s));
    const int size = type_size(type);
    RowAlign al, pa;
    al.add(dX, lddx * size);
    al.add(dH, lddh * size);
    al.add(dR, lddr * size);
    al.add(X, ldx * size);
    pa.add(w, 0);
    NormBeforeBwdArgs a{};
    a.dX = dX, a.dH = dH, a.dR = dR, a.X = X;
    a.lddx = lddx, a.lddh = lddh, a.lddr = lddr, a.ldx = ldx;
    a.w = w, a.w_off = w_offset, a.eps = eps;
    a.partials = dw ? static_cast<float *>(workspace) : nullptr;
    a.status = dev.status, a.wait_ns = wait_limit();
    a.m = m, a.d = d;
    return guarded([&] { return cuda_status(launch_norm_before_bwd(a, dw, type, access_of(al, type, nullptr, &pa), dev.sm_count, s)); });
}

Q4MM_API int q4_norm_after_backward(void *dB, int64_t lddb, float *dw, void *dgate, int64_t lddgate, const void *dY,
                                    int64_t lddy, const void *B, int64_t ldb, int type, const float *w, float w_offset,
                                    const void *gate, int64_t ldg, int gate_kind, float scale, float eps, int64_t m,
                                    int64_t d, void *workspace, size_t workspace_bytes, q4mm_stream_t stream)
{
    if (!is_float_type(type) || m < 0 || m > kMaxRows || d < 1 || d > kMaxCols || !positive(eps)) return Q4_ERR_INVALID_ARG;
    Checker c(m);
    c.matrix(dB, lddb, d, type);
    c.matrix(dY, lddy, d, type);
    c.matrix(B, ldb, d, type);
    c.vector(w, 4, true);
    c.vector(dw, 4, true);
    check_gate(c, gate, ldg, gate_kind, d, type);
    if (c.rc == Q4_OK && dgate) check_gate(c, dgate, lddgate, gate_kind, d, type);
    if (c.rc == Q4_OK && dgate && gate_kind == Q4_GATE_NONE) c.fail(Q4_ERR_INVALID_ARG);
    c.vector(workspace, 16, true);
    if (c.rc != Q4_OK) return c.rc;
    const bool columns = dw || (dgate && gate_kind == Q4_GATE_CHANNEL);
    if (columns && m > 0 && (!workspace || workspace_bytes < q4_norm_workspace_size(m, d))) return Q4_ERR_WORKSPACE;
    if (m == 0 && !columns) return Q4_OK;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    cudaStream_t s = as_stream(stream);
    if (m == 0) {
        const size_t bytes = sizeof(float) * static_cast<size_t>(d);
        cudaError_t e = dw ? cudaMemsetAsync(dw, 0, bytes, s) : cudaSuccess;
        if (e == cudaSuccess && dgate && gate_kind == Q4_GATE_CHANNEL) e = cudaMemsetAsync(dgate, 0, bytes, s);
        return cuda_status(e);
    }
    const int size = type_size(type);
    RowAlign al, pa;
    al.add(dB, lddb * size);
    al.add(dY, lddy * size);
    al.add(B, ldb * size);
    if (gate_kind == Q4_GATE_FULL) {
        al.add(gate, ldg * size);
        al.add(dgate, lddgate * size);
    }
    pa.add(w, 0);
    if (gate_kind == Q4_GATE_CHANNEL) pa.add(gate, 0);
    NormAfterBwdArgs a{};
    a.dB = dB, a.dgate = dgate, a.dY = dY, a.B = B, a.gate = gate;
    a.lddb = lddb, a.lddg = lddgate, a.lddy = lddy, a.ldb = ldb, a.ldg = ldg;
    a.w = w, a.w_off = w_offset;
    a.gate_kind = gate_kind, a.scale = scale, a.eps = eps;
    a.partials = columns ? static_cast<float *>(workspace) : nullptr;
    a.status = dev.status, a.wait_ns = wait_limit();
    a.m = m, a.d = d;
    return guarded([&] { return cuda_status(launch_norm_after_bwd(a, dw, type, access_of(al, type, nullptr, &pa), dev.sm_count, s)); });
}

static bool valid_moe(int64_t tokens, int64_t top_k)
{
    return tokens >= 0 && top_k >= 1 && top_k <= kMoeMaxTopK && tokens <= kMaxPairs / top_k;
}

Q4MM_API size_t q4_moe_workspace_size(int64_t tokens, int64_t top_k, int64_t n_experts)
{
    if (!valid_moe(tokens, top_k) || n_experts < 1 || n_experts > kMoeMaxExperts || tokens == 0) return 0;
    return moe_scratch(tokens * top_k, n_experts);
}

Q4MM_API int q4_moe_dispatch(void *Xs, int64_t ldxs, int64_t *offsets, int32_t *row_of, int32_t *pair_of,
                             const void *ids, int id_bytes, const void *X, int64_t ldx, int type, int64_t tokens,
                             int64_t top_k, int64_t n_experts, int64_t d, void *workspace, size_t workspace_bytes,
                             q4mm_stream_t stream)
{
    if (!valid_moe(tokens, top_k) || n_experts < 1 || n_experts > kMoeMaxExperts || (id_bytes != 4 && id_bytes != 8) ||
        (tokens > 0 && (X == nullptr) != (Xs == nullptr)))
        return Q4_ERR_INVALID_ARG;
    Checker c(tokens);
    c.vector(offsets, 8);
    c.per_row(row_of, 4);
    c.vector(pair_of, 4, true);
    c.per_row(ids, static_cast<uintptr_t>(id_bytes));
    if (X || Xs) {
        if (!is_float_type(type) || d < 1 || d > kMaxCols) return Q4_ERR_INVALID_ARG;
        c.matrix(X, ldx, d, type);
        c.matrix(Xs, ldxs, d, type);
    }
    c.vector(workspace, 16, true);
    if (c.rc != Q4_OK) return c.rc;
    const size_t need = q4_moe_workspace_size(tokens, top_k, n_experts);
    if (need > 0 && (!workspace || workspace_bytes < need)) return Q4_ERR_WORKSPACE;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    cudaStream_t s = as_stream(stream);
    if (tokens == 0) return cuda_status(cudaMemsetAsync(offsets, 0, sizeof(int64_t) * static_cast<size_t>(n_experts + 1), s));
    MoeDispatchArgs a{};
    a.offsets = offsets, a.row_of = row_of, a.pair_of = pair_of;
    a.ids = ids, a.id_bytes = id_bytes;
    a.tokens = tokens, a.pairs = tokens * top_k;
    a.top_k = static_cast<int>(top_k), a.experts = static_cast<int>(n_experts);
    a.hist = static_cast<int32_t *>(workspace);
    bool whole = true;
    if (X) {
        const int size = type_size(type);
        RowAlign al;
        al.add(X, ldx * size);
        al.add(Xs, ldxs * size);
        a.X = X, a.Xs = Xs;
        a.ldx = ldx * size, a.ldxs = ldxs * size;
        a.bytes = d * size;
        whole = al.bytes() == 16 && a.bytes % 16 == 0;
    }
    return guarded([&] { return cuda_status(launch_moe_dispatch(a, whole, dev.sm_count, s)); });
}

Q4MM_API int q4_moe_combine(void *Y, int64_t ldy, const void *base, int64_t ldbase, const void *Ys, int64_t ldys,
                            int type, const int32_t *row_of, const float *weights, int64_t tokens, int64_t top_k,
                            int64_t d, q4mm_stream_t stream)
{
    if (!is_float_type(type) || !valid_moe(tokens, top_k) || d < 1 || d > kMaxCols) return Q4_ERR_INVALID_ARG;
    Checker c(tokens);
    c.matrix(Y, ldy, d, type);
    c.matrix(base, ldbase, d, type, true);
    c.matrix(Ys, ldys, d, type);
    c.per_row(row_of, 4);
    c.vector(weights, 4, true);
    if (c.rc != Q4_OK) return c.rc;
    if (tokens == 0) return Q4_OK;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    const int size = type_size(type);
    RowAlign al;
    al.add(Y, ldy * size);
    al.add(base, ldbase * size);
    al.add(Ys, ldys * size);
    MoeCombineArgs a{};
    a.Y = Y, a.base = base, a.Ys = Ys;
    a.ldy = ldy, a.ldbase = ldbase, a.ldys = ldys;
    a.row_of = row_of, a.weights = weights;
    a.tokens = tokens, a.pairs = tokens * top_k;
    a.top_k = static_cast<int>(top_k), a.d = d;
    return guarded([&] { return cuda_status(launch_moe_combine(a, type, vec_of(al, type), as_stream(stream))); });
}

Q4MM_API int q4_moe_combine_backward(void *dYs, int64_t lddys, float *dweights, const void *dY, int64_t lddy,
                                     const void *Ys, int64_t ldys, int type, const int32_t *row_of,
                                     const float *weights, int64_t tokens, int64_t top_k, int64_t d,
                                     q4mm_stream_t stream)
{
    if (!is_float_type(type) || !valid_moe(tokens, top_k) || d < 1 || d > kMaxCols) return Q4_ERR_INVALID_ARG;
    Checker c(tokens);
    c.matrix(dYs, lddys, d, type);
    c.matrix(dY, lddy, d, type);
    c.matrix(Ys, ldys, d, type);
    c.per_row(row_of, 4);
    c.vector(weights, 4, true);
    c.vector(dweights, 4, true);
    if (c.rc != Q4_OK) return c.rc;
    if (tokens == 0) return Q4_OK;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    const int size = type_size(type);
    RowAlign al;
    al.add(dYs, lddys * size);
    al.add(dY, lddy * size);
    al.add(Ys, ldys * size);
    MoeCombineBwdArgs a{};
    a.dYs = dYs, a.dweights = dweights, a.dY = dY, a.Ys = Ys;
    a.lddys = lddys, a.lddy = lddy, a.ldys = ldys;
    a.row_of = row_of, a.weights = weights;
    a.tokens = tokens, a.pairs = tokens * top_k;
    a.top_k = static_cast<int>(top_k), a.d = d;
    return guarded([&] { return cuda_status(launch_moe_combine_bwd(a, type, vec_of(al, type), as_stream(stream))); });
}

} // extern "C"
