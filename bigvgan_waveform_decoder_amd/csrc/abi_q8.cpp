// C-ABI of the 8-bit serving operators (include/avae.h): argument checks and
// error reporting.  Every check runs before the first launch; the calls
// never allocate or synchronise.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>

#include "avae.h"
#include "avae_internal.h"

using avae::abi_fail;
using avae::CacheQ8;
using avae::Ragged;

namespace {

constexpr long long kMaxElems = 1LL << 46;  // keeps every byte offset in 64 bits
constexpr long long kMaxGroups = (1 << 24) - 1;  // of 256 threads: under 2^32 a launch

bool bad_dtype(int d) { return d != AVAE_F32 && d != AVAE_BF16 && d != AVAE_F16; }
int elem_size(int d) { return d == AVAE_F32 ? 4 : 2; }
bool misaligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

int done(hipError_t e, const char* who) {
    if (e != hipSuccess) return abi_fail(AVAE_EHIP, "%s: %s", who, hipGetErrorString(e));
    return AVAE_OK;
}

// Rows of `width` elements at stride ld.
int check_rows(const char* who, const char* what, int rows, long long width, long long ld) {
    if (ld < width)
        return abi_fail(AVAE_ESHAPE, "%s: %s has a row stride of %lld for %lld elements", who, what,
                        ld, width);
    if (ld > kMaxElems / (rows > 0 ? rows : 1))
        return abi_fail(AVAE_ESHAPE, "%s: %s is too large", who, what);
    return AVAE_OK;
}

int check_dtype(const char* who, int dtype, const void* p, const char* what) {
    if (bad_dtype(dtype)) return abi_fail(AVAE_EINVAL, "%s: dtype %d is none", who, dtype);
    if (misaligned(p, elem_size(dtype)))
        return abi_fail(AVAE_EINVAL, "%s: %s is not aligned to its elements", who, what);
    return AVAE_OK;
}

int check_cache(const char* who, const avae_kv_q8* kv, CacheQ8* out) {
    if (!kv || !kv->k || !kv->v || !kv->k_scale || !kv->v_scale)
        return abi_fail(AVAE_EINVAL, "%s: null cache pointer", who);
    if (kv->n_pages < 1 || kv->heads < 1 || kv->page < 1 || kv->dim < 1)
        return abi_fail(AVAE_EINVAL, "%s: cache sizes must be at least 1", who);
    if (kv->page != 16 && kv->page != 32 && kv->page != 64 && kv->page != 128 && kv->page != 256)
        return abi_fail(AVAE_ESHAPE, "%s: a page holds 16, 32, 64, 128 or 256 tokens, not %d", who,
                        kv->page);
    if (kv->dim != 64 && kv->dim != 128 && kv->dim != 256)
        return abi_fail(AVAE_ESHAPE, "%s: a head has 64, 128 or 256 dims, not %d", who, kv->dim);
    if (kv->heads > 4096) return abi_fail(AVAE_ESHAPE, "%s: more than 4096 heads", who);
    if (misaligned(kv->k, 16) || misaligned(kv->v, 16))
        return abi_fail(AVAE_EINVAL, "%s: k and v must be aligned to 16 bytes", who);
    if (misaligned(kv->k_scale, 4) || misaligned(kv->v_scale, 4))
        return abi_fail(AVAE_EINVAL, "%s: the scales are not aligned to 4 bytes", who);
    *out = CacheQ8{};
    out->k = kv->k;
    out->v = kv->v;
    out->k_scale = kv->k_scale;
    out->v_scale = kv->v_scale;
    out->n_pages = kv->n_pages;
    out->heads = kv->heads;
    out->page = kv->page;
    for (out->shift = 4; 1 << out->shift < kv->page;) ++out->shift;
    out->dim = kv->dim;
    return AVAE_OK;
}

int check_ragged(const char* who, const avae_ragged* r, CacheQ8* c, Ragged* out) {
    if (!r) return abi_fail(AVAE_EINVAL, "%s: null sequence description", who);
    if (r->seqs < 0 || r->total < 0 || r->max_rows < 0)
        return abi_fail(AVAE_EINVAL, "%s: negative size", who);
    if (r->seqs > 0 && (!r->cu || !r->lens || !r->table))
        return abi_fail(AVAE_EINVAL, "%s: null cu, lens or table", who);
    if (r->seqs > 65535) return abi_fail(AVAE_ESHAPE, "%s: more than 65535 sequences", who);
    if (r->seqs > 0 && (r->table_cols < 1 || r->table_ld < r->table_cols))
        return abi_fail(AVAE_ESHAPE, "%s: table of %d columns at a row stride of %lld", who,
                        r->table_cols, r->table_ld);
    if ((long long)r->table_cols * c->page > (1 << 29))
        return abi_fail(AVAE_ESHAPE, "%s: a table row covers more than 2^29 tokens", who);
    if (r->table_ld > kMaxElems / 65536)
        return abi_fail(AVAE_ESHAPE, "%s: the table is too large", who);
    if (r->max_rows > r->total)
        return abi_fail(AVAE_ESHAPE, "%s: max_rows %d is over total %d", who, r->max_rows,
                        r->total);
    if (r->total > (1 << 30)) return abi_fail(AVAE_ESHAPE, "%s: more than 2^30 rows", who);
    if (misaligned(r->cu, 4) || misaligned(r->lens, 4) || misaligned(r->table, 4))
        return abi_fail(AVAE_EINVAL, "%s: cu, lens or table is not aligned to 4 bytes", who);
    c->table = r->table;
    c->table_ld = r->table_ld;
    c->table_cols = r->table_cols;
    *out = Ragged{r->cu, r->lens, r->seqs, r->total, r->max_rows};
    return AVAE_OK;
}

int check_strides(const char* who, const char* what, long long tok, long long head, int total,
                  int heads, int dim) {
    if (head < dim && heads > 1)
        return abi_fail(AVAE_ESHAPE, "%s: %s has a head stride of %lld for %d dims", who, what,
                        head, dim);
    if (tok < 0 || head < 0 || tok > kMaxElems / (total > 0 ? total : 1) ||
        head > kMaxElems / heads)
        return abi_fail(AVAE_ESHAPE, "%s: %s has strides out of range", who, what);
    return AVAE_OK;
}

}  // namespace

#define AVAE_CHECK(expr)              \
    do {                              \
        const int rc_ = (expr);       \
        if (rc_ != AVAE_OK) return rc_; \
    } while (0)

extern "C" int avae_rms_norm_q8(const void* x, long long ldx, const void* residual, long long ldr,
                                const float* weight, int M, int C, int dtype, float eps, void* sum,
                                long long ldsum, signed char* q, long long ldq, float* scale,
                                void* stream) {
    const char* who = "avae_rms_norm_q8";
    if (M < 0 || C < 1) return abi_fail(AVAE_EINVAL, "%s: M >= 0 and C >= 1 are needed", who);
    if (!(eps >= 0.0f) || std::isinf(eps))
        return abi_fail(AVAE_EINVAL, "%s: eps must be finite and not negative", who);
    if (bad_dtype(dtype)) return abi_fail(AVAE_EINVAL, "%s: dtype %d is none", who, dtype);
    if ((residual == nullptr) != (sum == nullptr))
        return abi_fail(AVAE_EINVAL, "%s: residual and sum are given together or not at all", who);
    if (M == 0) return AVAE_OK;
    if (!x || !weight || !q || !scale) return abi_fail(AVAE_EINVAL, "%s: null pointer", who);
    AVAE_CHECK(check_dtype(who, dtype, x, "x"));
    AVAE_CHECK(check_dtype(who, dtype, residual, "residual"));
    AVAE_CHECK(check_dtype(who, dtype, sum, "sum"));
    AVAE_CHECK(check_dtype(who, AVAE_F32, weight, "weight"));
    AVAE_CHECK(check_dtype(who, AVAE_F32, scale, "scale"));
    AVAE_CHECK(check_rows(who, "x", M, C, ldx));
    AVAE_CHECK(check_rows(who, "q", M, C, ldq));
    if (residual) {
        AVAE_CHECK(check_rows(who, "residual", M, C, ldr));
        AVAE_CHECK(check_rows(who, "sum", M, C, ldsum));
        if (sum == x || sum == residual)
            return abi_fail(AVAE_EINVAL, "%s: sum must not be x or residual", who);
    }
    return done(avae::launch_rows_q8(dtype, x, ldx, residual, ldr, weight, M, C, eps, sum, ldsum,
                                     (int8_t*)q, ldq, scale, (hipStream_t)stream),
                who);
}

extern "C" int avae_quant_q8(const void* x, long long ldx, int M, int C, int dtype, signed char* q,
                             long long ldq, float* scale, void* stream) {
    const char* who = "avae_quant_q8";
    if (M < 0 || C < 1) return abi_fail(AVAE_EINVAL, "%s: M >= 0 and C >= 1 are needed", who);
    if (bad_dtype(dtype)) return abi_fail(AVAE_EINVAL, "%s: dtype %d is none", who, dtype);
    if (M == 0) return AVAE_OK;
    if (!x || !q || !scale) return abi_fail(AVAE_EINVAL, "%s: null pointer", who);
    AVAE_CHECK(check_dtype(who, dtype, x, "x"));
    AVAE_CHECK(check_dtype(who, AVAE_F32, scale, "scale"));
    AVAE_CHECK(check_rows(who, "x", M, C, ldx));
    AVAE_CHECK(check_rows(who, "q", M, C, ldq));
    return done(avae::launch_rows_q8(dtype, x, ldx, nullptr, 0, nullptr, M, C, 0.0f, nullptr, 0,
                                     (int8_t*)q, ldq, scale, (hipStream_t)stream),
                who);
}

extern "C" int avae_dequant_q8(const signed char* q, long long ldq, const float* scale, int M,
                               int C, int dtype, void* y, long long ldy, void* stream) {
    const char* who = "avae_dequant_q8";
    if (M < 0 || C < 1) return abi_fail(AVAE_EINVAL, "%s: M >= 0 and C >= 1 are needed", who);
    if (bad_dtype(dtype)) return abi_fail(AVAE_EINVAL, "%s: dtype %d is none", who, dtype);
    if (M == 0) return AVAE_OK;
    if (!y || !q || !scale) return abi_fail(AVAE_EINVAL, "%s: null pointer", who);
    AVAE_CHECK(check_dtype(who, dtype, y, "y"));
    AVAE_CHECK(check_dtype(who, AVAE_F32, scale, "scale"));
    AVAE_CHECK(check_rows(who, "q", M, C, ldq));
    AVAE_CHECK(check_rows(who, "y", M, C, ldy));
    return done(avae::launch_dequant_q8(dtype, (const int8_t*)q, ldq, scale, M, C, y, ldy,
                                        (hipStream_t)stream),
                who);
}

extern "C" size_t avae_linear_q8_workspace_bytes(int M, int N, int K) {
    if (M < 1 || N < 1 || K < 1 || K > AVAE_LINEAR_Q8_MAX_K) return 0;
    return avae::linear_q8_workspace_bytes(M, N, K);
}

extern "C" int avae_linear_q8(const signed char* a, long long lda, const float* a_scale,
                              const signed char* w, long long ldw, const float* w_scale,
                              const float* bias, int M, int N, int K, int act, int dtype, void* y,
                              long long ldy, void* workspace, size_t ws_bytes, void* stream) {
    const char* who = "avae_linear_q8";
    if (M < 0 || N < 1 || K < 1)
        return abi_fail(AVAE_EINVAL, "%s: M >= 0, N >= 1 and K >= 1 are needed", who);
    if (bad_dtype(dtype)) return abi_fail(AVAE_EINVAL, "%s: dtype %d is none", who, dtype);
    if (act != AVAE_ACT_NONE && act != AVAE_ACT_SILU)
        return abi_fail(AVAE_EINVAL, "%s: activation %d is none", who, act);
    if (K > AVAE_LINEAR_Q8_MAX_K)
        return abi_fail(AVAE_ESHAPE, "%s: K %d is over %d: the sum could leave int32", who, K,
                        AVAE_LINEAR_Q8_MAX_K);
    if (M == 0) return AVAE_OK;
    if (!a || !a_scale || !w || !w_scale || !y)
        return abi_fail(AVAE_EINVAL, "%s: null pointer", who);
    AVAE_CHECK(check_dtype(who, dtype, y, "y"));
    AVAE_CHECK(check_dtype(who, AVAE_F32, a_scale, "a_scale"));
    AVAE_CHECK(check_dtype(who, AVAE_F32, w_scale, "w_scale"));
    AVAE_CHECK(check_dtype(who, AVAE_F32, bias, "bias"));
    AVAE_CHECK(check_rows(who, "a", M, K, lda));
    AVAE_CHECK(check_rows(who, "w", N, K, ldw));
    AVAE_CHECK(check_rows(who, "y", M, N, ldy));
    if (M > (1 << 21) || N >= (1 << 28))
        return abi_fail(AVAE_ESHAPE, "%s: M is over 2^21 or N not under 2^28", who);
    const size_t need = avae::linear_q8_workspace_bytes(M, N, K);
    if (need && (!workspace || ws_bytes < need || misaligned(workspace, 16)))
        return abi_fail(AVAE_EWORKSPACE, "%s: %zu bytes of workspace, aligned to 16, are needed",
                        who, need);
    return done(avae::launch_linear_q8((const int8_t*)a, lda, a_scale, (const int8_t*)w, ldw,
                                       w_scale, bias, M, N, K, act, dtype, y, ldy, workspace,
                                       (hipStream_t)stream),
                who);
}

extern "C" int avae_kv_write_q8(const void* k, long long k_tok, long long k_head, const void* v,
                                long long v_tok, long long v_head, int dtype,
                                const avae_kv_q8* cache, const avae_ragged* rows, void* stream) {
    const char* who = "avae_kv_write_q8";
    CacheQ8 c;
    Ragged r;
    if (bad_dtype(dtype)) return abi_fail(AVAE_EINVAL, "%s: dtype %d is none", who, dtype);
    AVAE_CHECK(check_cache(who, cache, &c));
    AVAE_CHECK(check_ragged(who, rows, &c, &r));
    if (r.seqs == 0 || r.total == 0 || r.max_rows == 0) return AVAE_OK;
    if (!k || !v) return abi_fail(AVAE_EINVAL, "%s: null pointer", who);
    AVAE_CHECK(check_dtype(who, dtype, k, "k"));
    AVAE_CHECK(check_dtype(who, dtype, v, "v"));
    AVAE_CHECK(check_strides(who, "k", k_tok, k_head, r.total, c.heads, c.dim));
    AVAE_CHECK(check_strides(who, "v", v_tok, v_head, r.total, c.heads, c.dim));
    if (avae::kv_write_q8_pages(c, r) > kMaxGroups)
        return abi_fail(AVAE_ESHAPE, "%s: %d rows of one sequence at once touch more than 2^24 pages",
                        who, r.max_rows);
    return done(avae::launch_kv_write_q8(dtype, k, k_tok, k_head, v, v_tok, v_head, c, r,
                                         (hipStream_t)stream),
                who);
}

extern "C" int avae_kv_read_q8(const avae_kv_q8* cache, const avae_ragged* rows, int dtype, void* k,
                               void* v, void* stream) {
    const char* who = "avae_kv_read_q8";
    CacheQ8 c;
    Ragged r;
    if (bad_dtype(dtype)) return abi_fail(AVAE_EINVAL, "%s: dtype %d is none", who, dtype);
    AVAE_CHECK(check_cache(who, cache, &c));
    AVAE_CHECK(check_ragged(who, rows, &c, &r));
    if (r.seqs == 0 || r.total == 0 || r.max_rows == 0) return AVAE_OK;
    if (!k || !v) return abi_fail(AVAE_EINVAL, "%s: null pointer", who);
    AVAE_CHECK(check_dtype(who, dtype, k, "k"));
    AVAE_CHECK(check_dtype(who, dtype, v, "v"));
    return done(avae::launch_kv_read_q8(dtype, c, r, k, v, (hipStream_t)stream), who);
}

extern "C" size_t avae_attn_q8_workspace_bytes(const avae_kv_q8* cache, const avae_ragged* rows,
                                               int q_heads, int dtype, int max_len, int window) {
    if (bad_dtype(dtype) || !cache || !rows || cache->heads < 1 || cache->dim < 1 || q_heads < 1 || rows->seqs < 1 ||
        rows->total < 1 || rows->max_rows < 1 || max_len < 0 || window < 0 || q_heads % cache->heads)
        return 0;
    return avae::attn_q8_workspace_bytes(rows->seqs, rows->total, rows->max_rows, max_len, q_heads,
                                         cache->heads, cache->dim, elem_size(dtype), window);
}

extern "C" int avae_attn_q8(const void* q, long long q_tok, long long q_head, int q_heads,
                            int dtype, const avae_kv_q8* cache, const avae_ragged* rows,
                            const int* first, int max_len, float scale, int causal, int window,
                            void* out, float* lse, void* workspace, size_t ws_bytes,
                            void* stream) {
    const char* who = "avae_attn_q8";
    CacheQ8 c;
    Ragged r;
    if (bad_dtype(dtype)) return abi_fail(AVAE_EINVAL, "%s: dtype %d is none", who, dtype);
    AVAE_CHECK(check_cache(who, cache, &c));
    AVAE_CHECK(check_ragged(who, rows, &c, &r));
    if (q_heads < 1 || q_heads % c.heads)
        return abi_fail(AVAE_ESHAPE, "%s: %d query heads over %d cache heads", who, q_heads,
                        c.heads);
    if (q_heads / c.heads > 1024)
        return abi_fail(AVAE_ESHAPE, "%s: more than 1024 query heads a cache head", who);
    if (!std::isfinite(scale)) return abi_fail(AVAE_EINVAL, "%s: scale is not finite", who);
    if (max_len < 0 || window < 0)
        return abi_fail(AVAE_EINVAL, "%s: max_len and window are not negative", who);
    if (window > 0 && !causal)
        return abi_fail(AVAE_EINVAL, "%s: a window needs causal attention", who);
    if (r.seqs == 0 || r.total == 0 || r.max_rows == 0) return AVAE_OK;
    if ((long long)max_len > (long long)c.table_cols * c.page)
        return abi_fail(AVAE_ESHAPE, "%s: max_len %d is over the table's %lld tokens", who, max_len,
                        (long long)c.table_cols * c.page);
    if ((long long)r.max_rows * (q_heads / c.heads) > (1LL << 30))
        return abi_fail(AVAE_ESHAPE, "%s: more than 2^30 query rows a cache head", who);
    if (!q || !out) return abi_fail(AVAE_EINVAL, "%s: null pointer", who);
    AVAE_CHECK(check_dtype(who, dtype, q, "q"));
    AVAE_CHECK(check_dtype(who, dtype, out, "out"));
    AVAE_CHECK(check_dtype(who, AVAE_F32, lse, "lse"));
    if ((long long)r.total * q_heads > (1LL << 30))
        return abi_fail(AVAE_ESHAPE, "%s: more than 2^30 output rows", who);
    if (misaligned(out, 4 * elem_size(dtype)))
        return abi_fail(AVAE_EINVAL, "%s: out must be aligned to four elements", who);
    if (misaligned(first, 4))
        return abi_fail(AVAE_EINVAL, "%s: first is not aligned to 4 bytes", who);
    AVAE_CHECK(check_strides(who, "q", q_tok, q_head, r.total, q_heads, c.dim));
    const size_t need = avae::attn_q8_workspace_bytes(r.seqs, r.total, r.max_rows, max_len, q_heads,
                                                      c.heads, c.dim, elem_size(dtype), window);
    if (need && (!workspace || ws_bytes < need || misaligned(workspace, 16)))
        return abi_fail(AVAE_EWORKSPACE, "%s: %zu bytes of workspace, aligned to 16, are needed",
                        who, need);
    const long long groups = avae::attn_q8_workgroups(
        r.seqs, r.total, r.max_rows, max_len, q_heads, c.heads, c.dim, elem_size(dtype), window);
    if (groups > kMaxGroups)
        return abi_fail(AVAE_ESHAPE,
                        "%s: %d sequences of up to %d rows are %lld workgroups, over 2^24: give the "
                        "most rows that one has, or split the call",
                        who, r.seqs, r.max_rows, groups);
    avae::AttnQ8 a{};
    a.q = q;
    a.q_tok = q_tok;
    a.q_head = q_head;
    a.out = out;
    a.lse = lse;
    a.first = first;
    a.q_heads = q_heads;
    a.max_len = max_len;
    a.causal = causal ? 1 : 0;
    a.window = window < (1 << 30) ? window : 1 << 30;
    a.scale = scale;
    return done(avae::launch_attn_q8(dtype, a, c, r, workspace, (hipStream_t)stream), who);
}
