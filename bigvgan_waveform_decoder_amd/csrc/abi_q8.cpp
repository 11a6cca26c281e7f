// C-ABI of the 8-bit serving operators (include/avae.h): argument checks and
// error reporting.  Every check runs before the first launch; the calls
// never allocate or synchronise.
#include <hip/hip_runtime.h>

#include <algorithm>
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

// The arguments that both attentions have; `nothing`: no row to compute.
static int check_attn(const char* who, const void* q, long long q_tok, long long q_head,
                      int q_heads, int dtype, const avae_kv_q8* cache, const avae_ragged* rows,
                      const int* first, int max_len, float scale, int causal, int window,
                      int prefix, bool rules, void* out, float* lse, void* workspace, size_t ws_bytes,
                      avae::AttnQ8* to, CacheQ8* cache_to, Ragged* rows_to, bool* nothing) {
    CacheQ8& c = *cache_to;
    Ragged& r = *rows_to;
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
    *nothing = r.seqs == 0 || r.total == 0 || r.max_rows == 0;
    if (*nothing) return AVAE_OK;
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
                                                      c.heads, c.dim, elem_size(dtype), window,
                                                      prefix, rules);
    if (need && (!workspace || ws_bytes < need || misaligned(workspace, 16)))
        return abi_fail(AVAE_EWORKSPACE, "%s: %zu bytes of workspace, aligned to 16, are needed",
                        who, need);
    const long long groups = avae::attn_q8_workgroups(
        r.seqs, r.total, r.max_rows, max_len, q_heads, c.heads, c.dim, elem_size(dtype), window,
        prefix, rules);
    if (groups > kMaxGroups)
        return abi_fail(AVAE_ESHAPE,
                        "%s: %d sequences of up to %d rows are %lld workgroups, over 2^24: give the "
                        "most rows that one has, or split the call",
                        who, r.seqs, r.max_rows, groups);
    avae::AttnQ8& a = *to;
    a = avae::AttnQ8{};
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
    return AVAE_OK;
}

extern "C" int avae_attn_q8(const void* q, long long q_tok, long long q_head, int q_heads,
                            int dtype, const avae_kv_q8* cache, const avae_ragged* rows,
                            const int* first, int max_len, float scale, int causal, int window,
                            void* out, float* lse, void* workspace, size_t ws_bytes,
                            void* stream) {
    const char* who = "avae_attn_q8";
    avae::AttnQ8 a;
    CacheQ8 c;
    Ragged r;
    bool nothing = false;
    AVAE_CHECK(check_attn(who, q, q_tok, q_head, q_heads, dtype, cache, rows, first, max_len, scale,
                          causal, window, 0, false, out, lse, workspace, ws_bytes, &a, &c, &r, &nothing));
    if (nothing) return AVAE_OK;
    return done(avae::launch_attn_q8(dtype, a, c, r, workspace, (hipStream_t)stream), who);
}

// What turns the heads (null: nothing does).
static int check_rope(const char* who, const avae_rope* rope, int dim, const int* positions,
                      avae::RopeQ8* out) {
    *out = avae::RopeQ8{};
    if (misaligned(positions, 4))
        return abi_fail(AVAE_EINVAL, "%s: positions is not aligned to 4 bytes", who);
    out->positions = positions;
    if (!rope || rope->rot == 0) return AVAE_OK;
    if (!rope->freq || misaligned(rope->freq, 4))
        return abi_fail(AVAE_EINVAL, "%s: null or misaligned frequencies", who);
    if (rope->rot < 0 || rope->rot % 2 || rope->rot > dim)
        return abi_fail(AVAE_ESHAPE, "%s: %d of %d dims cannot be turned in pairs", who, rope->rot,
                        dim);
    if (!std::isfinite(rope->amp)) return abi_fail(AVAE_EINVAL, "%s: amp is not finite", who);
    out->freq = rope->freq;
    out->half = rope->rot / 2;
    out->apart = rope->interleaved ? 0 : out->half;
    out->amp = rope->amp;
    return AVAE_OK;
}

// Sequences whose pages nobody looks at: cu and lens alone.
static int check_rows_of(const char* who, const avae_ragged* r, Ragged* out) {
    if (r->seqs < 0 || r->total < 0 || r->max_rows < 0)
        return abi_fail(AVAE_EINVAL, "%s: negative size", who);
    if (r->seqs > 0 && (!r->cu || !r->lens))
        return abi_fail(AVAE_EINVAL, "%s: null cu or lens", who);
    if (r->seqs > 65535) return abi_fail(AVAE_ESHAPE, "%s: more than 65535 sequences", who);
    if (r->max_rows > r->total)
        return abi_fail(AVAE_ESHAPE, "%s: max_rows %d is over total %d", who, r->max_rows,
                        r->total);
    if (r->total > (1 << 30)) return abi_fail(AVAE_ESHAPE, "%s: more than 2^30 rows", who);
    if (misaligned(r->cu, 4) || misaligned(r->lens, 4))
        return abi_fail(AVAE_EINVAL, "%s: cu or lens is not aligned to 4 bytes", who);
    *out = Ragged{r->cu, r->lens, r->seqs, r->total, r->max_rows};
    return AVAE_OK;
}

extern "C" int avae_rope_freq(int rot, double theta, int kind, double factor, double context,
                              double low, double high, float* freq, float* amp) {
    const char* who = "avae_rope_freq";
    if (!freq || !amp) return abi_fail(AVAE_EINVAL, "%s: null pointer", who);
    if (rot < 2 || rot % 2 || rot > 65536)
        return abi_fail(AVAE_ESHAPE, "%s: rot %d is no even number from 2 to 65536", who, rot);
    if (!(theta > 1.0) || std::isinf(theta))
        return abi_fail(AVAE_EINVAL, "%s: theta must be over 1 and finite", who);
    if (kind < AVAE_ROPE_PLAIN || kind > AVAE_ROPE_RAMP)
        return abi_fail(AVAE_EINVAL, "%s: scaling %d is none", who, kind);
    if (kind != AVAE_ROPE_PLAIN && (!(factor >= 1.0) || std::isinf(factor)))
        return abi_fail(AVAE_EINVAL, "%s: factor must be at least 1 and finite", who);
    if (kind == AVAE_ROPE_BASE && rot == 2)
        return abi_fail(AVAE_ESHAPE, "%s: a single pair has no base to raise", who);
    const bool bands = kind == AVAE_ROPE_BANDS || kind == AVAE_ROPE_RAMP;
    if (bands && !(context >= 1.0 && std::isfinite(context) && low > 0.0 && high > low &&
                   std::isfinite(high)))
        return abi_fail(AVAE_EINVAL,
                        "%s: context >= 1 and 0 < low < high, all finite, are needed", who);
    const double tau = 6.283185307179586476925286766559;
    const int half = rot / 2;
    if (kind == AVAE_ROPE_BASE) theta *= std::pow(factor, (double)rot / (rot - 2));
    // the pair that turns `turns` times over the context
    auto pair_of = [&](double turns) {
        return half * std::log(context / (tau * turns)) / std::log(theta);
    };
    const double first = bands ? std::max(std::floor(pair_of(high)), 0.0) : 0.0;
    const double last = bands ? std::min(std::ceil(pair_of(low)), (double)(rot - 1)) : 0.0;
    for (int i = 0; i < half; ++i) {
        const double f = std::pow(theta, -(double)i / half);
        double keep = 1.0;  // the share of f itself, the rest is f / factor
        if (kind == AVAE_ROPE_LINEAR) keep = 0.0;
        if (kind == AVAE_ROPE_BANDS) keep = (context * f / tau - low) / (high - low);
        if (kind == AVAE_ROPE_RAMP) keep = 1.0 - (i - first) / std::max(last - first, 1e-3);
        keep = std::min(std::max(keep, 0.0), 1.0);
        freq[i] = (float)(f * keep + f / (kind == AVAE_ROPE_BASE ? 1.0 : factor) * (1.0 - keep));
    }
    *amp = kind == AVAE_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return AVAE_OK;
}

extern "C" int avae_qk_norm_rope(const void* q, long long q_tok, long long q_head, int q_heads,
                                 const float* q_weight, const void* k, long long k_tok,
                                 long long k_head, int k_heads, const float* k_weight, int dim,
                                 int dtype, float eps, const avae_rope* rope, const int* positions,
                                 const avae_ragged* rows, int total, void* q_out, long long qo_tok,
                                 long long qo_head, void* k_out, long long ko_tok,
                                 long long ko_head, void* stream) {
    const char* who = "avae_qk_norm_rope";
    if (bad_dtype(dtype)) return abi_fail(AVAE_EINVAL, "%s: dtype %d is none", who, dtype);
    if (dim < 2 || dim % 2 || dim > 512)
        return abi_fail(AVAE_ESHAPE, "%s: a head of %d dims: an even number from 2 to 512 is needed",
                        who, dim);
    if (q_heads < 1 || k_heads < 0 || q_heads > 65536 || k_heads > 65536)
        return abi_fail(AVAE_ESHAPE, "%s: %d query and %d key heads", who, q_heads, k_heads);
    if (!(eps >= 0.0f) || std::isinf(eps))
        return abi_fail(AVAE_EINVAL, "%s: eps must be finite and not negative", who);
    avae::RopeQ8 turn;
    AVAE_CHECK(check_rope(who, rope, dim, positions, &turn));
    Ragged r{};
    if (rows) {
        AVAE_CHECK(check_rows_of(who, rows, &r));
        if (rows->total != total)
            return abi_fail(AVAE_ESHAPE, "%s: total is %d here and %d in rows", who, total,
                            rows->total);
        if (r.seqs == 0 || r.max_rows == 0) return AVAE_OK;
    } else {
        if (total < 0 || total > (1 << 30))
            return abi_fail(AVAE_ESHAPE, "%s: total %d is not in 0 .. 2^30", who, total);
        if (total > 0 && !positions)
            return abi_fail(AVAE_EINVAL, "%s: neither rows nor positions are given", who);
        r.total = total;
    }
    if (total == 0) return AVAE_OK;
    const avae::HeadsQ8 hq{q, q_out, q_weight, q_tok, q_head, qo_tok, qo_head, q_heads};
    const avae::HeadsQ8 hk{k, k_out, k_weight, k_tok, k_head, ko_tok, ko_head, k_heads};
    for (const avae::HeadsQ8* h : {&hq, &hk}) {
        if (h->heads == 0) continue;
        if (!h->x || !h->y) return abi_fail(AVAE_EINVAL, "%s: null pointer", who);
        AVAE_CHECK(check_dtype(who, dtype, h->x, "an input"));
        AVAE_CHECK(check_dtype(who, dtype, h->y, "an output"));
        AVAE_CHECK(check_dtype(who, AVAE_F32, h->weight, "a weight"));
        AVAE_CHECK(check_strides(who, "an input", h->tok, h->head, total, h->heads, dim));
        AVAE_CHECK(check_strides(who, "an output", h->y_tok, h->y_head, total, h->heads, dim));
        // heads beside one another in a token, or tokens in a head
        const bool heads_in_tokens = h->y_tok >= (h->heads - 1) * h->y_head + dim;
        const bool tokens_in_heads = h->y_tok >= dim && h->y_head >= (total - 1) * h->y_tok + dim;
        if (total > 1 && !(heads_in_tokens || tokens_in_heads))
            return abi_fail(AVAE_ESHAPE, "%s: an output's heads overlap", who);
        if (h->x == h->y && ((total > 1 && h->tok != h->y_tok) ||
                             (h->heads > 1 && h->head != h->y_head)))
            return abi_fail(AVAE_EINVAL, "%s: in place needs one set of strides", who);
    }
    return done(avae::launch_qk_norm_rope(dtype, hq, hk, turn, r, dim, eps, (hipStream_t)stream),
                who);
}

extern "C" int avae_kv_write_rope_q8(const void* k, long long k_tok, long long k_head,
                                     const void* v, long long v_tok, long long v_head, int dtype,
                                     const float* k_weight, float eps, const avae_rope* rope,
                                     const int* positions, const avae_kv_q8* cache,
                                     const avae_ragged* rows, void* stream) {
    const char* who = "avae_kv_write_rope_q8";
    CacheQ8 c;
    Ragged r;
    avae::RopeQ8 turn;
    if (bad_dtype(dtype)) return abi_fail(AVAE_EINVAL, "%s: dtype %d is none", who, dtype);
    if (!(eps >= 0.0f) || std::isinf(eps))
        return abi_fail(AVAE_EINVAL, "%s: eps must be finite and not negative", who);
    AVAE_CHECK(check_cache(who, cache, &c));
    AVAE_CHECK(check_ragged(who, rows, &c, &r));
    AVAE_CHECK(check_rope(who, rope, c.dim, positions, &turn));
    if (r.seqs == 0 || r.total == 0 || r.max_rows == 0) return AVAE_OK;
    if (!k || !v) return abi_fail(AVAE_EINVAL, "%s: null pointer", who);
    AVAE_CHECK(check_dtype(who, dtype, k, "k"));
    AVAE_CHECK(check_dtype(who, dtype, v, "v"));
    AVAE_CHECK(check_dtype(who, AVAE_F32, k_weight, "k_weight"));
    AVAE_CHECK(check_strides(who, "k", k_tok, k_head, r.total, c.heads, c.dim));
    AVAE_CHECK(check_strides(who, "v", v_tok, v_head, r.total, c.heads, c.dim));
    if (avae::kv_write_q8_pages(c, r) > kMaxGroups)
        return abi_fail(AVAE_ESHAPE, "%s: %d rows of one sequence at once touch more than 2^24 pages",
                        who, r.max_rows);
    return done(avae::launch_kv_write_rope_q8(dtype, k, k_tok, k_head, v, v_tok, v_head, k_weight,
                                              eps, turn, c, r, (hipStream_t)stream),
                who);
}

extern "C" int avae_tree_mask(const int* parents, const avae_ragged* rows, int words, int* mask,
                              long long ld, int* positions, void* stream) {
    const char* who = "avae_tree_mask";
    Ragged r;
    if (!rows) return abi_fail(AVAE_EINVAL, "%s: null sequence description", who);
    AVAE_CHECK(check_rows_of(who, rows, &r));
    if (words < 0 || words > AVAE_TREE_MAX_WORDS)
        return abi_fail(AVAE_ESHAPE, "%s: %d words a row are not in 0 .. %d", who, words,
                        AVAE_TREE_MAX_WORDS);
    if (r.max_rows > 32 * words)
        return abi_fail(AVAE_ESHAPE, "%s: %d drafts of a sequence have no room in %d words", who,
                        r.max_rows, words);
    if (r.seqs == 0 || r.total == 0 || r.max_rows == 0) return AVAE_OK;
    if (!parents || !mask) return abi_fail(AVAE_EINVAL, "%s: null pointer", who);
    if (misaligned(parents, 4) || misaligned(mask, 4) || misaligned(positions, 4))
        return abi_fail(AVAE_EINVAL, "%s: parents, mask or positions is not aligned to 4 bytes",
                        who);
    AVAE_CHECK(check_rows(who, "mask", r.total, words, ld));
    return done(avae::launch_tree_mask(parents, r, words, mask, ld, positions, (hipStream_t)stream),
                who);
}

static int prefix_of(const avae_attn_rules* x) {
    return x && x->prefix && x->max_prefix > 0 ? x->max_prefix : 0;
}

extern "C" size_t avae_attn_rules_q8_workspace_bytes(const avae_kv_q8* cache,
                                                     const avae_ragged* rows, int q_heads,
                                                     int dtype, int max_len, int window,
                                                     const avae_attn_rules* rules) {
    if (bad_dtype(dtype) || !cache || !rows || cache->heads < 1 || cache->dim < 1 || q_heads < 1 ||
        rows->seqs < 1 || rows->total < 1 || rows->max_rows < 1 || max_len < 0 || window < 0 ||
        q_heads % cache->heads)
        return 0;
    return avae::attn_q8_workspace_bytes(rows->seqs, rows->total, rows->max_rows, max_len, q_heads,
                                         cache->heads, cache->dim, elem_size(dtype), window,
                                         prefix_of(rules), true);
}

extern "C" int avae_attn_rules_q8(const void* q, long long q_tok, long long q_head, int q_heads,
                                  int dtype, const avae_kv_q8* cache, const avae_ragged* rows,
                                  const int* first, int max_len, float scale, int causal,
                                  int window, const avae_attn_rules* rules, void* out, float* lse,
                                  void* workspace, size_t ws_bytes, void* stream) {
    const char* who = "avae_attn_rules_q8";
    if (!rules) return abi_fail(AVAE_EINVAL, "%s: null rules", who);
    if (rules->cap != 0.0f && !(rules->cap >= 1e-30f && rules->cap <= 1e30f))
        return abi_fail(AVAE_EINVAL, "%s: the cap is neither 0 nor in 1e-30 .. 1e30", who);
    if (misaligned(rules->slopes, 4) || misaligned(rules->prefix, 4) || misaligned(rules->tree, 4))
        return abi_fail(AVAE_EINVAL, "%s: slopes, prefix or tree is not aligned to 4 bytes", who);
    if (rules->prefix && !causal)
        return abi_fail(AVAE_EINVAL, "%s: a prefix needs causal attention", who);
    if (rules->max_prefix < 0)
        return abi_fail(AVAE_EINVAL, "%s: max_prefix is not negative", who);
    if (rules->tree && (!causal || window > 0 || rules->slopes || rules->prefix))
        return abi_fail(AVAE_EINVAL,
                        "%s: a tree goes with causal attention, no window, slopes or prefix", who);
    if (rules->tree && rows) {
        if (rules->tree_words < 0 || rules->tree_words > AVAE_TREE_MAX_WORDS)
            return abi_fail(AVAE_ESHAPE, "%s: %d words a row are not in 0 .. %d", who,
                            rules->tree_words, AVAE_TREE_MAX_WORDS);
        if (rows->max_rows > 32 * rules->tree_words)
            return abi_fail(AVAE_ESHAPE, "%s: %d drafts of a sequence have no room in %d words", who,
                            rows->max_rows, rules->tree_words);
        AVAE_CHECK(check_rows(who, "tree", rows->total, rules->tree_words, rules->tree_ld));
    }
    avae::AttnQ8 a;
    CacheQ8 c;
    Ragged r;
    bool nothing = false;
    AVAE_CHECK(check_attn(who, q, q_tok, q_head, q_heads, dtype, cache, rows, first, max_len, scale,
                          causal, window, prefix_of(rules), true, out, lse, workspace, ws_bytes, &a, &c,
                          &r, &nothing));
    if (nothing) return AVAE_OK;
    const avae::AttnRules x{rules->cap, rules->slopes, rules->prefix, rules->max_prefix,
                            (const unsigned*)rules->tree, rules->tree_ld, rules->tree_words, 0,
                            0};
    return done(avae::launch_attn_rules_q8(dtype, a, x, c, r, workspace, (hipStream_t)stream), who);
}
