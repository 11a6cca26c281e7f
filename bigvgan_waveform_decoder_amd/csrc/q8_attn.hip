// Attention over the 8-bit paged cache.
//
// For a query row at position p of its sequence, over the keys t it sees
// (first <= t <= p, t > p - window):
//   s_t = scale * (q . k8_t) * k_scale[page(t)],   p_t = exp(s_t - max s),
//   out = sum_t p_t * v_scale[page(t)] * v8_t / sum_t p_t.
// A row that sees none gives zeros and lse = -inf.
//
// Both products run on the matrix cores in float16 with float32 sums: an
// 8-bit value is exact in float16.  The query row is brought to
// [2^14, 2^15) by a power of two (exact for bfloat16 and float16 values
// except where they fall 2^-25 below the row's largest); a float32 row is
// split into two float16 parts (22 bits).  p_t * v_scale is brought to at
// most 2^15 by the largest v_scale of the keys at hand and rounded to
// float16 (2^-11 of itself at most, an eighth of a bfloat16 output's own
// rounding), for float32 output again in two parts.
//
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T
// (v_mfma_f32_16x16x32_f16: lane l = 16 g + n holds A[n][8g..8g+7],
// B[8g..8g+7][n] and D[4g..4g+3][n]), so a query row is a column: its
// maximum, sum and rescaling factor live in its own four lanes, and the
// probabilities that a lane computes for keys 4g..4g+3 of two 16-key tiles
// are already the B operand of the second product, in a key order that V is
// read in too.
#include "avae.h"
#include "avae_internal.h"
#include "q8.h"

namespace avae {
namespace {

using namespace q8;

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;

__device__ inline float neg_inf() { return __uint_as_float(0xff800000u); }

// Two float16 values from bytes `sel` (0x64 in the upper half of each): a
// byte u there is 1024 + u; u is the stored value + 128.
__device__ inline h2 to_half2(unsigned bytes, unsigned sel) {
    const unsigned u = __builtin_amdgcn_perm(0x64646464u, bytes, sel);
    return __builtin_bit_cast(h2, u) - (h2){(_Float16)1152, (_Float16)1152};
}

// Eight 8-bit values (two words, each already xor 0x80808080) in float16.
__device__ inline h8 to_half8(unsigned lo, unsigned hi) {
    h2 r[4] = {to_half2(lo, 0x04010400u), to_half2(lo, 0x04030402u), to_half2(hi, 0x04010400u),
               to_half2(hi, 0x04030402u)};
    return __builtin_bit_cast(h8, r);
}

template <int N>
struct Words {
    unsigned w[N];
};

template <int N>
__device__ inline Words<N> load_bytes(const int8_t* p) {  // 4 N bytes, 4 N-byte aligned
    struct alignas(4 * N) Raw {
        unsigned w[N];
    };
    const Raw raw = *reinterpret_cast<const Raw*>(p);
    Words<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = raw.w[i] ^ 0x80808080u;
    return r;
}

// One wave: 16 query rows of one kv head, 32 keys a step.
template <typename T, int D>
__global__ __launch_bounds__(64) void attn_q8_kernel(AttnQ8 a, CacheQ8 c, Ragged r) {
    constexpr bool kSplit = sizeof(T) == 4;  // float32 rows in two float16 parts
    constexpr int KB = D / 32;               // key operands (32 dims each)
    constexpr int DT = D / 16;               // output tiles
    const int lane = threadIdx.x, n16 = lane & 15, g = lane >> 4;
    const int b = blockIdx.z, head = blockIdx.y;
    int cu0, n, len;
    if (!ragged_rows(r, b, cu0, n, len)) {
        // a sequence of no tokens that has rows: they see nothing
        len = 0;
        cu0 = r.cu[b];
        n = r.cu[b + 1] - cu0;
        if (cu0 < 0 || n <= 0 || r.cu[b + 1] > r.total) return;
    }
    const int group = a.q_heads / c.heads;
    const int row = blockIdx.x * 16 + n16;
    if (blockIdx.x * 16 >= (long long)n * group) return;
    const bool live = row < (long long)n * group;
    const int tok = live ? row / group : 0;
    const int q_head = head * group + (live ? row % group : 0);
    const int pos = len - n + tok;
    const int first = a.first ? max(a.first[b], 0) : 0;
    // keys [lo, hi) that this lane's row sees
    int hi = live ? (a.causal ? pos + 1 : len) : 0;
    hi = max(hi, 0);
    int lo = a.window ? max(first, pos - a.window + 1) : first;
    lo = min(lo, hi);
    // the whole tile's range
    int any_lo = live && lo < hi ? lo : 0x7fffffff, any_hi = hi;
    for (int o = 1; o < 16; o <<= 1) {
        any_lo = min(any_lo, __shfl_xor(any_lo, o));
        any_hi = max(any_hi, __shfl_xor(any_hi, o));
    }

    // the query row: power of two, then one or two float16 parts
    h8 qh[KB], ql[kSplit ? KB : 1];
    float q_back;
    {
        const T* qr = (const T*)a.q + (long long)(cu0 + tok) * a.q_tok + (long long)q_head * a.q_head;
        float top = 0.0f;
        for (int j = 0; j < KB; ++j)
            for (int i = 0; i < 8; ++i)
                top = fmaxf(top, fabsf((float)qr[64 * (j >> 1) + 16 * g + 8 * (j & 1) + i]));
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const int e = min(max((int)((__float_as_uint(top) >> 23) & 255) - 127, -100), 120);
        const float up = __uint_as_float((unsigned)(127 + 14 - e) << 23);
        q_back = __uint_as_float((unsigned)(127 - 14 + e) << 23) * a.scale * kLog2e;
        for (int j = 0; j < KB; ++j)
            for (int i = 0; i < 8; ++i) {
                const float x =
                    live ? (float)qr[64 * (j >> 1) + 16 * g + 8 * (j & 1) + i] * up : 0.0f;
                const _Float16 h = (_Float16)x;
                qh[j][i] = h;
                if (kSplit) ql[j][i] = (_Float16)(x - (float)h);
            }
    }

    // the largest value scale of the keys at hand
    float v_ref = 0.0f;
    const int page_lo = any_lo < any_hi ? any_lo / c.page : 0;
    const int page_hi = any_lo < any_hi ? (any_hi - 1) / c.page + 1 : 0;
    for (int col = page_lo + lane; col < page_hi; col += 64) {
        const int page = page_of(c, b, col);
        if (page >= 0) v_ref = fmaxf(v_ref, c.v_scale[(long long)page * c.heads + head]);
    }
    for (int o = 32; o > 0; o >>= 1) v_ref = fmaxf(v_ref, __shfl_xor(v_ref, o));
    if (!(v_ref > 0.0f)) v_ref = 1.0f;

    f4 acc[DT] = {};
    float m = neg_inf(), l = 0.0f;
    if (any_lo < any_hi)
        for (int t0 = any_lo & ~31; t0 < any_hi; t0 += 32) {
            f4 s[2];
            float pv[2];
            Words<D / 64> vw[8];
            bool seen[2][4];
            float top = neg_inf();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k0 = t0 + 16 * h;
                int page = page_of(c, b, k0 / c.page);
                const bool there = page >= 0;
                page = max(page, 0);
                const long long at = (long long)page * c.heads + head;
                const int8_t* kp = c.k + (at * c.page + k0 % c.page) * D;
                const int8_t* vp = c.v + (at * c.page + k0 % c.page) * D;
                const float ks = c.k_scale[at] * q_back;
                pv[h] = 32768.0f * (c.v_scale[at] / v_ref);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    vw[4 * h + i] = load_bytes<D / 64>(vp + (4 * g + i) * D + (D / 16) * n16);
                f4 sum = {};
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    const Words<4> kw = load_bytes<4>(kp + n16 * D + 64 * j + 16 * g);
                    const h8 k_lo = to_half8(kw.w[0], kw.w[1]), k_hi = to_half8(kw.w[2], kw.w[3]);
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_lo, qh[2 * j], sum, 0, 0, 0);
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_hi, qh[2 * j + 1], sum, 0, 0, 0);
                    if (kSplit) {
                        sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_lo, ql[2 * j], sum, 0, 0, 0);
                        sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_hi, ql[2 * j + 1], sum, 0, 0,
                                                                     0);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = k0 + 4 * g + i;
                    seen[h][i] = there && key >= lo && key < hi;
                    s[h][i] = seen[h][i] ? sum[i] * ks : neg_inf();
                    top = fmaxf(top, s[h][i]);
                }
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m_new = fmaxf(m, top);
            const float m_at = m_new == neg_inf() ? 0.0f : m_new;
            const float back = exp2f(m - m_at);
            m = m_new;
            l *= back;
            h8 ph, pl;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = seen[h][i] ? exp2f(s[h][i] - m_at) : 0.0f;
                    l += p;
                    const float x = seen[h][i] ? p * pv[h] : 0.0f;
                    const _Float16 hx = (_Float16)x;
                    ph[4 * h + i] = hx;
                    if (kSplit) pl[4 * h + i] = (_Float16)(x - (float)hx);
                }
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
                // bytes of eight keys, four dims: pairs of keys, then halves
                unsigned lo01[4], hi01[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lo01[i] = __builtin_amdgcn_perm(vw[2 * i + 1].w[w], vw[2 * i].w[w], 0x05010400u);
                    hi01[i] = __builtin_amdgcn_perm(vw[2 * i + 1].w[w], vw[2 * i].w[w], 0x07030602u);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h2 x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = to_half2(e < 2 ? lo01[i] : hi01[i],
                                        (e & 1) ? 0x04030402u : 0x04010400u);
                    const h8 vv = __builtin_bit_cast(h8, x);
                    f4 o = acc[4 * w + e] * back;
                    o = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, ph, o, 0, 0, 0);
                    if (kSplit) o = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, pl, o, 0, 0, 0);
                    acc[4 * w + e] = o;
                }
            }
        }

    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (!live) return;
    const float by = l == 0.0f ? 0.0f : v_ref / (32768.0f * l);  // a NaN sum stays NaN
    T* out = (T*)a.out + ((long long)(cu0 + tok) * a.q_heads + q_head) * D;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < DT; ++t) out[DT * (4 * g + i) + t] = round_to<T>(acc[t][i] * by);
    if (a.lse && g == 0)
        a.lse[(long long)(cu0 + tok) * a.q_heads + q_head] =
            l == 0.0f ? neg_inf() : (m + log2f(l)) * 0.6931471805599453f;
}

template <typename T>
hipError_t attn_q8(const AttnQ8& a, const CacheQ8& c, const Ragged& r, hipStream_t stream) {
    const int group = a.q_heads / c.heads;
    const dim3 grid((unsigned)(((long long)r.max_rows * group + 15) / 16), c.heads, r.seqs);
    if (c.dim == 64)
        hipLaunchKernelGGL((attn_q8_kernel<T, 64>), grid, dim3(64), 0, stream, a, c, r);
    else if (c.dim == 128)
        hipLaunchKernelGGL((attn_q8_kernel<T, 128>), grid, dim3(64), 0, stream, a, c, r);
    else
        hipLaunchKernelGGL((attn_q8_kernel<T, 256>), grid, dim3(64), 0, stream, a, c, r);
    return hipGetLastError();
}

}  // namespace

size_t attn_q8_workspace_bytes(int seqs, int max_rows, int max_len, int q_heads, int heads,
                               int dim, int window) {
    return 0;
}

hipError_t launch_attn_q8(int dtype, const AttnQ8& a, const CacheQ8& c, const Ragged& r, void* ws,
                          hipStream_t stream) {
    prof_pre(stream);
    const hipError_t e = dtype == AVAE_F32    ? attn_q8<float>(a, c, r, stream)
                         : dtype == AVAE_BF16 ? attn_q8<__bf16>(a, c, r, stream)
                                              : attn_q8<_Float16>(a, c, r, stream);
    // lengths are on the device: counted as if every row saw max_len keys
    const double pairs = (double)r.total * a.q_heads * a.max_len;
    prof_post(stream, "attn_q8_kernel", 4.0 * pairs * c.dim,
              2.0 * r.seqs * (double)a.max_len * c.heads * c.dim);
    return e;
}

}  // namespace avae
