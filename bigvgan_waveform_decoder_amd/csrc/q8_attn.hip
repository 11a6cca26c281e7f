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
#include <algorithm>

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

// Natural logarithm of a sum of exponentials held as 2^m * l.
__device__ inline float lse_of(float m, float l) {
    return l == 0.0f ? neg_inf() : (m + log2f(l)) * 0.6931471805599453f;
}

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

// What a tile of 16 query rows sees.  Rows are the sequence's new tokens
// times the query heads of one cache head; lane 16 g + n has row n.
struct Row {
    int tok, q_head;  // of the packed rows
    int lo, hi;       // keys [lo, hi)
    bool live;
};

__device__ inline Row row_of(const AttnQ8& a, const CacheQ8& c, int b, int head, int cu0, int n,
                             int len, int row) {
    const int group = a.q_heads / c.heads;
    Row r;
    r.live = row < n * group;
    const int i = r.live ? row / group : 0;
    r.tok = cu0 + i;
    r.q_head = head * group + (r.live ? row - i * group : 0);
    const int pos = len - n + i;
    const int first = a.first ? max(a.first[b], 0) : 0;
    r.hi = r.live ? max(a.causal ? pos + 1 : len, 0) : 0;
    r.lo = min(a.window ? max(first, pos - a.window + 1) : first, r.hi);
    return r;
}

// Smallest and largest key bounds of a tile's rows that see any key, over
// the 16 lanes of each group.
__device__ inline void tile_bounds(const Row& r, int& any_lo, int& any_hi, int& all_lo,
                                   int& all_hi) {
    const bool sees = r.live && r.lo < r.hi;
    any_lo = sees ? r.lo : 0x7fffffff;
    any_hi = sees ? r.hi : 0;
    all_lo = r.live ? r.lo : 0;
    all_hi = r.live ? r.hi : 0x7fffffff;
    for (int o = 1; o < 16; o <<= 1) {
        any_lo = min(any_lo, __shfl_xor(any_lo, o));
        any_hi = max(any_hi, __shfl_xor(any_hi, o));
        all_lo = max(all_lo, __shfl_xor(all_lo, o));
        all_hi = min(all_hi, __shfl_xor(all_hi, o));
    }
}

// A query row in float16 (two parts for float32), brought up by a power of
// two; lane 16 g + n holds dims 64 j + 16 g .. + 15 of row n in operands 2 j
// and 2 j + 1.  `back` undoes the power.
template <typename T, int D>
struct Query {
    static constexpr bool kSplit = sizeof(T) == 4;
    static constexpr int KB = D / 32;
    h8 hi[KB], lo[kSplit ? KB : 1];
    float back;

    __device__ void load(const AttnQ8& a, const Row& r, int g) {
        const T* q = (const T*)a.q + (long long)r.tok * a.q_tok + (long long)r.q_head * a.q_head;
        float x[8 * KB];
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 8 * KB; ++j) {
            x[j] = r.live ? (float)q[64 * (j >> 4) + 16 * g + (j & 15)] : 0.0f;
            top = fmaxf(top, fabsf(x[j]));
        }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const int e = min(max((int)((__float_as_uint(top) >> 23) & 255) - 127, -100), 120);
        const float up = __uint_as_float((unsigned)(127 + 14 - e) << 23);
        back = __uint_as_float((unsigned)(127 - 14 + e) << 23);
#pragma unroll
        for (int j = 0; j < 8 * KB; ++j) {
            const float v = x[j] * up;
            const _Float16 h = (_Float16)v;
            hi[j / 8][j % 8] = h;
            if (kSplit) lo[j / 8][j % 8] = (_Float16)(v - (float)h);
        }
    }
};

constexpr int kWaves = 4;

// Few query rows: one tile of 16 rows a workgroup, the keys of one chunk
// dealt to its waves 32 at a time, straight from memory to the matrix cores'
// registers.  Each wave keeps its own maximum, sum and output; they are
// joined in LDS, and where the keys are split over workgroups a second
// kernel joins the chunks.  HBM-bound: the cache is read once.
template <typename T, int D>
__global__ __launch_bounds__(64 * kWaves) void attn_q8_few_kernel(AttnQ8 a, CacheQ8 c, Ragged r,
                                                                  int splits, int chunk,
                                                                  float* part) {
    constexpr bool kSplit = Query<T, D>::kSplit;
    constexpr int DT = D / 16;  // output tiles
    constexpr int LD = D + 4;
    __shared__ float s_out[kWaves * 16 * LD];
    __shared__ float s_m[kWaves * 16], s_l[kWaves * 16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15, g = lane >> 4;
    const int b = blockIdx.z, head = blockIdx.y;
    const int split = blockIdx.x % splits, tile = blockIdx.x / splits;
    int cu0, n, len;
    if (!ragged_rows(r, b, cu0, n, len)) {
        if (cu0 < 0 || n <= 0 || cu0 + (long long)n > r.total) return;
        len = 0;  // rows of a sequence without tokens see nothing
    }
    const int group = a.q_heads / c.heads;
    if (tile * 16 >= n * group) return;
    const Row row = row_of(a, c, b, head, cu0, n, len, tile * 16 + n16);
    int any_lo, any_hi, all_lo, all_hi;
    tile_bounds(row, any_lo, any_hi, all_lo, all_hi);
    const int base = any_lo < any_hi ? (any_lo & ~31) : 0;
    const int t_lo = base + split * chunk, t_hi = min(t_lo + chunk, any_hi);

    Query<T, D> q;
    q.load(a, row, g);
    const float to_log2 = q.back * a.scale * kLog2e;

    f4 acc[DT] = {};
    float m = neg_inf(), l = 0.0f, v_run = 0.0f;
    for (int t0 = t_lo + 32 * wave; t0 < t_hi; t0 += 32 * kWaves) {
        f4 s[2];
        float vs[2];
        Words<D / 64> vw[8];
        Words<4> kw[2][D / 64];
        float ks[2];
        bool there[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k0 = t0 + 16 * h;
            const int page = page_of(c, b, k0 / c.page);
            // a half that no row sees may lie in a page that holds anything
            there[h] = page >= 0 && k0 < any_hi && k0 + 16 > any_lo;
            const long long at = (long long)max(page, 0) * c.heads + head;
            const int8_t* kp = c.k + (at * c.page + k0 % c.page) * D;
            const int8_t* vp = c.v + (at * c.page + k0 % c.page) * D;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                kw[h][j] = load_bytes<4>(kp + n16 * D + 64 * j + 16 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                vw[4 * h + i] = load_bytes<D / 64>(vp + (4 * g + i) * D + (D / 16) * n16);
            ks[h] = c.k_scale[at];
            vs[h] = c.v_scale[at];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f4 sum = {};
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const h8 k_lo = to_half8(kw[h][j].w[0], kw[h][j].w[1]);
                const h8 k_hi = to_half8(kw[h][j].w[2], kw[h][j].w[3]);
                sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_lo, q.hi[2 * j], sum, 0, 0, 0);
                sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_hi, q.hi[2 * j + 1], sum, 0, 0, 0);
                if (kSplit) {
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_lo, q.lo[2 * j], sum, 0, 0, 0);
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_hi, q.lo[2 * j + 1], sum, 0, 0,
                                                                 0);
                }
            }
            s[h] = sum * (ks[h] * to_log2);
        }
        // keys that not every row sees, or that are not there
        const bool whole = there[0] && there[1] && t0 >= all_lo && t0 + 32 <= all_hi;
        unsigned hidden = 0;
        if (!whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = t0 + 16 * h + 4 * g + i;
                    if (!(there[h] && key >= row.lo && key < row.hi)) {
                        hidden |= 1u << (4 * h + i);
                        s[h][i] = neg_inf();
                    }
                }
        }
        float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                          fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m_new = fmaxf(m, top);
        const float m_at = m_new == neg_inf() ? 0.0f : m_new;
        // the largest value scale so far stands at 2^15
        const float v_new = fmaxf(v_run, fmaxf(there[0] ? vs[0] : 0.0f, there[1] ? vs[1] : 0.0f));
        const float inv = 1.0f / fmaxf(v_new, 1e-38f);
        float back = __builtin_amdgcn_exp2f(m - m_at);
        l *= back;
        back *= v_run * inv;
        if (!__all(back == 1.0f)) {
#pragma unroll
            for (int t = 0; t < DT; ++t) acc[t] *= back;
        }
        m = m_new;
        v_run = v_new;
        h8 ph, pl;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float pv = 32768.0f * (vs[h] * inv);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = __builtin_amdgcn_exp2f(s[h][i] - m_at);
                l += p;
                float x = p * pv;
                // a page's NaN scale stays with the rows that see it
                if (!whole && (hidden >> (4 * h + i) & 1)) x = 0.0f;
                const _Float16 hx = (_Float16)x;
                ph[4 * h + i] = hx;
                if (kSplit) pl[4 * h + i] = (_Float16)(x - (float)hx);
            }
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
                f4 o = acc[4 * w + e];
                o = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, ph, o, 0, 0, 0);
                if (kSplit) o = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, pl, o, 0, 0, 0);
                acc[4 * w + e] = o;
            }
        }
    }

    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
        s_m[wave * 16 + n16] = m;
        s_l[wave * 16 + n16] = l;
    }
    if (row.live) {
        const float unit = v_run * (1.0f / 32768.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < DT; t += 4)
                *reinterpret_cast<f4*>(s_out + (wave * 16 + n16) * LD + DT * (4 * g + i) + t) =
                    (f4){acc[t][i], acc[t + 1][i], acc[t + 2][i], acc[t + 3][i]} * unit;
    }
    __syncthreads();
    // each thread joins four dims of a row
    for (int e = threadIdx.x; e < 16 * (D / 4); e += 64 * kWaves) {
        const int i = e / (D / 4), d = e % (D / 4) * 4;
        const Row to = row_of(a, c, b, head, cu0, n, len, tile * 16 + i);
        if (!to.live) break;  // rows come in order
        float top = neg_inf(), sum = 0.0f;
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_m[w * 16 + i]);
        const float at = top == neg_inf() ? 0.0f : top;
        f4 o = {};
        for (int w = 0; w < kWaves; ++w) {
            const float by = __builtin_amdgcn_exp2f(s_m[w * 16 + i] - at);
            sum += by * s_l[w * 16 + i];
            o += by * *reinterpret_cast<const f4*>(s_out + (w * 16 + i) * LD + d);
        }
        const long long out_row = (long long)to.tok * a.q_heads + to.q_head;
        if (splits > 1) {
            float* pr = part + (out_row * splits + split) * (D + 4);
            *reinterpret_cast<f4*>(pr + 4 + d) = o;
            if (d == 0) {
                pr[0] = top;
                pr[1] = sum;
            }
        } else {
            const float by = sum == 0.0f ? 0.0f : 1.0f / sum;  // a NaN sum stays NaN
            Pack<T, 4> y;
#pragma unroll
            for (int j = 0; j < 4; ++j) y.v[j] = round_to<T>(o[j] * by);
            *reinterpret_cast<Pack<T, 4>*>((T*)a.out + out_row * D + d) = y;
            if (a.lse && d == 0) a.lse[out_row] = lse_of(top, sum);
        }
    }
}

// Joins the chunks of one output row: a thread for four dims, the chunks
// dealt to the workgroup's lanes beyond them.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_q8_join_kernel(AttnQ8 a, int splits,
                                                           const float* __restrict__ part) {
    constexpr int COLS = D / 4, LANES = 256 / COLS;
    __shared__ f4 s_out[256];
    __shared__ float s_m[256], s_l[256];
    const long long row = blockIdx.x;
    const int col = threadIdx.x % COLS, at = threadIdx.x / COLS;
    const float* pr = part + row * splits * (D + 4);
    float m = neg_inf(), l = 0.0f;
    f4 o = {};
    for (int s = at; s < splits; s += LANES) {
        const float pm = pr[s * (D + 4)], pl = pr[s * (D + 4) + 1];
        const f4 po = *reinterpret_cast<const f4*>(pr + s * (D + 4) + 4 + 4 * col);
        if (pm == neg_inf() && pl == 0.0f) continue;  // the chunk has no key of this row
        const float m_new = fmaxf(m, pm);
        const float old = __builtin_amdgcn_exp2f(m - m_new), now = __builtin_amdgcn_exp2f(pm - m_new);
        l = l * old + pl * now;
        o = o * old + po * now;
        m = m_new;
    }
    s_out[threadIdx.x] = o;
    s_m[threadIdx.x] = m;
    s_l[threadIdx.x] = l;
    __syncthreads();
    if (at != 0) return;
    float top = m;
    for (int k = 1; k < LANES; ++k) top = fmaxf(top, s_m[k * COLS + col]);
    const float ref = top == neg_inf() ? 0.0f : top;
    float sum = 0.0f;
    f4 out = {};
    for (int k = 0; k < LANES; ++k) {
        const float by = __builtin_amdgcn_exp2f(s_m[k * COLS + col] - ref);
        sum += by * s_l[k * COLS + col];
        out += by * s_out[k * COLS + col];
    }
    const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
    Pack<T, 4> y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y.v[j] = round_to<T>(out[j] * by);
    *reinterpret_cast<Pack<T, 4>*>((T*)a.out + row * D + 4 * col) = y;
    if (a.lse && col == 0) a.lse[row] = lse_of(top, sum);
}

// How the keys of a row tile are cut: about kChunks pieces in all, each of at
// least 32 keys a wave.  The lengths are on the device, so this goes by the
// longest; pieces past a sequence's end are empty.
struct Cut {
    int tiles, splits, chunk;
};

constexpr int kChunks = 4096;

Cut cut(int seqs, int max_rows, int max_len, int q_heads, int heads, int window) {
    const int group = q_heads / heads;
    Cut r;
    r.tiles = (int)(((long long)max_rows * group + 15) / 16);
    long long span = max_len;  // keys of one row tile
    if (window > 0) span = std::min<long long>(span, (long long)window + 16 / group + 33);
    const long long all = span * seqs * heads * r.tiles;
    const long long step = 32 * kWaves;
    long long chunk = (all / kChunks + step - 1) / step * step;
    chunk = std::min(std::max(chunk, step), (span + step - 1) / step * step);
    r.chunk = (int)std::max(chunk, step);
    r.splits = (int)std::max<long long>(1, (span + r.chunk - 1) / r.chunk);
    return r;
}

template <typename T, int D>
hipError_t run(const AttnQ8& a, const CacheQ8& c, const Ragged& r, float* part,
               hipStream_t stream) {
    const Cut k = cut(r.seqs, r.max_rows, a.max_len, a.q_heads, c.heads, a.window);
    hipLaunchKernelGGL((attn_q8_few_kernel<T, D>), dim3(k.tiles * k.splits, c.heads, r.seqs),
                       dim3(64 * kWaves), 0, stream, a, c, r, k.splits, k.chunk, part);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && k.splits > 1) {
        hipLaunchKernelGGL((attn_q8_join_kernel<T, D>), dim3((unsigned)(r.total * a.q_heads)),
                           dim3(256), 0, stream, a, k.splits, part);
        e = hipGetLastError();
    }
    return e;
}

template <typename T>
hipError_t attn_q8(const AttnQ8& a, const CacheQ8& c, const Ragged& r, float* part,
                   hipStream_t stream) {
    if (c.dim == 64) return run<T, 64>(a, c, r, part, stream);
    if (c.dim == 128) return run<T, 128>(a, c, r, part, stream);
    return run<T, 256>(a, c, r, part, stream);
}

}  // namespace

size_t attn_q8_workspace_bytes(int seqs, int total, int max_rows, int max_len, int q_heads,
                               int heads, int dim, int window) {
    const Cut k = cut(seqs, max_rows, max_len, q_heads, heads, window);
    return k.splits > 1 ? (size_t)total * q_heads * k.splits * (dim + 4) * sizeof(float) : 0;
}

hipError_t launch_attn_q8(int dtype, const AttnQ8& a, const CacheQ8& c, const Ragged& r, void* ws,
                          hipStream_t stream) {
    prof_pre(stream);
    float* part = (float*)ws;
    const hipError_t e = dtype == AVAE_F32    ? attn_q8<float>(a, c, r, part, stream)
                         : dtype == AVAE_BF16 ? attn_q8<__bf16>(a, c, r, part, stream)
                                              : attn_q8<_Float16>(a, c, r, part, stream);
    // lengths are on the device: counted as if every row saw max_len keys
    const double pairs = (double)r.total * a.q_heads * a.max_len;
    prof_post(stream, "attn_q8_kernel", 4.0 * pairs * c.dim,
              2.0 * r.seqs * (double)a.max_len * c.heads * c.dim);
    return e;
}

}  // namespace avae
