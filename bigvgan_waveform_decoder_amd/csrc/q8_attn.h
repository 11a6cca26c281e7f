// Attention over the 8-bit paged cache: the kernels, for the plain form and
// the one with rules (q8_attn.hip, q8_attn_rules.hip, q8_attn_caps.hip).
//
// For a query row at position p of its sequence, over the keys t it sees
// (first <= t <= p, t > p - window):
//   s_t = scale * (q . k8_t) * k_scale[page(t)],   p_t = exp(s_t - max s),
//   out = sum_t p_t * v_scale[page(t)] * v8_t / sum_t p_t.
// A row that sees none gives zeros and lse = -inf.
//
// Rules change the scores, s = cap tanh(s / cap) and s -= slope |p - t|, or
// what a row sees: keys before a prefix whatever p and the window are, or of
// its own call's rows those of a bit mask.
//
// Both products run on the matrix cores in float16 with float32 sums: an
// 8-bit value is exact in float16.  The query row is brought to
// [2^14, 2^15) by a power of two (exact for bfloat16 and float16 values
// except where they fall 2^-25 below the row's largest); a float32 row is
// split into two float16 parts (22 bits).  p_t * v_scale is brought to at
// most 2^15 by the largest v_scale of the keys that the row has seen and
// rounded to float16: 2^-11 of itself at most, an eighth of a bfloat16
// output's own rounding; for float16 and float32 outputs in two parts.  (One
// part made float16 outputs' error 1.3 times a correctly rounded one's; two
// take 275 us for one's 230 at 2 x 4096 causal rows of 16 heads of 128.)
//
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T
// (v_mfma_f32_16x16x32_f16: lane l = 16 g + n holds A[n][8g..8g+7],
// B[8g..8g+7][n] and D[4g..4g+3][n]), so a query row is a column: its
// maximum, sum and rescaling factor live in its own four lanes, and the
// probabilities that a lane computes for keys 4g..4g+3 of two 16-key tiles
// are already the B operand of the second product, in a key order that V is
// read in too.
#pragma once

#include <algorithm>
#include <type_traits>

#include "avae.h"
#include "avae_internal.h"
#include "q8.h"

namespace avae {
namespace {

using namespace q8;

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;

__device__ inline float neg_inf() { return __uint_as_float(0xff800000u); }
__device__ inline float nan() { return __uint_as_float(0x7fc00000u); }
__device__ inline bool finite(float x) { return fabsf(x) < __uint_as_float(0x7f800000u); }

// The larger of a lane's value and that of the lane 32 (16) further on.
__device__ inline float max_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float max_quarters(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

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

// Eight stored values (two words) in float16.
__device__ inline h8 to_half8(unsigned lo, unsigned hi) {
    lo ^= 0x80808080u;
    hi ^= 0x80808080u;
    h2 r[4] = {to_half2(lo, 0x04010400u), to_half2(lo, 0x04030402u), to_half2(hi, 0x04010400u),
               to_half2(hi, 0x04030402u)};
    return __builtin_bit_cast(h8, r);
}

// Bytes 0, 1 (2, 3) of two keys' words, key by key, with the same offset.
__device__ inline unsigned pair_lo(unsigned a, unsigned b) {
    return __builtin_amdgcn_perm(b, a, 0x05010400u) ^ 0x80808080u;
}
__device__ inline unsigned pair_hi(unsigned a, unsigned b) {
    return __builtin_amdgcn_perm(b, a, 0x07030602u) ^ 0x80808080u;
}

template <int N>
struct Words {
    unsigned w[N];
};

template <int N>
__device__ inline Words<N> load_words(const int8_t* p) {  // 4 N bytes, 4 N-byte aligned
    struct alignas(4 * N) Raw {
        unsigned w[N];
    };
    const Raw raw = *reinterpret_cast<const Raw*>(p);
    Words<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = raw.w[i];
    return r;
}

// Types whose probabilities are taken in two float16 parts: one part's
// rounding is as large as a float16 output's own.
template <typename T>
constexpr bool kTwoParts = !std::is_same<T, __bf16>::value;

// The attention without rules: nothing of theirs is compiled into it.
struct NoRules {};
template <typename R>
constexpr bool kRules = !std::is_same<R, NoRules>::value;

// Rules with a cap that 16-bit scores may lie far below: it is taken to the
// scores' own rounding, as float32's is.  Kernels of their own, since the
// others' registers are full (both in one, the capped prompts of [3849 rows,
// 6047 keys] and [3642, 4762] take 354 us for 335, trees of heads of 256 230 for
// 213; these kernels take 460 for such a prompt).
struct FineRules : AttnRules {
    explicit FineRules(const AttnRules& x) : AttnRules(x) {}
};
constexpr float kQuickCap = 256.0f;  // caps above it
template <typename T, typename R>
constexpr bool kQuick = sizeof(T) < 4 && !std::is_same<R, FineRules>::value;

// What a tile of 16 query rows sees.  Rows are the sequence's new tokens
// times the query heads of one cache head; lane 16 g + n has row n.
struct Row {
    int tok, q_head;  // of the packed rows
    int lo, hi;       // keys [lo, hi)
    bool live;
    int pos;          // with rules: its place,
    int first, pre;   // and keys [first, pre) besides
};

template <typename R>
__device__ inline Row row_of(const AttnQ8& a, const CacheQ8& c, const R& x, int b, int head,
                             int cu0, int n, int len, int row) {
    const int group = a.q_heads / c.heads;
    Row r;
    r.live = row < n * group;
    const int i = r.live ? row / group : 0;
    r.tok = cu0 + i;
    r.q_head = head * group + (r.live ? row - i * group : 0);
    const int pos = len - n + i;
    const int first = a.first ? max(a.first[b], 0) : 0;
    // (a length past the table adds no key)
    const int most = c.table_cols << c.shift;
    r.pos = pos;
    r.first = r.pre = 0;
    if constexpr (kRules<R>) {
        // a row before its sequence's first token sees nothing
        const bool sees = r.live && pos >= 0;
        int hi = a.causal && !x.tree ? pos + 1 : len;
        if (x.prefix) {
            const int pre = min(min(max(x.prefix[b], 0), x.max_prefix), len);
            if (a.window) {
                r.first = first;
                r.pre = sees ? min(pre, most) : 0;
            } else {
                hi = max(hi, pre);
            }
        }
        r.hi = sees ? min(max(hi, 0), most) : 0;
    } else {
        r.hi = r.live ? min(max(a.causal ? pos + 1 : len, 0), most) : 0;
    }
    r.lo = min(a.window ? max(first, pos - a.window + 1) : first, r.hi);
    return r;
}

// The lowest k bits.
__device__ inline unsigned ones_below(int k) {
    return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1;
}

// Which of its call's rows j .. j + 31 a row sees by the mask; what lies
// before the first of them is the past, all of it seen.
__device__ inline unsigned tree_bits(const AttnRules& x, int tok, int j) {
    const unsigned* words = x.tree + (long long)tok * x.tree_ld;
    const int i = j >> 5, by = j & 31;
    auto word = [&](int at) {
        return at < 0 ? ~0u : at < x.tree_words ? words[at] : 0u;
    };
    const unsigned low = word(i);
    return by ? low >> by | word(i + 1) << (32 - by) : low;
}

// Which of the keys t .. t + 31 a row sees.
__device__ inline unsigned keys_seen(const Row& r, const AttnRules& x, int start, int t) {
    unsigned seen = ones_below(r.hi - t) & ~ones_below(r.lo - t);
    if (x.tree && t + 32 > start) seen &= tree_bits(x, r.tok, t - start);
    return seen | (ones_below(r.pre - t) & ~ones_below(r.first - t));
}

// tanh(y) as (1 - e) / (1 + e) with e = exp(-2 |y|): 2^-24 off, and a cap
// multiplies that, which the rounding of 16-bit types hides up to caps of 256.
__device__ inline float tanh_far(float y) {
    const float e = __builtin_amdgcn_exp2f(fabsf(y) * (-2.0f * kLog2e));
    return copysignf((1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e), y);
}

// Small |y| by the odd series, right to y's own rounding, so that a score far
// below its cap stays what it is.  (Without it a cap of 1e6 made bfloat16
// scores 1.3% wrong, one of 1e30 all of them 0.)
__device__ inline float tanh_of(float y) {
    const float far = tanh_far(y);
    const float z = y * y;
    float p = fmaf(z, -8.8632355e-3f, 2.1869489e-2f);
    p = fmaf(z, p, -5.3968254e-2f);
    p = fmaf(z, p, 1.3333333e-1f);
    p = fmaf(z, p, -3.3333333e-1f);
    return fabsf(y) < 0.25f ? fmaf(y * z, p, y) : far;
}

// Scores in units of log2 e from products and what they are multiplied with:
// their factor over the cap where there is one.
template <typename T, typename R>
struct Shape {
    float cap, slope;  // in units of log2 e; the slope is the row's
    bool capped, sloped;
    // 16-bit types: cap tanh(y) = cap - 2 cap / (1 + exp(2 y)), the first term
    // left out of the scores since all of a row have it; 5 2^-24 cap off,
    // which for caps up to 256 their own rounding hides.
    static constexpr bool quick = kQuick<T, R>;

    __device__ Shape(const AttnRules& x, const Row& r)
        : cap(x.cap * kLog2e), slope(0.0f), capped(x.cap > 0.0f), sloped(x.slopes != nullptr) {
        // held at 2^96: its product with a distance below 2^31 stays in float32,
        // and an infinite slope would be NaN at the row's own place (a NaN stays)
        if (sloped) {
            slope = x.slopes[r.q_head] * kLog2e;
            if (fabsf(slope) > 0x1p96f) slope = copysignf(0x1p96f, slope);
        }
    }
    // The factor of a page's scores.  A scale that is not finite makes them NaN
    // whatever the cap (`held` alone would make a number of a NaN), and under
    // one a factor past float32 is held: 0 times an infinity is NaN.  (At a
    // third of float32's largest: the quick cap takes it 2 log2 e times.)
    __device__ float by(float ks, float to_log2) const {
        return finite(ks) ? held(ks * to_log2) : nan();
    }
    __device__ float held(float x) const {
        return capped ? fminf(fmaxf(x, -1.1e38f), 1.1e38f) : x;
    }
    // The cap,
    // of s = 2 y log2 e, over 2 cap
    __device__ float cap_quick(float s) const {
        return __builtin_amdgcn_rcpf(-1.0f - __builtin_amdgcn_exp2f(s));
    }
    // of s = y
    __device__ float cap_whole(float s) const { return cap * (quick ? tanh_far(s) : tanh_of(s)); }
    // The bias of a key that far away (past 2^24 to float32's rounding).
    __device__ float bend(float s, float distance) const {
        return fmaf(-slope, fabsf(distance), s);
    }
};

template <typename T, typename R>
__device__ inline Shape<T, R> shape_of(const R& x, const Row& r) {
    return Shape<T, R>(x, r);
}
template <typename T>
__device__ inline NoRules shape_of(const NoRules&, const Row&) {
    return {};
}

// Smallest and largest key bounds of a tile's rows that see any key, over
// the 16 lanes of each group; no row sees all keys from `whole` on.
__device__ inline void tile_bounds(const Row& r, int whole, int& any_lo, int& any_hi, int& all_lo,
                                   int& all_hi) {
    const bool sees = r.live && r.lo < r.hi;
    any_lo = sees ? r.lo : 0x7fffffff;
    any_hi = sees ? r.hi : 0;
    all_lo = r.live ? r.lo : 0;
    all_hi = r.live ? min(r.hi, whole) : 0x7fffffff;
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
        const int e = min(max((int)((__float_as_uint(top) >> 23) & 255) - 127, -100), 127);
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

// Waves a SIMD of the kernel for few rows: as many as its registers allow
// without spills, for the bytes in flight.
constexpr int few_residency(int dim, int elem, int waves = kWaves) {
    if (waves > kWaves) return waves / 4;  // one workgroup a CU
    return dim > 128 ? 2 : elem == 4 && dim == 128 ? 3 : 4;
}

// Waves of its workgroups where they take all the keys of their rows: what
// fits the registers.
constexpr int wide_waves(int dim, int elem) {
    return dim > 128 || (elem == 4 && dim == 128) ? 8 : 16;
}

// Few query rows: one tile of 16 rows a workgroup, the keys of one chunk
// dealt to its waves 32 at a time, straight from memory to the matrix cores'
// registers.  Each wave keeps its own maximum, sum and output; they are
// joined in LDS, and where the keys are split over workgroups a second
// kernel joins the chunks.
//
// HBM-bound: the cache is read once.  Measured, one row a sequence: 64
// sequences of 12000 keys, 4 heads of 128: 151 us (5.2 TB/s; a copy reaches
// 5.1), 8 heads of 64: 150; lengths from 200 to 24000: 189 (4.3 TB/s, the
// chunks of a sequence's end are shorter than the others); one sequence of
// 2400 keys 8.3 us and 3.8 for the join, both latency.
//
// With rules the keys in view may lie in two runs, [first, pre) and the
// window's; they are counted through, u, and cut as one.
template <typename T, int D, typename R, int W>
__global__ __launch_bounds__(64 * W, few_residency(D, sizeof(T), W)) void attn_q8_few_kernel(AttnQ8 a, CacheQ8 c, Ragged r, R x,
                                                                  int splits, int chunk, int span,
                                                                  int pieces, int pairs,
                                                                  float* part) {
    constexpr bool kSplit = Query<T, D>::kSplit;
    constexpr int DT = D / 16;  // output tiles
    constexpr int LD = D + 4;
    __shared__ float s_out[W * 16 * LD];
    __shared__ float s_m[W * 16], s_l[W * 16];
    const int lane = threadIdx.x & 63, wave = wave_id(), n16 = lane & 15, g = lane >> 4;
    // Sequences, heads and tiles side by side, chunks after one another:
    // workgroups go to the XCDs in turn, and the last chunks may be empty.
    const int all = r.seqs * pairs;
    const int split = blockIdx.x / all, in_all = blockIdx.x % all;
    const int b = in_all / pairs, tile = in_all % pairs / c.heads, head = in_all % c.heads;
    int cu0, n, len;
    if (!ragged_rows(r, b, cu0, n, len)) return;
    const int group = a.q_heads / c.heads;
    if (tile * 16 >= n * group) return;
    if (pieces) {
        // The host cut by the longest sequence; what there is in all gives
        // shorter chunks, as many as it left room for.
        long long keys = 0;
        for (int i = lane; i < r.seqs; i += 64) keys += min(max(r.lens[i], 0), span);
        for (int o = 32; o > 0; o >>= 1) keys += __shfl_xor(keys, o);
        const long long even = (keys * pairs + pieces - 1) / pieces;
        const int least = (span + splits - 1) / splits;
        chunk = (min(chunk, max((int)min(even, (long long)chunk), least)) + 32 * W - 1) &
                ~(32 * W - 1);
    }
    const Row row = row_of(a, c, x, b, head, cu0, n, len, tile * 16 + n16);
    int any_lo, any_hi, all_lo, all_hi;
    int whole = 0x7fffffff;
    if constexpr (kRules<R>)
        if (x.tree) whole = len - n;
    tile_bounds(row, whole, any_lo, any_hi, all_lo, all_hi);
    int base = any_lo < any_hi ? (any_lo & ~31) : 0;
    int t_lo = base + split * chunk, t_hi = min(t_lo + chunk, any_hi);
    // with a prefix besides the window: keys [first, pre) of all rows, then
    // those from `base` on
    int first = 0, pre = 0, all_pre = 0, in_pre = 0;
    if constexpr (kRules<R>) {
        pre = row.pre;
        all_pre = row.live ? row.pre : 0x7fffffff;
        for (int o = 1; o < 16; o <<= 1) {
            pre = max(pre, __shfl_xor(pre, o));
            all_pre = min(all_pre, __shfl_xor(all_pre, o));
        }
        pre = __builtin_amdgcn_readfirstlane(pre);
        first = __builtin_amdgcn_readfirstlane(row.first);
        if (first < pre) {
            const int from = first & ~31, to = (pre + 31) & ~31;
            in_pre = to - from;
            base = max(any_lo < any_hi ? any_lo & ~31 : 0, to);
            t_lo = split * chunk;
            t_hi = min(t_lo + chunk, in_pre + max(any_hi - base, 0));
        }
    }
    auto key_at = [&](int u) {
        if constexpr (kRules<R>)
            if (first < pre) return u < in_pre ? (first & ~31) + u : base + (u - in_pre);
        return u;
    };

    if (splits > 1 && t_lo >= t_hi) {  // a chunk without keys
        if (threadIdx.x < 16 && row.live) {
            float* pr = part + (((long long)row.tok * a.q_heads + row.q_head) * splits + split) *
                                   (D + 4);
            pr[0] = neg_inf();
            pr[1] = 0.0f;
        }
        return;
    }

    // the table entries of a step, read a step ahead of their use
    int entry[2];
    auto look_up = [&](int t0) {
        entry[0] = page_entry(c, b, t0 >> c.shift);
        entry[1] = page_entry(c, b, (t0 + 16) >> c.shift);
    };
    look_up(key_at(t_lo + 32 * wave));
    Query<T, D> q;
    q.load(a, row, g);
    const auto shape = shape_of<T>(x, row);
    float to_log2 = q.back * a.scale * kLog2e;
    if constexpr (kRules<R>)
        if (x.cap > 0.0f) to_log2 = shape.held(q.back * shape.held(a.scale / x.cap));

    f4 acc[DT] = {};
    // v_run: the largest value scale so far, the accumulated values' unit; at
    // least float32's smallest normal number, which has a reciprocal
    float m = neg_inf(), l = 0.0f, v_run = 0x1p-126f;
    for (int u0 = t_lo + 32 * wave; u0 < t_hi; u0 += 32 * W) {
        const int t0 = key_at(u0);
        f4 s[2];
        float vs[2];
        Words<D / 64> vw[8];
        Words<4> kw[2][D / 64];
        float ks[2];
        bool there[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k0 = t0 + 16 * h;
            const int page = page_checked(c, k0 >> c.shift, entry[h]);
            // a half that no row sees may lie in a page that holds anything
            there[h] = page >= 0 && k0 < any_hi && k0 + 16 > any_lo;
            if constexpr (kRules<R>) there[h] |= page >= 0 && k0 < pre && k0 + 16 > first;
            const long long at = (long long)max(page, 0) * c.heads + head;
            const int8_t* kp = c.k + (at * c.page + (k0 & (c.page - 1))) * D;
            const int8_t* vp = c.v + (at * c.page + (k0 & (c.page - 1))) * D;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                kw[h][j] = load_words<4>(kp + n16 * D + 64 * j + 16 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                vw[4 * h + i] = load_words<D / 64>(vp + (4 * g + i) * D + (D / 16) * n16);
            ks[h] = c.k_scale[at];
            vs[h] = c.v_scale[at];
        }
        look_up(key_at(u0 + 32 * W));
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
            if constexpr (kRules<R>) {
                s[h] = sum * shape.by(ks[h], to_log2);
                if (shape.capped) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[h][i] = shape.cap_whole(s[h][i]);
                }
                if (shape.sloped) {
                    const float away = (float)(row.pos - (t0 + 16 * h + 4 * g));
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[h][i] = shape.bend(s[h][i], away - i);
                }
            } else {
                s[h] = sum * (ks[h] * to_log2);
            }
        }
        bool part_seen = t0 < all_lo || t0 + 32 > all_hi;
        if constexpr (kRules<R>) part_seen &= t0 < first || t0 + 32 > all_pre;
        if (__builtin_amdgcn_readfirstlane(part_seen || !there[0] || !there[1] ||
                                           !finite(vs[0] + vs[1]))) {
            // Some of the keys are hidden from some of the rows, or a page's
            // value scale is NaN: that goes into the scores, so that it stays
            // with the rows that see it.  A page that a row does not see is
            // not in its largest value scale either.
            const int lo = row.lo - t0 - 4 * g, hi = row.hi - t0 - 4 * g;
            unsigned seen = 0;
            if constexpr (kRules<R>) seen = keys_seen(row, x, len - n, t0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[h][i] += finite(vs[h]) ? 0.0f : nan();
                    bool on = 16 * h + i >= lo && 16 * h + i < hi;
                    if constexpr (kRules<R>) on = seen >> (4 * g) & 1u << (16 * h + i);
                    s[h][i] = there[h] && on ? s[h][i] : neg_inf();
                }
                const int k0 = t0 + 16 * h;
                bool sees = there[h] && row.lo < k0 + 16 && row.hi > k0;
                if constexpr (kRules<R>) sees = there[h] && seen >> (16 * h) & 0xffffu;
                vs[h] = sees && finite(vs[h]) ? vs[h] : 0.0f;
            }
        }
        float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                          fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        top = max_halves(max_quarters(top));
        const float m_new = fmaxf(m, top);
        const float m_at = m_new == neg_inf() ? 0.0f : m_new;
        // the largest value scale so far stands at 2^15
        const float v_new = fmaxf(v_run, fmaxf(vs[0], vs[1]));
        const float inv = 1.0f / v_new;
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
                // both parts are of this number: the product would else be
                // fused with one conversion and not with the other, 2^-11 apart
                // where its rounding makes a tie
                if (kTwoParts<T>) asm("" : "+v"(x));
                const _Float16 hx = (_Float16)x;
                ph[4 * h + i] = hx;
                if (kTwoParts<T>) pl[4 * h + i] = (_Float16)(x - (float)hx);
            }
        }
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
            // bytes of eight keys, four dims: pairs of keys, then halves
            unsigned lo01[4], hi01[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo01[i] = pair_lo(vw[2 * i].w[w], vw[2 * i + 1].w[w]);
                hi01[i] = pair_hi(vw[2 * i].w[w], vw[2 * i + 1].w[w]);
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
                if (kTwoParts<T>) o = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, pl, o, 0, 0, 0);
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
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < DT; t += 4)
                *reinterpret_cast<f4*>(s_out + (wave * 16 + n16) * LD + DT * (4 * g + i) + t) =
                    (f4){acc[t][i], acc[t + 1][i], acc[t + 2][i], acc[t + 3][i]} *
                    (1.0f / 32768.0f) * v_run;
    }
    __syncthreads();
    // each thread joins four dims of a row
    for (int e = threadIdx.x; e < 16 * (D / 4); e += 64 * W) {
        const int i = e / (D / 4), d = e % (D / 4) * 4;
        const Row to = row_of(a, c, x, b, head, cu0, n, len, tile * 16 + i);
        if (!to.live) break;  // rows come in order
        float top = neg_inf(), sum = 0.0f;
        for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w * 16 + i]);
        const float at = top == neg_inf() ? 0.0f : top;
        f4 o = {};
        for (int w = 0; w < W; ++w) {
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

typedef float f16v __attribute__((ext_vector_type(16)));

// Scores of 32 keys by the rules, as the exponential takes them: s * by, a
// factor for each 16.  `away`: the row's distance from the lane's first key.
template <typename T, typename R>
__device__ inline void shape_scores(const Shape<T, R>& shape, f16v& s, float* by, float away) {
    if (shape.quick && shape.capped) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            by[u] *= 2.0f * kLog2e;
#pragma unroll
            for (int j = 8 * u; j < 8 * u + 8; ++j) s[j] = shape.cap_quick(s[j] * by[u]);
            by[u] = 2.0f * shape.cap;
        }
    } else if (shape.capped) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int j = 8 * u; j < 8 * u + 8; ++j) s[j] = shape.cap_whole(s[j] * by[u]);
            by[u] = 1.0f;
        }
    }
    if (shape.sloped) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int j = 8 * u; j < 8 * u + 8; ++j)
                s[j] = shape.bend(s[j] * by[u], away - (8 * (j >> 2) + (j & 3)));
            by[u] = 1.0f;
        }
    }
}

// The chunk of keys by which a launch's sequences are cut: the host knows
// only the longest one and left room for `splits` chunks of it; each lane
// tries another chunk that this room allows, and the one whose pieces are done
// first is taken, x.pieces of them at once and a start counted as kStart keys.
constexpr int kStart = 256;

__device__ inline int best_chunk(const AttnRules& x, const CacheQ8& c, const Ragged& r, int lane,
                                 int group, int height, int splits, int step) {
    const int least = ((x.span + splits - 1) / splits + step - 1) & ~(step - 1);
    const int more = (int)min((long long)least * lane / 16, (long long)max(x.span - least, 0));
    const int chunk = (least + more + step - 1) & ~(step - 1);
    int at, count, length = 0, tiles = 0;
    if (lane < r.seqs && ragged_rows(r, lane, at, count, length))
        tiles = ((count * group - 1) / height + 1) * c.heads;
    length = min(length, x.span);
    const float whole = (float)(chunk + kStart), inv = 1.0f / (float)chunk;
    // pieces of a whole chunk; all pieces; keys of those that are not whole
    float full = 0.0f, all = 0.0f, rest = 0.0f;
    for (int i = 0; i < r.seqs; ++i) {
        const float keys = (float)__builtin_amdgcn_readlane(length, i);
        const float times = (float)__builtin_amdgcn_readlane(tiles, i);
        const float n = floorf(keys * inv), left = keys - n * (float)chunk;
        full += times * n;
        rest += left > 0.0f ? times * (left + (float)kStart) : 0.0f;
        all += times * (left > 0.0f ? n + 1.0f : n);
    }
    // rounds of whole chunks with the rest beside them, or where that does
    // not fit what there is in all and a part of a chunk, by which ends differ
    const float at_once = 1.0f / (float)x.pieces;
    const float rounds = fmaxf(ceilf(full * at_once), 1.0f);
    float done = rounds * whole;
    if (all > rounds * (float)x.pieces)
        done = fmaxf(done, (full * whole + rest) * at_once + 0.25f * (float)chunk);
    // (positive: as bits in order; the lane in the last six, so that all agree)
    unsigned cost = (__float_as_uint(done) & ~63u) | (unsigned)lane;
    for (int o = 32; o > 0; o >>= 1) cost = min(cost, (unsigned)__shfl_xor((int)cost, o));
    return __builtin_amdgcn_readlane(chunk, __builtin_amdgcn_readfirstlane((int)(cost & 63u)));
}

// Where chunk `split` starts (past all keys if it is empty: a row sees fewer
// than 2^30).
__device__ inline int chunk_start(int base, int split, int chunk) {
    return (int)min((long long)base + (long long)split * chunk, 1LL << 30);
}

// 16 keys of one page: their scales, as the softmax takes them.
struct alignas(16) Group {
    float ks, vs, lg_vs;  // staged: vs is 1 / the value scale, lg_vs its logarithm
    int on;               // bit 0: some row sees them, bit 1: the value scale is not finite
};

// Many query rows: 32 rows of one cache head a wave, 64 keys a step.  A step's keys and values are brought to float16 once for all
// rows and staged in two LDS buffers, the next step's 8-bit values on their
// way to registers meanwhile.  The products are the same transposed ones on
// v_mfma_f32_32x32x16_f16 (lane 32 g + n holds A[n][8g..8g+7],
// B[8g..8g+7][n], and D[8 (r / 4) + 4 g + r % 4][n] in register r): a query
// row is a column and its probabilities are the next product's operand in
// the key order 16 u + 8 (j / 4) + 4 g + j % 4, in which V is staged too.
//
// LDS: keys as rows of dims, values as rows of keys (transposed on the way
// in: dim d in row d % 4 * (D / 4) + d / 4, so that a wave writes neighbouring
// rows and a lane ends with neighbouring dims).  Rows are 16 bytes longer
// than their contents: 16 of them at one column lie over all the banks.
//
// Bound by vector and matrix instructions in turn: of a step's cycles the
// vector unit is busy 53% and the matrix cores 32%.  Measured, bfloat16:
// 2 x 4096 rows on as many keys, 16 heads of 128, 400-408 us without order
// (675-687 TFLOP/s), 219-225 causal (620); float16 275-286, float32 303-312
// (split operands); heads of 64 146; 8 heads of 256 304-319, float32 462: that
// kernel alone spills, 26 registers a lane to 108 bytes of scratch (with rules
// 2).  Two workgroups of four waves a CU: one of eight shares the staging but
// keeps step, 521 against 427 us.
//
// With rules, prompts of 3849 rows after 2198 tokens and of 3642 after 1120, 12
// heads of 128, bfloat16: a cap and a prefix 335 us (vector unit busy 50%,
// matrix cores 19%), the prefix alone 278, a window of 2401 beside it 253, biases
// alone 311; cap and prefix in float16 376, in float32 567.
template <typename T, int D, typename R>
__global__ __launch_bounds__(64 * kWaves, D <= 128 ? 2 : 1) void attn_q8_many_kernel(AttnQ8 a, CacheQ8 c, Ragged r, R x,
                                                           int splits, int chunk, int tiles,
                                                           float* part) {
    constexpr bool kSplit = sizeof(T) == 4;
    static_assert(kWaves == 4, "a wave for each 16 tokens of a step");
    constexpr int HEIGHT = 32 * kWaves;
    constexpr int HS = kSplit || D > 128 ? 1 : 2;  // halves of a step whose scores are held
    constexpr int KC = D / 16;   // key operands of 16 dims
    constexpr int DT = D / 32;   // output tiles of 32 dims
    constexpr int KLD = D + 8, VLD = 64 + 8;  // row lengths
    __shared__ __align__(16) _Float16 s_k[2][64 * KLD];
    __shared__ __align__(16) _Float16 s_v[2][D * VLD];
    __shared__ Group s_group[2 + 16][4];  // two buffers, and room for writes that do not count
    const int lane = threadIdx.x & 63, wave = wave_id(), n32 = lane & 31, g = lane >> 5;
    // The longest tiles of all sequences and heads first: with causal rows
    // these are the last ones.
    const int pairs = c.heads * r.seqs, pair = blockIdx.x % pairs;
    const int head = pair % c.heads, b = pair / c.heads;
    const int split = blockIdx.x / pairs % splits, tile = tiles - 1 - blockIdx.x / pairs / splits;
    int cu0, n, len;
    if (!ragged_rows(r, b, cu0, n, len)) return;
    const int group = a.q_heads / c.heads, rows = n * group, r0 = tile * HEIGHT;
    if (r0 >= rows) return;
    if constexpr (kRules<R>)
        if (x.pieces) chunk = best_chunk(x, c, r, lane, group, HEIGHT, splits, 64);
    // keys that any of the workgroup's rows sees; bounds grow with the row
    const Row row1 = row_of(a, c, x, b, head, cu0, n, len, min(r0 + HEIGHT - 1, rows - 1));
    const int first = a.first ? max(a.first[b], 0) : 0;
    const int pos0 = len - n + r0 / group;
    const int any_lo = a.window ? max(first, pos0 - a.window + 1) : first, any_hi = row1.hi;
    int base = any_lo < any_hi ? any_lo & ~63 : 0;
    int t_lo = kRules<R> ? chunk_start(base, split, chunk) : base + split * chunk;
    int t_hi = any_lo < any_hi ? min(t_lo + chunk, any_hi) : 0;
    // with a prefix besides the window: keys [first, pre) of all rows, then
    // those from `base` on, counted through
    int pre = 0, in_pre = 0;
    if constexpr (kRules<R>) {
        pre = row1.pre;
        if (first < pre) {
            in_pre = ((pre + 63) & ~63) - (first & ~63);
            base = max(base, (pre + 63) & ~63);
            t_lo = chunk_start(0, split, chunk);
            t_hi = min(t_lo + chunk, in_pre + max(any_hi - base, 0));
        }
    }
    auto key_at = [&](int u) {
        if constexpr (kRules<R>)
            if (first < pre) return u < in_pre ? (first & ~63) + u : base + (u - in_pre);
        return u;
    };
    // keys that this wave's rows see
    const int w0 = min(r0 + 32 * wave, rows - 1), w1 = min(r0 + 32 * wave + 31, rows - 1);
    const Row wrow0 = row_of(a, c, x, b, head, cu0, n, len, w0);
    const Row wrow1 = row_of(a, c, x, b, head, cu0, n, len, w1);
    int all_hi = wrow0.hi;  // every row sees the keys from wrow1.lo to here
    if constexpr (kRules<R>)
        if (x.tree) all_hi = min(all_hi, len - n);
    const bool idle = r0 + 32 * wave >= rows;
    const Row row = row_of(a, c, x, b, head, cu0, n, len, r0 + 32 * wave + n32);

    const auto shape = shape_of<T>(x, row);
    h8 qh[KC], ql[kSplit ? KC : 1];
    float to_log2;  // not negative: the scale's sign goes into the rows; with a cap, over it
    {
        const T* q = (const T*)a.q + (long long)row.tok * a.q_tok + (long long)row.q_head * a.q_head;
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < KC; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf((float)q[16 * j + 8 * g + i]));
        top = max_halves(top);
        const int e = min(max((int)((__float_as_uint(top) >> 23) & 255) - 127, -100), 127);
        const float up = copysignf(__uint_as_float((unsigned)(127 + 14 - e) << 23), a.scale);
        to_log2 = __uint_as_float((unsigned)(127 - 14 + e) << 23) * fabsf(a.scale) * kLog2e;
        if constexpr (kRules<R>)
            if (x.cap > 0.0f)
                to_log2 = shape.held(__uint_as_float((unsigned)(127 - 14 + e) << 23) *
                                     shape.held(fabsf(a.scale) / x.cap));
#pragma unroll
        for (int j = 0; j < KC; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = (float)q[16 * j + 8 * g + i] * up;
                const _Float16 h = (_Float16)v;
                qh[j][i] = h;
                if (kSplit) ql[j][i] = (_Float16)(v - (float)h);
            }
    }

    // Staging: a wave brings 16 of a step's tokens, which lie in one page, so
    // that its addresses are a scalar and a lane's constant; the table entry
    // is read a step ahead of its use.
    constexpr int KJ = D / 64, VJ = (D + 127) / 128;  // pieces a lane
    int entry = 0;
    auto look_up = [&](int t0) { entry = page_entry(c, b, (t0 + 16 * wave) >> c.shift); };
    Words<4> kw[KJ];
    unsigned vw[VJ][8];
    Group next{};
    auto fetch = [&](int t0) {
        const int k0 = t0 + 16 * wave;
        const int page = page_checked(c, k0 >> c.shift, __builtin_amdgcn_readfirstlane(entry));
        const long long at = (long long)max(page, 0) * c.heads + head;
        const long long from = (at * c.page + (k0 & (c.page - 1))) * D;
#pragma unroll
        for (int j = 0; j < KJ; ++j) kw[j] = load_words<4>(c.k + from + (lane + 64 * j) * 16);
#pragma unroll
        for (int j = 0; j < VJ; ++j) {
            const int i = (lane + 64 * j) % (D / 2);
            const int8_t* v = c.v + from + i / (D / 4) * 4 * D + i % (D / 4) * 4;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                vw[j][k] = load_words<1>(v + ((k & 3) + 8 * (k >> 2)) * D).w[0];
        }
        // a group that no row sees may lie in a page that holds anything
        next.on = page >= 0 && k0 < any_hi && k0 + 16 > any_lo;
        if constexpr (kRules<R>) next.on |= page >= 0 && k0 < pre && k0 + 16 > first;
        next.ks = c.k_scale[at];
        next.vs = c.v_scale[at];
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            const int i = lane + 64 * j;
            h8* to = reinterpret_cast<h8*>(s_k[buf] + (16 * wave + i / (D / 16)) * KLD +
                                           i % (D / 16) * 16);
            to[0] = to_half8(kw[j].w[0], kw[j].w[1]);
            to[1] = to_half8(kw[j].w[2], kw[j].w[3]);
        }
#pragma unroll
        for (int j = 0; j < VJ; ++j) {
            const int i = (lane + 64 * j) % (D / 2);  // 64 dims: two lanes do the same
            unsigned lo01[4], hi01[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                lo01[k] = pair_lo(vw[j][2 * k], vw[j][2 * k + 1]);
                hi01[k] = pair_hi(vw[j][2 * k], vw[j][2 * k + 1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h2 x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = to_half2(e < 2 ? lo01[k] : hi01[k],
                                    (e & 1) ? 0x04030402u : 0x04010400u);
                *reinterpret_cast<h8*>(s_v[buf] + (e * (D / 4) + i % (D / 4)) * VLD +
                                       (2 * wave + i / (D / 4)) * 8) =
                    __builtin_bit_cast(h8, x);
            }
        }
        Group to = next;
        to.ks = to.on ? to.ks : 0.0f;
        to.vs = to.on ? to.vs : 0.0f;
        to.on |= finite(to.vs) ? 0 : 2;
        to.lg_vs = finite(to.vs) ? __builtin_amdgcn_logf(to.vs) : neg_inf();
        to.vs = __builtin_amdgcn_rcpf(to.vs);
        // one lane's write counts; the others go aside, so that no branch
        // parts the step
        s_group[lane == 0 ? buf : 2 + (lane >> 2)][lane == 0 ? wave : lane & 3] = to;
    };

    f16v acc[DT] = {};
    float m = neg_inf(), l = 0.0f;
    // The accumulated values are in units of 2^(lg_run - 15), lg_run the
    // largest logarithm of a value scale so far (below every one at first).
    float lg_run = -140.0f;

    // Scores of 32 HS keys; the halves in turn, so that a product does not
    // wait for the one before it.
    auto scores = [&](f16v(&s)[HS], const _Float16* kp) {
#pragma unroll
        for (int h = 0; h < HS; ++h) s[h] = (f16v){};
#pragma unroll
        for (int j = 0; j < KC; ++j)
#pragma unroll
            for (int h = 0; h < HS; ++h) {
                const h8 kv = *reinterpret_cast<const h8*>(kp + 32 * h * KLD + 16 * j);
                s[h] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kv, qh[j], s[h], 0, 0, 0);
                if (kSplit) s[h] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kv, ql[j], s[h], 0, 0, 0);
            }
    };
    auto largest = [&](const f16v& s, float by0, float by1) {
        float top[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            top[u] = s[8 * u];
#pragma unroll
            for (int j = 1; j < 8; ++j) top[u] = fmaxf(top[u], s[8 * u + j]);
        }
        return fmaxf(top[0] * by0, top[1] * by1);
    };
    // The rows' references: the largest score and value scale of the keys that
    // each has seen so far, moved only when a key passes them by so much that
    // p * vs would leave float16 (2^15 at the reference, 2^0.99 above it still
    // fits).
    auto refer = [&](float top, float lg_vs) {
        const float m_new = fmaxf(m, max_halves(top));
        const float lg_new = fmaxf(lg_run, lg_vs);
        if (__any(m_new - m + (lg_new - lg_run) > 0.99f)) {
            const float m_at = m_new == neg_inf() ? 0.0f : m_new;
            const float back = __builtin_amdgcn_exp2f(m - m_at);
            l *= back;
            const float to = back * __builtin_amdgcn_exp2f(lg_run - lg_new);
#pragma unroll
            for (int t = 0; t < DT; ++t) acc[t] *= to;
            m = m_new;
            lg_run = lg_new;
        }
    };
    // Probabilities of 16 keys times their value scale, in the accumulators'
    // units and straight from the exponent; the sum of the probabilities is
    // theirs over the same factor, kept 2^15 times as large: the factor alone
    // would leave float32 for the smallest value scales.
    auto weigh = [&](const f16v& s, int u, float by, const Group& gr, h8& ph, h8& pl) {
        const float m_at = m == neg_inf() ? 0.0f : m;
        const float lift = fmaxf(gr.lg_vs + 15.0f - lg_run, -60.0f) - m_at;
        const float drop = fminf(gr.vs * __builtin_amdgcn_exp2f(lg_run), 0x1p75f);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float x0 = __builtin_amdgcn_exp2f(fmaf(s[8 * u + j], by, lift));
            const float x1 = __builtin_amdgcn_exp2f(fmaf(s[8 * u + j + 1], by, lift));
            sum += x0 + x1;
            const h2 hx = __builtin_convertvector(((f2){x0, x1}), h2);
            ph[j] = hx[0];
            ph[j + 1] = hx[1];
            if (kTwoParts<T>) {
                pl[j] = (_Float16)(x0 - (float)hx[0]);
                pl[j + 1] = (_Float16)(x1 - (float)hx[1]);
            }
        }
        l = fmaf(sum, drop, l);
    };
    auto add_values = [&](const _Float16* vp, const h8& ph, const h8& pl) {
#pragma unroll
        for (int t = 0; t < DT; ++t) {
            const h8 vv = *reinterpret_cast<const h8*>(vp + 32 * t * VLD);
            acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, ph, acc[t], 0, 0, 0);
            if (kTwoParts<T>)
                acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, pl, acc[t], 0, 0, 0);
        }
    };

    if constexpr (kRules<R>)
        if (splits > 1 && t_lo >= t_hi) {  // a chunk without keys
            if (row.live && g == 0) {
                float* pr =
                    part + (((long long)row.tok * a.q_heads + row.q_head) * splits + split) * (D + 4);
                pr[0] = neg_inf();
                pr[1] = 0.0f;
            }
            return;
        }
    if (t_lo < t_hi) {
        look_up(key_at(t_lo));
        fetch(key_at(t_lo));
        look_up(key_at(t_lo + 64));
        stage(0);
        fetch(key_at(t_lo + 64));
        look_up(key_at(t_lo + 128));
        __syncthreads();
        for (int u0 = t_lo, buf = 0; u0 < t_hi; u0 += 64, buf ^= 1) {
            const int t0 = key_at(u0);
            const _Float16* kp = s_k[buf] + n32 * KLD + 8 * g;
            const _Float16* vp = s_v[buf] + n32 * VLD + 8 * g;
            const Group* gp = s_group[buf];
            int seen = t0 >= wrow1.lo && t0 + 64 <= all_hi;  // every row sees every key
            if constexpr (kRules<R>) seen |= t0 >= first && t0 + 64 <= wrow0.pre;
#pragma unroll
            for (int u = 0; u < 4; ++u) seen &= gp[u].on == 1;
            seen = __builtin_amdgcn_readfirstlane(seen);
            // this wave's rows may see none of the step's keys
            bool some = !idle && t0 < wrow1.hi && t0 + 64 > wrow0.lo;
            if constexpr (kRules<R>) some |= !idle && t0 < pre && t0 + 64 > first;
            // (what is staged past the last step is of no use, and harmless)
            if (!some) {
                stage(buf ^ 1);
                fetch(key_at(u0 + 128));
            }
            if (some)
#pragma unroll
                for (int h0 = 0; h0 < 2; h0 += HS) {
                    f16v s[HS];
                    float by[2 * HS], lg_vs[2 * HS], top = neg_inf(), lg = neg_inf();
                    scores(s, kp + 32 * h0 * KLD);
#pragma unroll
                    for (int u = 0; u < 2 * HS; ++u) {
                        if constexpr (kRules<R>)
                            by[u] = shape.by(gp[2 * h0 + u].ks, to_log2);
                        else
                            by[u] = gp[2 * h0 + u].ks * to_log2;
                        lg_vs[u] = gp[2 * h0 + u].lg_vs;
                    }
                    if (h0 == 0) {
                        stage(buf ^ 1);
                        fetch(key_at(u0 + 128));  // a step's time to arrive
                    }
                    if constexpr (kRules<R>) {
#pragma unroll
                        for (int h = 0; h < HS; ++h)
                            shape_scores(shape, s[h], by + 2 * h,
                                         (float)(row.pos - (t0 + 32 * (h0 + h) + 4 * g)));
                    }
                    if (!seen) {
                        // What is hidden from a row goes into its scores, and
                        // a value scale that is not finite too: so it stays
                        // with the rows that see it.  Scales of keys that a
                        // row does not see are not in its reference.
#pragma unroll
                        for (int h = 0; h < HS; ++h) {
                            const int t = t0 + 32 * (h0 + h) + 4 * g;
                            const int lo = row.lo - t, hi = row.hi - t;
                            unsigned keys = 0;
                            if constexpr (kRules<R>)
                                keys = keys_seen(row, x, len - n, t - 4 * g);
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const int at = 8 * (j >> 2) + (j & 3);
                                const int on = gp[2 * (h0 + h) + j / 8].on;
                                const float y = on & 2 ? nan() : s[h][j] * by[2 * h + j / 8];
                                bool sees = at >= lo && at < hi;
                                if constexpr (kRules<R>) sees = keys >> (4 * g) & 1u << at;
                                s[h][j] = on & 1 && sees ? y : neg_inf();
                            }
#pragma unroll
                            for (int u = 2 * h; u < 2 * h + 2; ++u) {
                                const int k0 = t0 + 32 * h0 + 16 * u;
                                by[u] = 1.0f;
                                bool sees = row.lo < k0 + 16 && row.hi > k0;
                                if constexpr (kRules<R>) sees = keys >> (16 * (u & 1)) & 0xffffu;
                                lg_vs[u] = sees ? lg_vs[u] : neg_inf();
                            }
                        }
                    }
#pragma unroll
                    for (int h = 0; h < HS; ++h) {
                        top = fmaxf(top, largest(s[h], by[2 * h], by[2 * h + 1]));
                        lg = fmaxf(lg, fmaxf(lg_vs[2 * h], lg_vs[2 * h + 1]));
                    }
                    refer(top, lg);
#pragma unroll
                    for (int u = 0; u < 2 * HS; ++u) {
                        h8 ph, pl;
                        weigh(s[u / 2], u & 1, by[u], gp[2 * h0 + u], ph, pl);
                        add_values(vp + 32 * h0 + 16 * u, ph, pl);
                    }
                }
            look_up(key_at(u0 + 192));
            __syncthreads();
        }
    }

    l = (l + __shfl_xor(l, 32)) * 0x1p-15f;
    if (!row.live) return;
    if constexpr (kRules<R>)
        if (shape.quick && shape.capped) m += shape.cap;
    const long long out_row = (long long)row.tok * a.q_heads + row.q_head;
    // the unit in two halves, since it may be below float32
    const float half = __builtin_amdgcn_exp2f(0.5f * (lg_run - 15.0f));
    const float by = splits > 1 ? half : l == 0.0f ? 0.0f : half / l;  // a NaN sum stays NaN
    float* pr = part + (out_row * splits + split) * (D + 4);
    // dims 4 p .. 4 p + 3 are in rows p, D / 4 + p, D / 2 + p, 3 D / 4 + p of
    // the stacked output tiles
#pragma unroll
    for (int p8 = 0; p8 < D / 4; p8 += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = e * (D / 4) + p8;
                o[e] = acc[at / 32][at % 32 / 8 * 4 + i] * by * half;
            }
            const int d = 4 * (p8 + 4 * g + i);
            if (splits > 1) {
                *reinterpret_cast<f4*>(pr + 4 + d) = o;
            } else {
                Pack<T, 4> y;
#pragma unroll
                for (int j = 0; j < 4; ++j) y.v[j] = round_to<T>(o[j]);
                *reinterpret_cast<Pack<T, 4>*>((T*)a.out + out_row * D + d) = y;
            }
        }
    if (g == 0) {
        if (splits > 1) {
            pr[0] = m;
            pr[1] = l;
        } else if (a.lse) {
            a.lse[out_row] = lse_of(m, l);
        }
    }
}

constexpr int kMaxSplits = 4224;  // over what the cut below can ask for

// The factor of a chunk with maximum pm and sum pl where the row's maximum is
// `at`.  A chunk without keys has written nothing else than pl = 0; a NaN sum
// stays NaN whatever the maximum (which passes NaN scores by).
__device__ inline float chunk_weight(float pm, float pl, float at) {
    if (pl != pl) return pl;
    return pl == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(pm - at);
}

#include "q8_attn_mid.h"

// The output row of a join's i-th: with rules counted in a sequence (blockIdx.y),
// so that rows of no sequence stay as they were; -1 past the end.
template <typename R>
__device__ inline long long joined_row(const AttnQ8& a, const R&, const Ragged& r, long long i) {
    if constexpr (kRules<R>) {
        int cu0, n, len;
        if (!ragged_rows(r, blockIdx.y, cu0, n, len)) return -1;
        return i < (long long)min(n, r.max_rows) * a.q_heads ? (long long)cu0 * a.q_heads + i : -1;
    } else {
        return i < (long long)r.total * a.q_heads ? i : -1;
    }
}

// Joins the chunks of one output row: first their weights, then the weighted
// sum, a thread for four dims and the chunks dealt to the workgroup's lanes.
template <typename T, int D, typename R>
__global__ __launch_bounds__(512) void attn_q8_join_kernel(AttnQ8 a, R x, Ragged r, int splits,
                                                           const float* __restrict__ part) {
    constexpr int COLS = D / 4, LANES = 512 / COLS;
    __shared__ float s_by[kMaxSplits];
    __shared__ f4 s_out[512];
    __shared__ float s_m[8], s_l[8];
    const long long row = joined_row(a, x, r, blockIdx.x);
    if (row < 0) return;
    const float* pr = part + row * splits * (D + 4);
    float m = neg_inf();
    for (int s = threadIdx.x; s < splits; s += 512) {
        const float pm = pr[(long long)s * (D + 4)];
        s_by[s] = pm;
        m = fmaxf(m, pm);
    }
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if ((threadIdx.x & 63) == 0) s_m[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, s_m[w]);
    const float at = m == neg_inf() ? 0.0f : m;
    float l = 0.0f;
    for (int s = threadIdx.x; s < splits; s += 512) {
        const float pl = pr[(long long)s * (D + 4) + 1], by = chunk_weight(s_by[s], pl, at);
        s_by[s] = by;
        l += by == 0.0f ? 0.0f : by * pl;
    }
    l = wave_sum(l);
    if ((threadIdx.x & 63) == 0) s_l[threadIdx.x >> 6] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) l += s_l[w];
    const int col = threadIdx.x % COLS;
    f4 o = {};
#pragma unroll 4
    for (int s = threadIdx.x / COLS; s < splits; s += LANES) {
        const float by = s_by[s];
        f4 x = *reinterpret_cast<const f4*>(pr + (long long)s * (D + 4) + 4 + 4 * col);
        if (by == 0.0f) x = (f4){};
        o += by * x;
    }
    s_out[threadIdx.x] = o;
    __syncthreads();
    if (threadIdx.x >= COLS) return;
#pragma unroll
    for (int k = 1; k < LANES; ++k) o += s_out[k * COLS + col];
    const float by = l == 0.0f ? 0.0f : 1.0f / l;
    Pack<T, 4> y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y.v[j] = round_to<T>(o[j] * by);
    *reinterpret_cast<Pack<T, 4>*>((T*)a.out + row * D + 4 * col) = y;
    if (a.lse && col == 0) a.lse[row] = lse_of(m, l);
}

// The same for up to 64 chunks, a wave a row: a lane for a chunk's weight,
// then for four dims of some of them.
template <typename T, int D, typename R>
__global__ __launch_bounds__(256) void attn_q8_join_few_kernel(AttnQ8 a, R x, Ragged r, int splits,
                                                               const float* __restrict__ part) {
    constexpr int COLS = D / 4, LANES = 64 / COLS;
    const int lane = threadIdx.x & 63;
    const long long row = joined_row(a, x, r, blockIdx.x * 4LL + wave_id());
    if (row < 0) return;
    const float* pr = part + row * splits * (D + 4);
    float m = neg_inf(), l = 0.0f;
    if (lane < splits) {
        m = pr[(long long)lane * (D + 4)];
        l = pr[(long long)lane * (D + 4) + 1];
    }
    float top = m;
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    const float at = top == neg_inf() ? 0.0f : top;
    const float by = chunk_weight(m, l, at);
    l = wave_sum(by == 0.0f ? 0.0f : by * l);
    const int col = lane % COLS;
    f4 o = {};
    for (int s0 = 0; s0 < splits; s0 += LANES) {
        // (every lane takes part in the exchange, those past the last chunk too)
        const int s = s0 + lane / COLS;
        const float from = __shfl(by, min(s, splits - 1)), w = s < splits ? from : 0.0f;
        if (w != 0.0f)
            o += w * *reinterpret_cast<const f4*>(pr + (long long)s * (D + 4) + 4 + 4 * col);
    }
    for (int i = COLS; i < 64; i <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += __shfl_xor(o[j], i);
    if (lane >= COLS) return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    Pack<T, 4> y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y.v[j] = round_to<T>(o[j] * inv);
    *reinterpret_cast<Pack<T, 4>*>((T*)a.out + row * D + 4 * col) = y;
    if (a.lse && col == 0) a.lse[row] = lse_of(top, l);
}

// How the rows are tiled and the keys of a tile cut.  The lengths are on the
// device, so this goes by the longest; chunks past a sequence's end are
// empty.
struct Cut {
    bool many;  // the kernel for many rows
    bool mid;   // the one for drafts
    bool wide;  // the one for few rows (drafts), with wide_waves (mid_wide_waves)
    int tiles, splits, chunk;
    int span;    // keys of one row tile at most, from an aligned start
    int pieces;  // few rows: chunks in all to aim at, 0 for the chunk as it is
};

inline int round_up_to(long long x, int step) { return (int)((x + step - 1) / step * step); }

inline Cut cut(int seqs, int max_rows, int max_len, int q_heads, int heads, int dim, int elem,
               int window, int prefix, bool rules) {
    const int group = q_heads / heads;
    const long long rows = (long long)max_rows * group;
    Cut r;
    // Either side of the limit, few / many rows' kernel in us, bfloat16, 12
    // over 4 heads of 128: [1 x 2400 keys] 30 rows 15.6 / 16.9, 33 rows 15.8 /
    // 17.1, 63 rows 20.6 / 18.4; [1 x 24000] 31 / 25, 30 / 25, 40 / 28; [64 x
    // 4000] 100 / 102, 116 / 105, 136 / 107.  (float32 would stay with the
    // first up to about 64 rows: [64 x 4000], 33 rows, 112 / 149.)
    r.many = rows > 32;
    // With rules, the kernel for drafts between them.  This one / the others in
    // us on the device, bfloat16, 12 over 4 heads of 128, drafts of one size:
    // [16 x 12000 keys] 24 rows 51 / 82, 48 rows 71 / 76, 96 rows 91 / 89, 192
    // rows 154 / 147; [64 x 4000] 24 rows 67 / 99, 96 rows 126 / 116; [16 x 500
    // to 24000] 48 rows 91 / 132, 96 rows 130 / 144, 192 rows 204 / 257, drafts
    // of 99 to 192 rows 166 / 211; [16 x 12000], 96 rows of heads of 64 69 / 67,
    // of 256 176 / 255, float32 117 / 119.  From 96 rows on this one is ahead
    // where the lengths differ (by up to a quarter) and behind where they are
    // equal (up to a twelfth), which the host does not see.
    r.mid = rules && rows > 16 && rows <= 192;
    const int height = r.mid ? 32 : r.many ? 32 * kWaves : 16;
    const int step = r.many && !r.mid ? 64 : 32 * kWaves;
    r.tiles = (int)((rows + height - 1) / height);
    r.span = max_len;
    if (window > 0)
        r.span = (int)std::min<long long>(
            r.span, (long long)window + height / group + 65 + (prefix > 0 ? prefix + 126LL : 0));
    const long long pairs = (long long)seqs * heads * r.tiles;
    r.pieces = 0;
    // With rules and few rows, larger workgroups that take all keys of theirs
    // where that is two steps, or where there is nearly one for every CU: no
    // second launch joins chunks.  Whole / split, us for a call, bfloat16, 12
    // over 4 heads of 128: [1 x 300 keys] 15.0 / 19.5, [1 x 700] 15.4 / 19.3,
    // [1 x 1500] 21.0 / 19.4, [32 x 1500] 22.3 / 22.0; on the device [64 x 1500]
    // 25 / 31, [64 x 6000] 82 / 90, [64 x 1000 to 2000] 28 / 36, [64 x 200 to
    // 6000] 54 / 60, but [64 x 200 to 24000] 209 / 200 and one of 24000 among 63
    // of 500 171 / 98: the longest sequence sets the time, and the lengths are
    // not known here.
    const int wide = r.mid ? mid_wide_waves(dim) : wide_waves(dim, elem);
    r.wide = rules && (r.mid || !r.many) && pairs <= 256 && r.span > step &&
             (r.span <= 64 * wide || (!r.mid && pairs >= 192));
    if (r.wide) {
        r.chunk = round_up_to(r.span, 32 * wide);
        r.splits = 1;
        return r;
    }
    if (r.mid) {
        // One resident round ([16 x 500 to 24000 keys], drafts of 99 to 192
        // rows: 184 us when measured; two workgroups a CU 193, four 196).
        const int resident = 256 * mid_residency(dim);
        r.chunk = std::max(round_up_to((r.span * pairs + resident - 1) / resident, step), step);
        if (seqs > 1 && seqs <= 64) r.pieces = resident;
    } else if (r.many && rules && r.tiles <= 4) {
        // Drafts over long sequences: cut so that two workgroups a CU have
        // work to the end ([16 x 500 to 24000 keys], drafts of 99 to 192 rows:
        // 315 us cut by the longest sequence alone, 225 so, when measured).
        const int resident = 512;
        r.chunk = std::max(round_up_to((r.span * pairs + resident - 1) / resident, step), 256);
        if (seqs > 1 && seqs <= 64) r.pieces = resident;
    } else if (r.many) {
        // Split only to give every CU a workgroup, in chunks of 128 keys or
        // more: the joined parts are float32 rows ([4 x 512 rows, 1000 keys,
        // 12 heads], 192 workgroups: 43 us whole, 52 in two parts; [5 x 17
        // rows, window 513, 2 heads], 20 workgroups: 26 whole, 21 in four).
        const long long parts = std::max(std::min(256 / pairs, (long long)r.span / 128), 1LL);
        r.chunk = std::max(round_up_to((r.span + parts - 1) / parts, step), step);
    } else {
        // One resident round of workgroups: every one pays for its start
        // ([64 x 12000 keys, 4 heads of 128]: 1024 chunks 151 us, 2048 156,
        // 4096 169).
        const int resident = 256 * few_residency(dim, elem);
        r.chunk = std::max(round_up_to((r.span * pairs + resident - 1) / resident, step), step);
        if (seqs > 1 && seqs <= 1024) r.pieces = resident;
    }
    r.chunk = std::min(r.chunk, std::max(round_up_to(r.span, step), step));
    r.splits = std::max((r.span + r.chunk - 1) / r.chunk, 1);
    if (r.pieces)  // room for chunks half as long where lengths differ
        r.splits = std::max(std::min(2 * r.splits, (r.span + step - 1) / step), 1);
    return r;
}

// Workgroups of the kernel for drafts: a number for each XCD, the tiles of
// one sequence, head and chunk on the same.
inline long long mid_blocks(const Cut& k, int heads, int seqs) {
    return ((long long)k.splits * heads * seqs + 7) / 8 * 8 * k.tiles;
}

// Which join: a wave a row wants rows for the CUs ([1 x 2400 keys, 12 heads]
// takes 15.6 us with it, 13.5 with a workgroup a row).
inline bool join_by_waves(int splits, long long rows) { return splits <= 64 && rows >= 2048; }

template <typename T, int D, typename R>
hipError_t run(const AttnQ8& a, R x, const CacheQ8& c, const Ragged& r, float* part,
               hipStream_t stream) {
    int prefix = 0;
    if constexpr (kRules<R>) prefix = x.prefix ? x.max_prefix : 0;
    const Cut k = cut(r.seqs, r.max_rows, a.max_len, a.q_heads, c.heads, D, sizeof(T), a.window,
                      prefix, kRules<R>);
    const long long blocks = (long long)k.tiles * k.splits * c.heads * r.seqs;
    if constexpr (kRules<R>) {
        x.pieces = k.pieces;
        x.span = k.span;
    }
    bool launched = false;
    if constexpr (kRules<R>) {
        launched = k.mid || k.wide;
        const dim3 grid((unsigned)(k.mid ? mid_blocks(k, c.heads, r.seqs) : blocks));
        constexpr int W = wide_waves(D, sizeof(T)), MW = mid_wide_waves(D);
        if (k.mid && k.wide)
            hipLaunchKernelGGL((attn_q8_mid_kernel<T, D, R, MW>), grid, dim3(64 * MW), 0, stream, a, c,
                               r, x, k.splits, k.chunk, k.tiles, part);
        else if (k.mid)
            hipLaunchKernelGGL((attn_q8_mid_kernel<T, D, R, kWaves>), grid, dim3(64 * kWaves), 0,
                               stream, a, c, r, x, k.splits, k.chunk, k.tiles, part);
        else if (k.wide)
            hipLaunchKernelGGL((attn_q8_few_kernel<T, D, R, W>), grid, dim3(64 * W), 0, stream, a,
                               c, r, x, k.splits, k.chunk, k.span, k.pieces, c.heads * k.tiles,
                               part);
    }
    if (launched)
        ;
    else if (k.many)
        hipLaunchKernelGGL((attn_q8_many_kernel<T, D, R>),
                           dim3((unsigned)blocks),
                           dim3(64 * kWaves), 0, stream, a, c, r, x, k.splits, k.chunk, k.tiles, part);
    else
        hipLaunchKernelGGL((attn_q8_few_kernel<T, D, R, kWaves>),
                           dim3((unsigned)blocks),
                           dim3(64 * kWaves), 0, stream, a, c, r, x, k.splits, k.chunk, k.span,
                           k.pieces, c.heads * k.tiles, part);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && k.splits > 1) {
        const long long rows = (long long)r.total * a.q_heads;
        const long long each = kRules<R> ? (long long)r.max_rows * a.q_heads : rows;
        const unsigned seqs = kRules<R> ? r.seqs : 1;
        if (join_by_waves(k.splits, rows))
            hipLaunchKernelGGL((attn_q8_join_few_kernel<T, D, R>),
                               dim3((unsigned)((each + 3) / 4), seqs), dim3(256), 0, stream, a, x,
                               r, k.splits, part);
        else
            hipLaunchKernelGGL((attn_q8_join_kernel<T, D, R>), dim3((unsigned)each, seqs),
                               dim3(512), 0, stream, a, x, r, k.splits, part);
        e = hipGetLastError();
    }
    return e;
}

template <typename T, typename R>
hipError_t attn_q8(const AttnQ8& a, const R& x, const CacheQ8& c, const Ragged& r, float* part,
                   hipStream_t stream) {
    if (c.dim == 64) return run<T, 64>(a, x, c, r, part, stream);
    if (c.dim == 128) return run<T, 128>(a, x, c, r, part, stream);
    return run<T, 256>(a, x, c, r, part, stream);
}

template <typename R>
hipError_t launch_attn(int dtype, const AttnQ8& a, const R& x, const CacheQ8& c, const Ragged& r,
                       void* ws, const char* name, hipStream_t stream) {
    prof_pre(stream);
    float* part = (float*)ws;
    hipError_t e = hipErrorInvalidValue;
    if (dtype == AVAE_BF16)
        e = attn_q8<__bf16>(a, x, c, r, part, stream);
    else if (dtype == AVAE_F16)
        e = attn_q8<_Float16>(a, x, c, r, part, stream);
    else if constexpr (!std::is_same<R, FineRules>::value)
        e = attn_q8<float>(a, x, c, r, part, stream);
    // lengths are on the device: counted as if every row saw max_len keys
    const double pairs = (double)r.total * a.q_heads * a.max_len;
    prof_post(stream, name, 4.0 * pairs * c.dim,
              2.0 * r.seqs * (double)a.max_len * c.heads * c.dim);
    return e;
}

}  // namespace
}  // namespace avae
