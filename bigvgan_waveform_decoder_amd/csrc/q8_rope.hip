// Heads turned by their position: the RMS norm of each query and key head
// with the rotation in the same pass, and the write into the 8-bit paged cache
// with norm and rotation on the way.
//
// The first `rot` dims of a head are rot / 2 pairs (a, b): dims (i, i + rot/2)
// or, interleaved, (2 i, 2 i + 1).  At position p pair i becomes
//   a' = amp (a cos(p f_i) - b sin(p f_i)),  b' = amp (b cos + a sin).
// With a weight, x is x / sqrt(mean x^2 + eps) * weight before that.
//
// The angle is taken in 64 bits: p f_i loses whole turns in 32 for far
// positions.  Quarter turns d = p (2 f_i / pi) are split into rint(d) (whose
// low two bits choose the quadrant) and a rest in [-1/2, 1/2], exact in 64
// bits; cosine and sine of the rest are Taylor sums: with the rest's rounding
// to float32 under 4 2^-24 off.
#include <algorithm>
#include <type_traits>

#include "avae.h"
#include "avae_internal.h"
#include "q8.h"

namespace avae {
namespace {

using namespace q8;

constexpr int kThreads = 256;

// P pairs of a head, which a lane holds.
template <int P, typename T = float>
struct Pairs {
    T a[P], b[P];
};

// How a lane's pairs lie: as two runs of P, the a's and the b's; as 2 P
// neighbours; or anyhow, one by one, where a head or its turned part is
// shorter than a run.  The dims that are not turned are pairs too, the first
// half of them with the second.
enum Lie { kRuns, kNeighbours, kAnyhow };

inline Lie lie_of(const RopeQ8& r, int dim, int pairs) {
    if (r.half > 0 && r.apart == 0) return dim >= 2 * pairs ? kNeighbours : kAnyhow;
    const int rest = dim / 2 - r.half;
    const bool whole = (r.half == 0 || r.half >= pairs) && (rest == 0 || rest >= pairs);
    return whole && (r.half + pairs - 1) / pairs + (rest + pairs - 1) / pairs <= 64 ? kRuns
                                                                                    : kAnyhow;
}

// Lanes that a head takes.
inline int lanes_of(const RopeQ8& r, int dim, int pairs, Lie lie) {
    const int parts = lie == kRuns ? (r.half + pairs - 1) / pairs +
                                         (dim / 2 - r.half + pairs - 1) / pairs
                                   : (dim + 2 * pairs - 1) / (2 * pairs);
    int lanes = 1;
    while (lanes < parts) lanes *= 2;
    return lanes;
}

// A lane's place in its head.  Runs are whole: where the last one of a part
// would pass its end it starts earlier, and its first `seen` pairs are the
// lane's before, too, which then both make and write.
template <int P, Lie LIE>
struct Place {
    int a, b;    // dims of the first pair
    int pair;    // its number
    int turned;  // how many are turned
    int seen;
    bool on;

    __device__ Place(const RopeQ8& r, int dim, int j) {
        const int pairs = dim / 2;
        if constexpr (LIE == kRuns) {
            const int lanes = (r.half + P - 1) / P;
            const bool far = j < lanes;
            const int first = far ? 0 : r.half, end = far ? r.half : pairs;
            const int at = first + P * (far ? j : j - lanes);
            on = at < end;
            pair = min(at, end - P);
            seen = on ? at - pair : P;
            turned = far ? P : 0;
            a = far ? pair : r.half + pair;
            b = a + (far ? r.half : pairs - r.half);
        } else {
            on = P * j < pairs;
            pair = LIE == kNeighbours ? min(P * j, pairs - P) : P * j;
            seen = on ? P * j - pair : P;
            turned = min(max(r.half - pair, 0), P);
            a = 2 * pair;
            b = 0;
        }
    }
};

// Dims of pair p where they lie anyhow.
__device__ inline int dim_a(int p, const RopeQ8& r) {
    return r.apart == 0 ? 2 * p : p < r.half ? p : r.half + p;
}
__device__ inline int dim_b(int p, const RopeQ8& r, int dim) {
    return r.apart == 0 ? 2 * p + 1 : p < r.half ? p + r.half : dim / 2 + p;
}

// The lane's pairs of a head, as they are stored.
template <int P, Lie LIE, typename T>
__device__ inline Pairs<P, T> load_pairs(const T* x, const Place<P, LIE>& at, const RopeQ8& r,
                                         int dim) {
    Pairs<P, T> f;
    if constexpr (LIE == kRuns) {
        __builtin_memcpy(f.a, x + at.a, sizeof(f.a));
        __builtin_memcpy(f.b, x + at.b, sizeof(f.b));
    } else if constexpr (LIE == kNeighbours) {
        T v[2 * P];
        __builtin_memcpy(v, x + at.a, sizeof(v));
#pragma unroll
        for (int e = 0; e < P; ++e) {
            f.a[e] = v[2 * e];
            f.b[e] = v[2 * e + 1];
        }
    } else {
#pragma unroll
        for (int e = 0; e < P; ++e) {
            const bool in = at.pair + e < dim / 2;
            f.a[e] = in ? x[dim_a(at.pair + e, r)] : (T)0.0f;
            f.b[e] = in ? x[dim_b(at.pair + e, r, dim)] : (T)0.0f;
        }
    }
    return f;
}

template <int P, Lie LIE, typename T>
__device__ inline void store_pairs(T* x, const Place<P, LIE>& at, const RopeQ8& r, int dim,
                                   const Pairs<P>& f) {
    if constexpr (LIE == kRuns) {
        store_values<P>(x + at.a, P, f.a);
        store_values<P>(x + at.b, P, f.b);
    } else if constexpr (LIE == kNeighbours) {
        float v[2 * P];
#pragma unroll
        for (int e = 0; e < P; ++e) {
            v[2 * e] = f.a[e];
            v[2 * e + 1] = f.b[e];
        }
        store_values<2 * P>(x + at.a, 2 * P, v);
    } else {
#pragma unroll
        for (int e = 0; e < P; ++e)
            if (at.pair + e < dim / 2) {
                x[dim_a(at.pair + e, r)] = round_to<T>(f.a[e]);
                x[dim_b(at.pair + e, r, dim)] = round_to<T>(f.b[e]);
            }
    }
}

// Four pairs in 8 bits (bytes: those of the a's, those of the b's).
template <Lie LIE>
__device__ inline void store_pair_bytes(int8_t* x, const Place<4, LIE>& at, const RopeQ8& r,
                                        int dim, unsigned a, unsigned b) {
    if constexpr (LIE == kRuns) {
        __builtin_memcpy(x + at.a, &a, 4);
        __builtin_memcpy(x + at.b, &b, 4);
    } else if constexpr (LIE == kNeighbours) {
        const unsigned w[2] = {__builtin_amdgcn_perm(b, a, 0x05010400u),
                               __builtin_amdgcn_perm(b, a, 0x07030602u)};
        __builtin_memcpy(x + at.a, w, 8);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[dim_a(at.pair + e, r)] = (int8_t)(a >> (8 * e));
            x[dim_b(at.pair + e, r, dim)] = (int8_t)(b >> (8 * e));
        }
    }
}

template <int P, typename T>
__device__ inline Pairs<P> as_floats(const Pairs<P, T>& r) {
    Pairs<P> f;
#pragma unroll
    for (int e = 0; e < P; ++e) {
        f.a[e] = (float)r.a[e];
        f.b[e] = (float)r.b[e];
    }
    return f;
}

// Quarter turns a position of a frequency.
__device__ inline double quarters(float freq) { return (double)freq * 0.63661977236758134308; }

// amp cos and amp sin of a pair at a position.
__device__ inline void angle(int pos, double quarter, float amp, float& c, float& s) {
    // adding 1.5 * 2^52 leaves the nearest whole number in the low bits
    constexpr double kRound = 6755399441055744.0;
    const double d = (double)pos * quarter;
    const double t = d + kRound;
    const int quadrant = (int)__double2loint(t);
    const float x = (float)(d - (t - kRound)) * 1.57079632679489662f;
    const float z = x * x;
    float sn = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
    sn = fmaf(z, sn, 8.3333333e-3f);
    sn = fmaf(z, sn, -1.6666667e-1f);
    sn = fmaf(x * z, sn, x);
    float cs = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
    cs = fmaf(z, cs, -1.3888889e-3f);
    cs = fmaf(z, cs, 4.1666667e-2f);
    cs = fmaf(z, cs, -0.5f);
    cs = fmaf(z, cs, 1.0f);
    const float co = (quadrant & 1) ? sn : cs, si = (quadrant & 1) ? cs : sn;
    c = (((quadrant + 1) & 2) ? -co : co) * amp;
    s = ((quadrant & 2) ? -si : si) * amp;
}

// Turns the first `turned` pairs.  (The others are left alone: 0 times an
// infinity is NaN.)
template <int P>
__device__ inline void turn(Pairs<P>& r, int turned, const float (&c)[P], const float (&s)[P]) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
        const float a = r.a[e], b = r.b[e];
        r.a[e] = e < turned ? fmaf(a, c[e], -b * s[e]) : a;
        r.b[e] = e < turned ? fmaf(b, c[e], a * s[e]) : b;
    }
}

// x / sqrt(mean x^2 + eps) * weight over a head that `lanes` neighbouring
// lanes hold, the first `seen` pairs of this one counted elsewhere.  Squares
// that leave float32's range are summed in 64 bits; a head of zeros stays
// zeros.
template <int P>
__device__ inline void norm(Pairs<P>& r, const Pairs<P>& w, int seen, int lanes, float per_dim,
                            float eps) {
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < P; ++e) {
        const float to = fmaf(r.a[e], r.a[e], fmaf(r.b[e], r.b[e], sum));
        sum = e < seen ? sum : to;
    }
    for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor(sum, o);
    if (sum >= 1e-24f && sum < 1e37f) {  // (a smaller one has squares below 2^-126 in it)
        const float by = __builtin_amdgcn_rsqf(fmaf(sum, per_dim, eps));
#pragma unroll
        for (int e = 0; e < P; ++e) {
            r.a[e] = r.a[e] * by * w.a[e];
            r.b[e] = r.b[e] * by * w.b[e];
        }
        return;
    }
    double all = 0.0;
#pragma unroll
    for (int e = 0; e < P; ++e)
        if (e >= seen) all += (double)r.a[e] * (double)r.a[e] + (double)r.b[e] * (double)r.b[e];
    for (int o = 1; o < lanes; o <<= 1) all += __shfl_xor(all, o);
    const double by = all == 0.0 ? 0.0 : 1.0 / sqrt(all * (double)per_dim + (double)eps);
#pragma unroll
    for (int e = 0; e < P; ++e) {
        r.a[e] = (float)((double)r.a[e] * by * (double)w.a[e]);
        r.b[e] = (float)((double)r.b[e] * by * (double)w.b[e]);
    }
}

constexpr int kMaxPairs = 256;  // of a head

// A wave takes 64 / lanes heads of a token, each in `lanes` neighbouring
// lanes, and goes on to other tokens with the same heads.  Its lanes share the
// angles: each takes one pair (or few), and they are exchanged through LDS, in
// this wave's own corner.  The next token's heads are on their way meanwhile.
//
// Bound by memory: every value is read and written once.  17254 tokens of 16
// heads of 128 in bfloat16 take 26 us, 5.5 TB/s (half of what is read comes from
// the last-level cache; vector unit busy 53%; 47 with 8-byte loads and each
// lane's angles made for itself); with 50 dims turned, which no run divides, 38
// in runs that overlap, 104 one by one: 9 lanes of a head's 16 have work there,
// 8 of 8 where all is turned.
template <typename T, int P, Lie LIE>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(HeadsQ8 q, HeadsQ8 k, RopeQ8 rope,
                                                                Ragged r, int dim, float eps,
                                                                int lanes, int parts) {
    __shared__ __align__(16) float s_cos[kThreads / 64][kMaxPairs + P];
    __shared__ __align__(16) float s_sin[kThreads / 64][kMaxPairs + P];
    const int b = blockIdx.y, lane = threadIdx.x & 63, wave = wave_id();
    int cu0 = 0, n = r.total, start = 0;
    if (r.cu) {
        int len;
        if (!ragged_rows(r, b, cu0, n, len)) return;
        start = len - n;
    }
    // a wave keeps its heads: the first waves take the first ones
    const int waves = gridDim.x * (kThreads / 64), id = blockIdx.x * (kThreads / 64) + wave;
    const int strides = waves / parts, part = id / strides;
    if (part >= parts) return;
    const Place<P, LIE> at(rope, dim, lane & (lanes - 1));
    const int h = part * (64 / lanes) + lane / lanes;
    const bool is_q = h < q.heads, on = at.on && h < q.heads + k.heads;
    const int head = is_q ? h : h - q.heads;
    const T* from = (const T*)(is_q ? q.x : k.x) + head * (is_q ? q.head : k.head);
    T* to = (T*)(is_q ? q.y : k.y) + head * (is_q ? q.y_head : k.y_head);
    const long long from_tok = is_q ? q.tok : k.tok, to_tok = is_q ? q.y_tok : k.y_tok;
    const float* weight = is_q ? q.weight : k.weight;
    const bool normed = weight != nullptr && h < q.heads + k.heads;
    const float per_dim = 1.0f / (float)dim;
    Pairs<P> w{};
    if (on && normed) w = load_pairs(weight, at, rope, dim);
    double quarter[kMaxPairs / 64];
#pragma unroll
    for (int e = 0; e < kMaxPairs / 64; ++e)
        quarter[e] = lane + 64 * e < rope.half ? quarters(rope.freq[lane + 64 * e]) : 0.0;

    Pairs<P, T> next{};
    int pos = 0;
    auto fetch = [&](int i) {
        if (i >= n) return;
        pos = rope.positions ? rope.positions[cu0 + i] : start + i;
        if (on) next = load_pairs(from + (long long)(cu0 + i) * from_tok, at, rope, dim);
    };
    int i = id - part * strides;
    fetch(i);
    for (; i < n; i += strides) {
        // the angles, to each lane those of its pairs
#pragma unroll
        for (int e = 0; e < kMaxPairs / 64; ++e)
            if (64 * e < rope.half)
                angle(pos, quarter[e], rope.amp, s_cos[wave][lane + 64 * e],
                      s_sin[wave][lane + 64 * e]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        float c[P] = {}, s[P] = {};
        if (at.turned > 0) {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                c[e] = s_cos[wave][at.pair + e];
                s[e] = s_sin[wave][at.pair + e];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        Pairs<P> x = as_floats(next);
        fetch(i + strides);
        if (normed) norm(x, w, on ? at.seen : P, lanes, per_dim, eps);
        turn(x, at.turned, c, s);
        if (on) store_pairs(to + (long long)(cu0 + i) * to_tok, at, rope, dim, x);
    }
}

// One page of one head, keys or values, as the cache's write has it: HELD
// groups of eight values a thread stay in registers between the pass for the
// maximum and the one that rounds; HELD 0 (larger pages) makes them twice.
//
// The scale is of what is stored, so the page is turned before its maximum is
// known, in float32: nothing is rounded between.  Bound by vector instructions,
// the angles' (the unit is busy 85%): prompts of 16 heads of 64 in float32, 126
// MB in all, take 32 us (3.9 TB/s), the same rows written as they are 24.  One
// workgroup for the keys of 2 to 16 heads, which makes their angles once, takes
// 33 to 43: it has its heads after one another, and there are fewer workgroups
// to hide that.
template <typename T, int HELD, Lie LIE>
__global__ __launch_bounds__(kThreads) void kv_write_rope_q8_kernel(
    const T* __restrict__ k, long long k_tok, long long k_head, const T* __restrict__ v,
    long long v_tok, long long v_head, const float* __restrict__ weight, float eps, RopeQ8 rope,
    CacheQ8 c, Ragged r, int lanes) {
    __shared__ unsigned s_max[kThreads / 64];
    const int b = blockIdx.z, head = blockIdx.y >> 1, is_v = blockIdx.y & 1;
    int cu0, n, len;
    if (!ragged_rows(r, b, cu0, n, len)) return;
    const int start = len - n;  // a start below 0 leaves the first tokens out
    const int col = (max(start, 0) >> c.shift) + blockIdx.x;
    if ((long long)col * c.page >= len) return;
    const int page = page_of(c, b, col);
    if (page < 0) return;
    const int p0 = col * c.page;
    const int lo = max(max(start, 0), p0) - p0;  // first new slot of this page
    const int hi = min(len, p0 + c.page) - p0;   // one past the last
    const long long x_tok = is_v ? v_tok : k_tok;
    const long long tok0 = (long long)cu0 + p0 - start;  // the packed row of the page's slot 0
    const T* x = (is_v ? v : k) + (is_v ? v_head : k_head) * head + tok0 * x_tok;
    const long long at = (long long)page * c.heads + head;
    int8_t* q = (is_v ? c.v : c.k) + at * c.page * c.dim;
    float* scales = is_v ? c.v_scale : c.k_scale;

    const int shift = __builtin_ctz(lanes);
    const Place<4, LIE> place(rope, c.dim, threadIdx.x & (lanes - 1));
    const int i0 = lo * lanes + threadIdx.x, i1 = hi * lanes;
    const float per_dim = 1.0f / (float)c.dim;
    double quarter[4] = {};
    Pairs<4> w{};
    if (!is_v && place.on) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < place.turned) quarter[e] = quarters(rope.freq[place.pair + e]);
        if (weight) w = load_pairs(weight, place, rope, c.dim);
    }
    // (values lie as the keys, and stay so)
    auto load = [&](int i, Pairs<4>& f) {
        f = Pairs<4>{};
        if (place.on) f = as_floats(load_pairs(x + (i >> shift) * x_tok, place, rope, c.dim));
    };
    auto make = [&](int i, Pairs<4>& f) {
        if (is_v) return;
        if (weight) norm(f, w, place.seen, lanes, per_dim, eps);
        if (rope.half) {
            const int slot = i >> shift;
            const int pos = rope.positions ? rope.positions[tok0 + slot] : p0 + slot;
            float cs[4], sn[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) angle(pos, quarter[e], rope.amp, cs[e], sn[e]);
            turn(f, place.turned, cs, sn);
        }
    };
    auto most = [&](const Pairs<4>& f, unsigned top) {
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(mag_bits(f.a[e]), mag_bits(f.b[e])));
        return top;
    };
    Pairs<4> held[HELD ? HELD : 1];
    unsigned top = 0;
    if constexpr (HELD > 0) {
#pragma unroll
        for (int t = 0; t < HELD; ++t)
            if (i0 + t * kThreads < i1) load(i0 + t * kThreads, held[t]);
#pragma unroll
        for (int t = 0; t < HELD; ++t)
            if (i0 + t * kThreads < i1) {
                make(i0 + t * kThreads, held[t]);
                top = most(held[t], top);
            }
    } else {
        for (int i = i0; i < i1; i += kThreads) {
            load(i, held[0]);
            make(i, held[0]);
            top = most(held[0], top);
        }
    }
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = top;
    const float was = lo > 0 ? scales[at] : 0.0f;
    __syncthreads();  // also: every thread has the old scale before it changes
    for (int i = 0; i < kThreads / 64; ++i) top = max(top, s_max[i]);
    const float fresh = scale_of(top);
    // a NaN on either side stays
    const float s = (was != was || fresh != fresh) ? __uint_as_float(0x7fc00000u)
                                                   : fmaxf(was, fresh);
    if (threadIdx.x == 0) scales[at] = s;
    const Quantiser quant(s);
    auto bytes = [&](const float(&f)[4]) {
        return to_bytes(quant.quotient(f[0]), quant.quotient(f[1]), quant.quotient(f[2]),
                        quant.quotient(f[3]));
    };
    if (lo > 0 && s > was)  // what the page held moves to the new range
        for (int i = threadIdx.x; i < lo * (c.dim / 4); i += kThreads) {
            float f[4];
            load_stored<4>(q + 4 * i, 4, f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] *= was;
            reinterpret_cast<unsigned*>(q)[i] = bytes(f);
        }
    auto store = [&](int i, const Pairs<4>& f) {
        if (place.on)
            store_pair_bytes(q + (long long)(i >> shift) * c.dim, place, rope, c.dim, bytes(f.a),
                             bytes(f.b));
    };
    if constexpr (HELD > 0) {
#pragma unroll
        for (int t = 0; t < HELD; ++t)
            if (i0 + t * kThreads < i1) store(i0 + t * kThreads, held[t]);
    } else {
        for (int i = i0; i < i1; i += kThreads) {
            load(i, held[0]);
            make(i, held[0]);
            store(i, held[0]);
        }
    }
}

constexpr int kWavesInAll = 256 * 40;

// A thread a draft: it follows its line of parents back and sets their bits.
// A parent comes before its child, so the line goes down and each word is
// written once.  Bound by the latency of a line's parents, one after another:
// 2.8 us for lines of up to 13 drafts.
__global__ __launch_bounds__(kThreads) void tree_mask_kernel(const int* __restrict__ parents,
                                                             Ragged r, int words,
                                                             unsigned* __restrict__ mask,
                                                             long long ld,
                                                             int* __restrict__ positions) {
    const int b = blockIdx.y;
    int cu0, n, len;
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (!ragged_rows(r, b, cu0, n, len) || i >= min(n, 32 * words)) return;
    unsigned* to = mask + (long long)(cu0 + i) * ld;
    int depth = 0, word = words - 1, at = i;
    unsigned bits = 0;
    for (;;) {
        for (; word > at >> 5; --word, bits = 0) to[word] = bits;
        bits |= 1u << (at & 31);
        const int up = parents[cu0 + at];
        if (up < 0 || up >= at) break;
        at = up;
        ++depth;
    }
    for (; word >= 0; --word, bits = 0) to[word] = bits;
    if (positions) positions[cu0 + i] = len - n + depth;
}

template <typename F>
void with_lie(Lie lie, F f) {
    if (lie == kRuns)
        f(std::integral_constant<Lie, kRuns>{});
    else if (lie == kNeighbours)
        f(std::integral_constant<Lie, kNeighbours>{});
    else
        f(std::integral_constant<Lie, kAnyhow>{});
}

template <typename T, int P, Lie LIE>
void turn_heads(const HeadsQ8& q, const HeadsQ8& k, const RopeQ8& rope, const Ragged& r, int dim,
                float eps, hipStream_t stream) {
    const int lanes = lanes_of(rope, dim, P, LIE), per = 64 / lanes;
    const int rows = r.cu ? r.max_rows : r.total, seqs = r.cu ? r.seqs : 1;
    const int parts = (q.heads + k.heads + per - 1) / per;
    // as many waves as the card holds, twice, or what there is for them; one
    // long sequence among many is not to go with a few
    const int most = std::max(std::max(kWavesInAll / seqs, 512) / parts, 1);
    const long long waves = (long long)std::min(rows, most) * parts;
    constexpr int kEach = kThreads / 64;
    const dim3 grid((unsigned)((waves + kEach - 1) / kEach), seqs);
    hipLaunchKernelGGL((qk_norm_rope_kernel<T, P, LIE>), grid, dim3(kThreads), 0, stream, q, k,
                       rope, r, dim, eps, lanes, parts);
}

template <typename T>
hipError_t qk(const HeadsQ8& q, const HeadsQ8& k, const RopeQ8& rope, const Ragged& r, int dim,
              float eps, hipStream_t stream) {
    // 16 bytes of a's and 16 of b's a lane, or 8 where heads are too short
    constexpr int P = 16 / sizeof(T);
    const Lie whole = lie_of(rope, dim, P), half = lie_of(rope, dim, 4);
    if (whole == kRuns)
        turn_heads<T, P, kRuns>(q, k, rope, r, dim, eps, stream);
    else if (whole == kNeighbours)
        turn_heads<T, P, kNeighbours>(q, k, rope, r, dim, eps, stream);
    else
        with_lie(half, [&](auto lie) {
            turn_heads<T, 4, decltype(lie)::value>(q, k, rope, r, dim, eps, stream);
        });
    return hipGetLastError();
}

template <typename T>
hipError_t kv_write_rope(const void* k, long long k_tok, long long k_head, const void* v,
                         long long v_tok, long long v_head, const float* weight, float eps,
                         const RopeQ8& rope, const CacheQ8& c, const Ragged& r,
                         hipStream_t stream) {
    const dim3 grid(kv_write_q8_pages(c, r), 2u * c.heads, r.seqs);
    const Lie how = lie_of(rope, c.dim, 4);
    const int lanes = lanes_of(rope, c.dim, 4, how);
    // groups of eight that one page can get
    const int most = std::min(c.page, r.max_rows) * lanes;
    with_lie(how, [&](auto lie) {
        constexpr Lie LIE = decltype(lie)::value;
#define AVAE_WRITE(HELD)                                                                          \
    hipLaunchKernelGGL((kv_write_rope_q8_kernel<T, HELD, LIE>), grid, dim3(kThreads), 0, stream,  \
                       (const T*)k, k_tok, k_head, (const T*)v, v_tok, v_head, weight, eps, rope, \
                       c, r, lanes)
        if (most <= kThreads)
            AVAE_WRITE(1);
        else if (most <= 4 * kThreads)
            AVAE_WRITE(4);
        else
            AVAE_WRITE(0);
#undef AVAE_WRITE
    });
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm_rope(int dtype, const HeadsQ8& q, const HeadsQ8& k, const RopeQ8& rope,
                               const Ragged& r, int dim, float eps, hipStream_t stream) {
    prof_pre(stream);
    const hipError_t e = dtype == AVAE_F32    ? qk<float>(q, k, rope, r, dim, eps, stream)
                         : dtype == AVAE_BF16 ? qk<__bf16>(q, k, rope, r, dim, eps, stream)
                                              : qk<_Float16>(q, k, rope, r, dim, eps, stream);
    const double n = (double)r.total * (q.heads + k.heads) * dim;
    prof_post(stream, "qk_norm_rope_kernel", 7.0 * n, 2.0 * n * (dtype == AVAE_F32 ? 4 : 2));
    return e;
}

hipError_t launch_kv_write_rope_q8(int dtype, const void* k, long long k_tok, long long k_head,
                                   const void* v, long long v_tok, long long v_head,
                                   const float* weight, float eps, const RopeQ8& rope,
                                   const CacheQ8& c, const Ragged& r, hipStream_t stream) {
    prof_pre(stream);
    const hipError_t e =
        dtype == AVAE_F32    ? kv_write_rope<float>(k, k_tok, k_head, v, v_tok, v_head, weight, eps,
                                                    rope, c, r, stream)
        : dtype == AVAE_BF16 ? kv_write_rope<__bf16>(k, k_tok, k_head, v, v_tok, v_head, weight,
                                                     eps, rope, c, r, stream)
                             : kv_write_rope<_Float16>(k, k_tok, k_head, v, v_tok, v_head, weight,
                                                       eps, rope, c, r, stream);
    const double n = 2.0 * r.total * c.heads * c.dim;
    prof_post(stream, "kv_write_rope_q8_kernel", 7.0 * n, n * ((dtype == AVAE_F32 ? 4 : 2) + 1));
    return e;
}

hipError_t launch_tree_mask(const int* parents, const Ragged& r, int words, int* mask,
                            long long ld, int* positions, hipStream_t stream) {
    prof_pre(stream);
    const dim3 grid((r.max_rows + kThreads - 1) / kThreads, r.seqs);
    hipLaunchKernelGGL(tree_mask_kernel, grid, dim3(kThreads), 0, stream, parents, r, words,
                       (unsigned*)mask, ld, positions);
    const hipError_t e = hipGetLastError();
    prof_post(stream, "tree_mask_kernel", 0.0, 4.0 * r.total * (words + 2));
    return e;
}

}  // namespace avae
