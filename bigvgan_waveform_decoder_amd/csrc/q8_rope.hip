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
// bits; cosine and sine of the rest are Taylor sums, 1.5 last places off at
// most.
#include <algorithm>

#include "avae.h"
#include "avae_internal.h"
#include "q8.h"

namespace avae {
namespace {

using namespace q8;

constexpr int kThreads = 256;

// A lane holds four pairs of a head: pairs 4 j .. 4 j + 3, the dims past the
// rotated ones counted as neighbours (2 p, 2 p + 1).
struct Pairs {
    float a[4], b[4];
};

// Dims of pair p; `apart` is rot / 2 where pairs are that far apart, 0 where
// they are neighbours.
__device__ inline int dim_a(int p, int apart) { return p < apart ? p : 2 * p; }
__device__ inline int dim_b(int p, int apart) { return p < apart ? p + apart : 2 * p + 1; }

// Pairs 4 j .. of a head of `dim` dims; 0 past them.
template <typename T>
__device__ inline void load_pairs(const T* x, int j, int apart, int dim, Pairs& r) {
    if (4 * j + 3 < apart) {
        load_values<4>(x + 4 * j, 4, r.a);
        load_values<4>(x + 4 * j + apart, 4, r.b);
    } else if (4 * j >= apart) {
        float v[8];
        load_values<8>(x + 8 * j, dim - 8 * j, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r.a[e] = v[2 * e];
            r.b[e] = v[2 * e + 1];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int da = dim_a(4 * j + e, apart), db = dim_b(4 * j + e, apart);
            r.a[e] = da < dim ? (float)x[da] : 0.0f;
            r.b[e] = db < dim ? (float)x[db] : 0.0f;
        }
    }
}

template <typename T>
__device__ inline void store_pairs(T* x, int j, int apart, int dim, const Pairs& r) {
    if (4 * j + 3 < apart) {
        store_values<4>(x + 4 * j, 4, r.a);
        store_values<4>(x + 4 * j + apart, 4, r.b);
    } else if (4 * j >= apart) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = r.a[e];
            v[2 * e + 1] = r.b[e];
        }
        store_values<8>(x + 8 * j, dim - 8 * j, v);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int da = dim_a(4 * j + e, apart), db = dim_b(4 * j + e, apart);
            if (da < dim) x[da] = round_to<T>(r.a[e]);
            if (db < dim) x[db] = round_to<T>(r.b[e]);
        }
    }
}

// Four pairs in 8 bits (bytes: those of the a's, those of the b's).
__device__ inline void store_pair_bytes(int8_t* x, int j, int apart, unsigned a, unsigned b) {
    if (4 * j + 3 < apart) {
        __builtin_memcpy(x + 4 * j, &a, 4);
        __builtin_memcpy(x + 4 * j + apart, &b, 4);
    } else if (4 * j >= apart) {
        const unsigned w[2] = {__builtin_amdgcn_perm(b, a, 0x05010400u),
                               __builtin_amdgcn_perm(b, a, 0x07030602u)};
        __builtin_memcpy(x + 8 * j, w, 8);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[dim_a(4 * j + e, apart)] = (int8_t)(a >> (8 * e));
            x[dim_b(4 * j + e, apart)] = (int8_t)(b >> (8 * e));
        }
    }
}

// amp cos and amp sin of the lane's pairs at a position.
struct Turn {
    double quarter[4];  // quarter turns a position
    int turned;         // how many of the four pairs are

    __device__ void load(const RopeQ8& r, int j) {
        turned = min(max(r.half - 4 * j, 0), 4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            quarter[e] = e < turned ? (double)r.freq[4 * j + e] * 0.63661977236758134308 : 0.0;
    }

    __device__ void at(int pos, float amp, float (&c)[4], float (&s)[4]) const {
        // adding 1.5 * 2^52 leaves the nearest whole number in the low bits
        constexpr double kRound = 6755399441055744.0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const double d = (double)pos * quarter[e];
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
            const float cf = ((quadrant + 1) & 2) ? -co : co, sf = (quadrant & 2) ? -si : si;
            c[e] = cf * amp;
            s[e] = sf * amp;
        }
    }
};

// (a pair that is not turned is left alone: 0 times an infinity is NaN)
__device__ inline void turn(Pairs& r, int turned, const float (&c)[4], const float (&s)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = r.a[e], b = r.b[e];
        r.a[e] = e < turned ? fmaf(a, c[e], -b * s[e]) : a;
        r.b[e] = e < turned ? fmaf(b, c[e], a * s[e]) : b;
    }
}

// x / sqrt(mean x^2 + eps) * weight over a head that `lanes` neighbouring
// lanes hold.  Squares that leave float32's range are summed in 64 bits; a
// head of zeros stays zeros.
__device__ inline void norm(Pairs& r, const Pairs& w, int lanes, int dim, float eps) {
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum = fmaf(r.a[e], r.a[e], fmaf(r.b[e], r.b[e], sum));
    for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor(sum, o);
    if (sum >= 1e-24f && sum < 1e37f) {  // (a smaller one has squares below 2^-126 in it)
        const float by = 1.0f / sqrtf(sum / (float)dim + eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r.a[e] = r.a[e] * by * w.a[e];
            r.b[e] = r.b[e] * by * w.b[e];
        }
        return;
    }
    double all = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        all += (double)r.a[e] * (double)r.a[e] + (double)r.b[e] * (double)r.b[e];
    for (int o = 1; o < lanes; o <<= 1) all += __shfl_xor(all, o);
    const double by = all == 0.0 ? 0.0 : 1.0 / sqrt(all / dim + (double)eps);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        r.a[e] = (float)((double)r.a[e] * by * (double)w.a[e]);
        r.b[e] = (float)((double)r.b[e] * by * (double)w.b[e]);
    }
}

// A wave a token and IT rounds of 64 / lanes heads: each head lies in `lanes`
// neighbouring lanes, and a lane's cosines serve all its heads.
template <typename T, int IT>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(HeadsQ8 q, HeadsQ8 k, RopeQ8 rope,
                                                                Ragged r, int dim, float eps,
                                                                int lanes, int parts) {
    const int b = blockIdx.y, lane = threadIdx.x & 63;
    int cu0 = 0, n = r.total, start = 0;
    if (r.cu) {
        int len;
        if (!ragged_rows(r, b, cu0, n, len)) return;
        start = len - n;
    }
    const int j = lane & (lanes - 1), per = 64 / lanes, heads = q.heads + k.heads;
    const bool there = 8 * j < dim;
    Turn turns;
    turns.load(rope, j);
    const long long items = (long long)n * parts;
    for (long long item = blockIdx.x * 4LL + wave_id(); item < items; item += gridDim.x * 4LL) {
        const int i = (int)(item / parts), part = (int)(item - (long long)i * parts);
        const long long tok = cu0 + i;
        const int h0 = part * IT * per + lane / lanes;
        Pairs x[IT];
#pragma unroll
        for (int t = 0; t < IT; ++t) {
            const int h = h0 + t * per;
            const bool is_q = h < q.heads;
            const T* from = (const T*)(is_q ? q.x : k.x) + tok * (is_q ? q.tok : k.tok) +
                            (is_q ? h * q.head : (h - q.heads) * k.head);
            x[t] = Pairs{};
            if (there && h < heads) load_pairs(from, j, rope.apart, dim, x[t]);
        }
        float c[4], s[4];
        turns.at(rope.positions ? rope.positions[tok] : start + i, rope.amp, c, s);
#pragma unroll
        for (int t = 0; t < IT; ++t) {
            const int h = h0 + t * per;
            if (h >= heads) break;
            const bool is_q = h < q.heads;
            const float* weight = is_q ? q.weight : k.weight;
            if (weight) {
                Pairs w{};
                if (there) load_pairs(weight, j, rope.apart, dim, w);
                norm(x[t], w, lanes, dim, eps);
            }
            turn(x[t], turns.turned, c, s);
            T* to = (T*)(is_q ? q.y : k.y) + tok * (is_q ? q.y_tok : k.y_tok) +
                    (is_q ? h * q.y_head : (h - q.heads) * k.y_head);
            if (there) store_pairs(to, j, rope.apart, dim, x[t]);
        }
    }
}

// One page of one head, keys or values, as the cache's write has it: HELD
// groups of eight values a thread stay in registers between the pass for the
// maximum and the one that rounds; HELD 0 (larger pages) makes them twice.
template <typename T, int HELD>
__global__ __launch_bounds__(kThreads) void kv_write_rope_q8_kernel(
    const T* __restrict__ k, long long k_tok, long long k_head, const T* __restrict__ v,
    long long v_tok, long long v_head, const float* __restrict__ weight, float eps, RopeQ8 rope,
    CacheQ8 c, Ragged r) {
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

    const int lanes = c.dim / 8, shift = __builtin_ctz(lanes);
    const int j = threadIdx.x & (lanes - 1);
    const int i0 = lo * lanes + threadIdx.x, i1 = hi * lanes;
    const int apart = is_v ? 0 : rope.apart;
    Turn turns{};
    Pairs w{};
    if (!is_v) {
        turns.load(rope, j);
        if (weight) load_pairs(weight, j, apart, c.dim, w);
    }
    auto load = [&](int i, Pairs& f) {
        load_pairs(x + (i >> shift) * x_tok, j, apart, c.dim, f);
    };
    auto make = [&](int i, Pairs& f) {
        if (is_v) return;
        if (weight) norm(f, w, lanes, c.dim, eps);
        if (rope.half) {
            const int slot = i >> shift;
            float cs[4], sn[4];
            turns.at(rope.positions ? rope.positions[tok0 + slot] : p0 + slot, rope.amp, cs, sn);
            turn(f, turns.turned, cs, sn);
        }
    };
    auto most = [&](const Pairs& f, unsigned top) {
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(mag_bits(f.a[e]), mag_bits(f.b[e])));
        return top;
    };
    Pairs held[HELD ? HELD : 1];
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
    auto store = [&](int i, const Pairs& f) {
        store_pair_bytes(q + (long long)(i >> shift) * c.dim, j, apart, bytes(f.a), bytes(f.b));
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

// A thread a draft: it follows its line of parents back and sets their bits.
// A parent comes before its child, so the line goes down and each word is
// written once.
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

template <typename T>
hipError_t qk(const HeadsQ8& q, const HeadsQ8& k, const RopeQ8& rope, const Ragged& r, int dim,
              float eps, hipStream_t stream) {
    int lanes = 1;
    while (8 * lanes < dim) lanes *= 2;
    const int per = 64 / lanes, heads = q.heads + k.heads;
    const int rows = r.cu ? r.max_rows : r.total, seqs = r.cu ? r.seqs : 1;
    constexpr int IT = 4;
    const int parts1 = (heads + per - 1) / per;
    const bool few = (long long)rows * seqs * parts1 <= 8192;
    const int parts = few ? parts1 : (parts1 + IT - 1) / IT;
    // (as many workgroups as keep the card busy: they take item after item)
    const long long most = std::max((1 << 20) / seqs, 1);
    const dim3 grid((unsigned)std::min(((long long)rows * parts + 3) / 4, most), seqs);
    if (few)
        hipLaunchKernelGGL((qk_norm_rope_kernel<T, 1>), grid, dim3(kThreads), 0, stream, q, k, rope,
                           r, dim, eps, lanes, parts);
    else
        hipLaunchKernelGGL((qk_norm_rope_kernel<T, IT>), grid, dim3(kThreads), 0, stream, q, k,
                           rope, r, dim, eps, lanes, parts);
    return hipGetLastError();
}

template <typename T>
hipError_t kv_write_rope(const void* k, long long k_tok, long long k_head, const void* v,
                         long long v_tok, long long v_head, const float* weight, float eps,
                         const RopeQ8& rope, const CacheQ8& c, const Ragged& r,
                         hipStream_t stream) {
    const dim3 grid(kv_write_q8_pages(c, r), 2u * c.heads, r.seqs);
    // groups of eight that one page can get
    const int most = std::min(c.page, r.max_rows) * (c.dim / 8);
#define AVAE_WRITE(HELD)                                                                          \
    hipLaunchKernelGGL((kv_write_rope_q8_kernel<T, HELD>), grid, dim3(kThreads), 0, stream,       \
                       (const T*)k, k_tok, k_head, (const T*)v, v_tok, v_head, weight, eps, rope, \
                       c, r)
    if (most <= kThreads)
        AVAE_WRITE(1);
    else if (most <= 4 * kThreads)
        AVAE_WRITE(4);
    else
        AVAE_WRITE(0);
#undef AVAE_WRITE
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
