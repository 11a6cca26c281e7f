// The 8-bit paged cache of keys and values: quantised as it is written, and
// read back.
//
// A page holds P tokens of every head, [head][token][dim], and one scale for
// each head.  A page that gets its first token takes max|x| * (1 / 127) of
// its new tokens as its scale.  One that holds tokens already keeps its scale
// if the new tokens fit it; else it grows to theirs and the held values move
// to the new range, q' = rint(q * old / new).  So writing the same tokens
// again changes nothing, and one workgroup owns each (page, head): no
// atomics, and the result does not depend on the order of the workgroups.
//
// HBM-bound: three ragged float32 prompts, 13600 tokens of 16 heads of 64,
// take 25 us to write and 25 to read back (5.6 TB/s each); 64 appended
// tokens 3.8 us, the latency of length, page, scale and values one after the
// other.
#include <algorithm>

#include "avae.h"
#include "avae_internal.h"
#include "q8.h"

namespace avae {
namespace {

using namespace q8;

constexpr int kThreads = 256;

// One page of one head, keys or values.  HELD groups of four values a thread
// stay in registers between the pass for the maximum and the one that rounds;
// HELD 0 (pages larger than that) reads them twice.
template <typename T, int HELD>
__global__ __launch_bounds__(kThreads) void kv_write_q8_kernel(
    const T* __restrict__ k, long long k_tok, long long k_head, const T* __restrict__ v,
    long long v_tok, long long v_head, CacheQ8 c, Ragged r) {
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
    const T* x = (is_v ? v : k) + (is_v ? v_head : k_head) * head +
                 (long long)(cu0 + p0 - start) * x_tok;
    const long long at = (long long)page * c.heads + head;
    int8_t* q = (is_v ? c.v : c.k) + at * c.page * c.dim;
    float* scales = is_v ? c.v_scale : c.k_scale;

    const int quads = c.dim / 4, quad_shift = __builtin_ctz(quads);  // groups of four in a token
    const int i0 = lo * quads + threadIdx.x, i1 = hi * quads;
    auto load = [&](int i, float(&f)[4]) {
        load_values<4>(x + (i >> quad_shift) * x_tok + (i & (quads - 1)) * 4, 4, f);
    };
    float held[HELD ? HELD : 1][4];
    unsigned top = 0;
    if constexpr (HELD > 0) {
#pragma unroll
        for (int j = 0; j < HELD; ++j)
            if (i0 + j * kThreads < i1) load(i0 + j * kThreads, held[j]);
#pragma unroll
        for (int j = 0; j < HELD; ++j)
            if (i0 + j * kThreads < i1)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = max(top, mag_bits(held[j][e]));
    } else {
        for (int i = i0; i < i1; i += kThreads) {
            load(i, held[0]);
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, mag_bits(held[0][e]));
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
    auto store = [&](int i, const float(&f)[4]) {
        reinterpret_cast<unsigned*>(q)[i] = to_bytes(quant.quotient(f[0]), quant.quotient(f[1]),
                                                     quant.quotient(f[2]), quant.quotient(f[3]));
    };
    if (lo > 0 && s > was)  // what the page held moves to the new range
        for (int i = threadIdx.x; i < lo * quads; i += kThreads) {
            float f[4];
            load_stored<4>(q + 4 * i, 4, f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] *= was;
            store(i, f);
        }
    if constexpr (HELD > 0) {
#pragma unroll
        for (int j = 0; j < HELD; ++j)
            if (i0 + j * kThreads < i1) store(i0 + j * kThreads, held[j]);
    } else {
        for (int i = i0; i < i1; i += kThreads) {
            load(i, held[0]);
            store(i, held[0]);
        }
    }
}

// A wave a token: 16 bytes of keys and of values a lane and step.
template <typename T>
__global__ __launch_bounds__(kThreads) void kv_read_q8_kernel(CacheQ8 c, Ragged r, int from,
                                                              T* __restrict__ k,
                                                              T* __restrict__ v) {
    const int b = blockIdx.y, lane = threadIdx.x & 63;
    int cu0, n, len;
    const int i = from + blockIdx.x * 4 + wave_id();  // the i-th of the sequence's last n tokens
    if (!ragged_rows(r, b, cu0, n, len) || i >= n) return;
    const int pos = len - n + i;
    const int col = pos >> c.shift;
    const int page = pos >= 0 ? page_of(c, b, col) : -1;
    const int row = c.heads * c.dim, dim_shift = __builtin_ctz(c.dim);
    const long long out = (long long)(cu0 + i) * row;
    constexpr int N = 16 / sizeof(T);
    for (int j = lane * N; j < row; j += 64 * N) {
        float kv[N] = {}, vv[N] = {};
        if (page >= 0) {
            const long long at = (long long)page * c.heads + (j >> dim_shift);
            const long long e = (at * c.page + (pos & (c.page - 1))) * c.dim + (j & (c.dim - 1));
            load_stored<N>(c.k + e, N, kv);
            load_stored<N>(c.v + e, N, vv);
            const float ks = c.k_scale[at], vs = c.v_scale[at];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                kv[i] *= ks;
                vv[i] *= vs;
            }
        }
        stream_values(k + out + j, N, kv);
        stream_values(v + out + j, N, vv);
    }
}

template <typename T>
hipError_t kv_write(const void* k, long long k_tok, long long k_head, const void* v,
                    long long v_tok, long long v_head, const CacheQ8& c, const Ragged& r,
                    hipStream_t stream) {
    const dim3 grid(kv_write_q8_pages(c, r), 2u * c.heads, r.seqs);
    // groups of four that one page can get
    const int most = std::min(c.page, r.max_rows) * (c.dim / 4);
#define AVAE_WRITE(HELD)                                                                          \
    hipLaunchKernelGGL((kv_write_q8_kernel<T, HELD>), grid, dim3(kThreads), 0, stream,            \
                       (const T*)k, k_tok, k_head, (const T*)v, v_tok, v_head, c, r)
    if (most <= 2 * kThreads)
        AVAE_WRITE(2);
    else if (most <= 8 * kThreads)
        AVAE_WRITE(8);
    else
        AVAE_WRITE(0);
#undef AVAE_WRITE
    return hipGetLastError();
}

template <typename T>
hipError_t kv_read(const CacheQ8& c, const Ragged& r, void* k, void* v, hipStream_t stream) {
    // (a launch has fewer than 2^32 threads a dimension)
    constexpr int kRun = 1 << 24;
    for (long long from = 0; from < r.max_rows; from += kRun) {
        const long long rows = std::min<long long>(r.max_rows - from, kRun);
        hipLaunchKernelGGL(kv_read_q8_kernel<T>, dim3((unsigned)((rows + 3) / 4), r.seqs),
                           dim3(kThreads), 0, stream, c, r, (int)from, (T*)k, (T*)v);
    }
    return hipGetLastError();
}

}  // namespace

int kv_write_q8_pages(const CacheQ8& c, const Ragged& r) {
    return std::min((r.max_rows + c.page - 2) / c.page + 1, c.table_cols);
}

hipError_t launch_kv_write_q8(int dtype, const void* k, long long k_tok, long long k_head,
                              const void* v, long long v_tok, long long v_head, const CacheQ8& c,
                              const Ragged& r, hipStream_t stream) {
    prof_pre(stream);
    const hipError_t e =
        dtype == AVAE_F32
            ? kv_write<float>(k, k_tok, k_head, v, v_tok, v_head, c, r, stream)
        : dtype == AVAE_BF16
            ? kv_write<__bf16>(k, k_tok, k_head, v, v_tok, v_head, c, r, stream)
            : kv_write<_Float16>(k, k_tok, k_head, v, v_tok, v_head, c, r, stream);
    const double n = 2.0 * r.total * c.heads * c.dim;
    prof_post(stream, "kv_write_q8_kernel", 4.0 * n, n * ((dtype == AVAE_F32 ? 4 : 2) + 1));
    return e;
}

hipError_t launch_kv_read_q8(int dtype, const CacheQ8& c, const Ragged& r, void* k, void* v,
                             hipStream_t stream) {
    prof_pre(stream);
    const hipError_t e = dtype == AVAE_F32    ? kv_read<float>(c, r, k, v, stream)
                         : dtype == AVAE_BF16 ? kv_read<__bf16>(c, r, k, v, stream)
                                              : kv_read<_Float16>(c, r, k, v, stream);
    const double n = 2.0 * r.total * c.heads * c.dim;
    prof_post(stream, "kv_read_q8_kernel", n, n * (1 + (dtype == AVAE_F32 ? 4 : 2)));
    return e;
}

}  // namespace avae
