// The 8-bit paged cache of keys and values: quantised as it is written, and
// read back.
//
// A page holds P tokens of every head, [head][token][dim], and one scale for
// each head.  A page that gets its first token takes max|x| / 127 of its new
// tokens as its scale.  One that holds tokens already keeps its scale if the
// new tokens fit it; else it grows to theirs and the held values move to the
// new range, q' = rint(q * old / new).  So writing the same tokens again
// changes nothing, and one workgroup owns each (page, head): no atomics, and
// the result does not depend on the order of the workgroups.
#include "avae.h"
#include "avae_internal.h"
#include "q8.h"

namespace avae {
namespace {

using namespace q8;

constexpr int kThreads = 256;

template <typename T>
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
    const int lo = max(max(start, 0), p0) - p0;     // first new slot of this page
    const int hi = min(len, p0 + c.page) - p0;      // one past the last
    const T* x = is_v ? v : k;
    const long long x_tok = is_v ? v_tok : k_tok;
    x += (is_v ? v_head : k_head) * head + (long long)(cu0 + p0 - start) * x_tok;
    const long long at = (long long)page * c.heads + head;
    int8_t* q = (is_v ? c.v : c.k) + at * c.page * c.dim;
    float* scales = is_v ? c.v_scale : c.k_scale;

    unsigned top = 0;
    for (int i = lo * c.dim + threadIdx.x; i < hi * c.dim; i += kThreads)
        top = max(top, mag_bits((float)x[(i / c.dim) * x_tok + i % c.dim]));
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = top;
    const float held = lo > 0 ? scales[at] : 0.0f;
    __syncthreads();  // also: every thread has the old scale before it changes
    for (int i = 0; i < kThreads / 64; ++i) top = max(top, s_max[i]);
    const float fresh = scale_of(top);
    // a NaN on either side stays
    const float s = (held != held || fresh != fresh) ? __uint_as_float(0x7fc00000u)
                                                     : fmaxf(held, fresh);
    if (threadIdx.x == 0) scales[at] = s;
    if (lo > 0 && s > held)
        for (int i = threadIdx.x; i < lo * c.dim; i += kThreads)
            q[i] = (int8_t)quantise((float)q[i] * held, s);
    for (int i = lo * c.dim + threadIdx.x; i < hi * c.dim; i += kThreads)
        q[i] = (int8_t)quantise((float)x[(i / c.dim) * x_tok + i % c.dim], s);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void kv_read_q8_kernel(CacheQ8 c, Ragged r,
                                                              T* __restrict__ k,
                                                              T* __restrict__ v) {
    const int b = blockIdx.y;
    int cu0, n, len;
    const int i = blockIdx.x;  // the i-th of the sequence's last n tokens
    if (!ragged_rows(r, b, cu0, n, len) || i >= n) return;
    const int pos = len - n + i;
    const int col = pos >> c.shift;
    const int page = pos >= 0 ? page_of(c, b, col) : -1;
    const bool there = page >= 0;
    const int row = c.heads * c.dim;
    const long long out = (long long)(cu0 + i) * row;
    for (int j = threadIdx.x; j < row; j += kThreads) {
        const int head = j / c.dim;
        float kv = 0.0f, vv = 0.0f;
        if (there) {
            const long long at = (long long)page * c.heads + head;
            const long long e = (at * c.page + (pos - col * c.page)) * c.dim + j % c.dim;
            kv = (float)c.k[e] * c.k_scale[at];
            vv = (float)c.v[e] * c.v_scale[at];
        }
        k[out + j] = round_to<T>(kv);
        v[out + j] = round_to<T>(vv);
    }
}

}  // namespace

hipError_t launch_kv_write_q8(int dtype, const void* k, long long k_tok, long long k_head,
                              const void* v, long long v_tok, long long v_head, const CacheQ8& c,
                              const Ragged& r, hipStream_t stream) {
    // pages that max_rows tokens can touch, at any place in the first of them
    const dim3 grid((unsigned)((r.max_rows + c.page - 2) / c.page + 1), 2u * c.heads, r.seqs);
    prof_pre(stream);
    if (dtype == AVAE_F32)
        hipLaunchKernelGGL(kv_write_q8_kernel<float>, grid, dim3(kThreads), 0, stream,
                           (const float*)k, k_tok, k_head, (const float*)v, v_tok, v_head, c, r);
    else if (dtype == AVAE_BF16)
        hipLaunchKernelGGL(kv_write_q8_kernel<__bf16>, grid, dim3(kThreads), 0, stream,
                           (const __bf16*)k, k_tok, k_head, (const __bf16*)v, v_tok, v_head, c, r);
    else
        hipLaunchKernelGGL(kv_write_q8_kernel<_Float16>, grid, dim3(kThreads), 0, stream,
                           (const _Float16*)k, k_tok, k_head, (const _Float16*)v, v_tok, v_head, c,
                           r);
    const hipError_t e = hipGetLastError();
    const double n = 2.0 * r.total * c.heads * c.dim;
    prof_post(stream, "kv_write_q8_kernel", 4.0 * n, n * ((dtype == AVAE_F32 ? 4 : 2) + 1));
    return e;
}

hipError_t launch_kv_read_q8(int dtype, const CacheQ8& c, const Ragged& r, void* k, void* v,
                             hipStream_t stream) {
    const dim3 grid((unsigned)r.max_rows, (unsigned)r.seqs);
    prof_pre(stream);
    if (dtype == AVAE_F32)
        hipLaunchKernelGGL(kv_read_q8_kernel<float>, grid, dim3(kThreads), 0, stream, c, r,
                           (float*)k, (float*)v);
    else if (dtype == AVAE_BF16)
        hipLaunchKernelGGL(kv_read_q8_kernel<__bf16>, grid, dim3(kThreads), 0, stream, c, r,
                           (__bf16*)k, (__bf16*)v);
    else
        hipLaunchKernelGGL(kv_read_q8_kernel<_Float16>, grid, dim3(kThreads), 0, stream, c, r,
                           (_Float16*)k, (_Float16*)v);
    const hipError_t e = hipGetLastError();
    const double n = 2.0 * r.total * c.heads * c.dim;
    prof_post(stream, "kv_read_q8_kernel", n, n * (1 + (dtype == AVAE_F32 ? 4 : 2)));
    return e;
}

}  // namespace avae
