// Rows in 8 bits with one float32 scale each: root-mean-square norm with the
// residual's addition, the plain row quantiser, and the read-back.
//
//   h = x + residual,  v = h * weight,  s = max|v| / 127,  q = rint(v / s),
//   scale = s / sqrt(mean(h^2) + eps)
//
// The 8-bit values do not depend on the statistics (the row's factor
// 1 / sqrt(..) cancels in v / s), so the maximum and the sum of squares come
// from the same pass and q is the same whatever the order of the sum.  h is
// kept in float32 for the norm; only the returned sum is rounded to the
// residual stream's type.  HBM-bound: every element is read once and written
// once.
#include "avae.h"
#include "avae_internal.h"
#include "q8.h"

namespace avae {
namespace {

using namespace q8;

constexpr int kThreads = 256;

template <typename T, bool RES, bool NORM>
__global__ __launch_bounds__(kThreads) void rows_q8_kernel(
    const T* __restrict__ x, long long ldx, const T* __restrict__ res, long long ldr,
    const float* __restrict__ w, int C, float eps, T* __restrict__ sum, long long lds,
    int8_t* __restrict__ q, long long ldq, float* __restrict__ scale) {
    __shared__ unsigned s_max[kThreads / 64];
    __shared__ float s_sq[kThreads / 64];
    const long long row = blockIdx.x;
    const T* xr = x + row * ldx;
    const T* rr = RES ? res + row * ldr : nullptr;
    unsigned top = 0;
    float sq = 0.0f;
    for (int c = threadIdx.x; c < C; c += kThreads) {
        float h = (float)xr[c];
        if (RES) {
            h += (float)rr[c];
            sum[row * lds + c] = round_to<T>(h);
        }
        sq += h * h;
        top = max(top, mag_bits(NORM ? h * w[c] : h));
    }
    top = wave_max(top);
    sq = wave_sum(sq);
    if ((threadIdx.x & 63) == 0) {
        s_max[threadIdx.x >> 6] = top;
        s_sq[threadIdx.x >> 6] = sq;
    }
    __syncthreads();
    top = 0;
    sq = 0.0f;
    for (int i = 0; i < kThreads / 64; ++i) {
        top = max(top, s_max[i]);
        sq += s_sq[i];
    }
    const float s = scale_of(top);
    if (threadIdx.x == 0) scale[row] = NORM ? s * (1.0f / sqrtf(sq / (float)C + eps)) : s;
    for (int c = threadIdx.x; c < C; c += kThreads) {
        float h = (float)xr[c];
        if (RES) h += (float)rr[c];
        q[row * ldq + c] = (int8_t)quantise(NORM ? h * w[c] : h, s);
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dequant_q8_kernel(const int8_t* __restrict__ q,
                                                              long long ldq,
                                                              const float* __restrict__ scale,
                                                              int C, T* __restrict__ y,
                                                              long long ldy) {
    const long long row = blockIdx.x;
    const float s = scale[row];
    for (int c = threadIdx.x; c < C; c += kThreads)
        y[row * ldy + c] = round_to<T>((float)q[row * ldq + c] * s);
}

template <typename T>
hipError_t rows_q8(const void* x, long long ldx, const void* res, long long ldr, const float* w,
                   int M, int C, float eps, void* sum, long long lds, int8_t* q, long long ldq,
                   float* scale, hipStream_t stream) {
    const dim3 grid((unsigned)M), block(kThreads);
    const T* px = (const T*)x;
    const T* pr = (const T*)res;
    T* ps = (T*)sum;
    if (res && w)
        hipLaunchKernelGGL((rows_q8_kernel<T, true, true>), grid, block, 0, stream, px, ldx, pr,
                           ldr, w, C, eps, ps, lds, q, ldq, scale);
    else if (w)
        hipLaunchKernelGGL((rows_q8_kernel<T, false, true>), grid, block, 0, stream, px, ldx, pr,
                           ldr, w, C, eps, ps, lds, q, ldq, scale);
    else
        hipLaunchKernelGGL((rows_q8_kernel<T, false, false>), grid, block, 0, stream, px, ldx, pr,
                           ldr, w, C, eps, ps, lds, q, ldq, scale);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rows_q8(int dtype, const void* x, long long ldx, const void* res, long long ldr,
                          const float* w, int M, int C, float eps, void* sum, long long lds,
                          int8_t* q, long long ldq, float* scale, hipStream_t stream) {
    prof_pre(stream);
    hipError_t e;
    if (dtype == AVAE_F32)
        e = rows_q8<float>(x, ldx, res, ldr, w, M, C, eps, sum, lds, q, ldq, scale, stream);
    else if (dtype == AVAE_BF16)
        e = rows_q8<__bf16>(x, ldx, res, ldr, w, M, C, eps, sum, lds, q, ldq, scale, stream);
    else
        e = rows_q8<_Float16>(x, ldx, res, ldr, w, M, C, eps, sum, lds, q, ldq, scale, stream);
    const double n = (double)M * C, es = dtype == AVAE_F32 ? 4 : 2;
    prof_post(stream, "rows_q8_kernel", 6.0 * n, n * (es * (res ? 3 : 1) + 1));
    return e;
}

hipError_t launch_dequant_q8(int dtype, const int8_t* q, long long ldq, const float* scale, int M,
                             int C, void* y, long long ldy, hipStream_t stream) {
    prof_pre(stream);
    const dim3 grid((unsigned)M), block(kThreads);
    if (dtype == AVAE_F32)
        hipLaunchKernelGGL(dequant_q8_kernel<float>, grid, block, 0, stream, q, ldq, scale, C,
                           (float*)y, ldy);
    else if (dtype == AVAE_BF16)
        hipLaunchKernelGGL(dequant_q8_kernel<__bf16>, grid, block, 0, stream, q, ldq, scale, C,
                           (__bf16*)y, ldy);
    else
        hipLaunchKernelGGL(dequant_q8_kernel<_Float16>, grid, block, 0, stream, q, ldq, scale, C,
                           (_Float16*)y, ldy);
    const hipError_t e = hipGetLastError();
    const double n = (double)M * C;
    prof_post(stream, "dequant_q8_kernel", n, n * (1 + (dtype == AVAE_F32 ? 4 : 2)));
    return e;
}

}  // namespace avae
