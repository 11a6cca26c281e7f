// Rows in 8 bits with one float32 scale each: root-mean-square norm with the
// residual's addition, the plain row quantiser, and the read-back.
//
//   h = x + residual,  v = h * weight,  s = max|v| * (1 / 127),  q = rint(v / s),
//   scale = s / sqrt(mean(h^2) + eps)
//
// The 8-bit values do not depend on the statistics (the row's factor
// 1 / sqrt(..) cancels in v / s), so the maximum and the sum of squares come
// from the same pass and q is the same whatever the order of the sum.  h is
// kept in float32 for the norm; only the returned sum is rounded to the
// residual stream's type.
//
// HBM-bound: every element is read once and written once.  Measured:
// [8192, 8192] bfloat16 with residual 90 us (5.2 TB/s; a plain copy reaches
// 5.1 here), [6000, 1536] 13.4 us (4.8), one row of 1536 3.1 us, which is
// two memory latencies and the reduction; the read-back of [8192, 8192]
// 33 us (6.2 TB/s), of float32 rows of odd length 3.7 TB/s (their stores
// straddle cache lines).
#include <algorithm>

#include "avae.h"
#include "avae_internal.h"
#include "q8.h"

namespace avae {
namespace {

using namespace q8;

// Whether float32 holds a finite row's sum of squares: it may pass the
// largest number (|h| above 1.8e19), or its squares fall below the normal
// range where eps is too small to hide it.
__device__ inline bool squares_hold(float sq, float eps) {
    return sq < __uint_as_float(kInfBits) && (sq >= 0x1p-80f || eps >= 0x1p-100f);
}

// The scale of a normed row, for a row of zeros 0 whatever eps is.
__device__ inline float normed_scale(float s, float sq, int C, float eps) {
    return s == 0.0f ? 0.0f : s * (1.0f / sqrtf(sq / (float)C + eps));
}

// The same for the rare rows whose squares float32 does not hold: read again,
// summed in 64 bits by the row's THREADS threads; thread 0 has the result.
template <typename T, bool RES, int THREADS>
__device__ float normed_scale_wide(const T* x, const T* res, int C, int tid, float s, float eps,
                                   double* s_part) {
    double sq = 0.0;
    for (int c = tid; c < C; c += THREADS) {
        float h = (float)x[c];
        if (RES) h += (float)res[c];
        sq += (double)h * (double)h;
    }
    for (int o = 32; o > 0; o >>= 1) sq += __shfl_xor(sq, o);
    if (THREADS > 64) {
        if ((tid & 63) == 0) s_part[tid >> 6] = sq;
        __syncthreads();
        sq = 0.0;
        for (int i = 0; i < THREADS / 64; ++i) sq += s_part[i];
    }
    return (float)((double)s / sqrt(sq / C + (double)eps));
}

// One row a group of THREADS threads (64 of a workgroup of 256, or a whole
// workgroup of 256 or 1024), its values held in registers between the pass
// that finds the maximum and the one that rounds: 8 HELD a thread.
template <typename T, bool RES, bool NORM, int THREADS, int HELD>
__global__ __launch_bounds__(THREADS < 256 ? 256 : THREADS) void rows_q8_kernel(
    const T* __restrict__ x, long long ldx, const T* __restrict__ res, long long ldr,
    const float* __restrict__ w, int M, int C, float eps, T* __restrict__ sum, long long lds,
    int8_t* __restrict__ q, long long ldq, float* __restrict__ scale) {
    constexpr int WAVES = THREADS / 64;
    __shared__ unsigned s_max[WAVES];
    __shared__ float s_sq[WAVES];
    const int wave = wave_id();
    const long long row = THREADS == 64 ? blockIdx.x * 4LL + wave : blockIdx.x;
    if (row >= M) return;  // whole waves, and only where a wave has a row to itself
    const int tid = THREADS == 64 ? threadIdx.x & 63 : threadIdx.x;
    float v[HELD][8], r[RES ? HELD : 1][8];
    unsigned top = 0;
    float sq = 0.0f;
    // all of the row is on its way before any of it is used
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
        const int c = (tid + j * THREADS) * 8;
        load_values<8>(x + row * ldx + c, C - c, v[j]);
    }
    if (RES) {
#pragma unroll
        for (int j = 0; j < HELD; ++j) {
            const int c = (tid + j * THREADS) * 8;
            load_values<8>(res + row * ldr + c, C - c, r[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
        const int c = (tid + j * THREADS) * 8, left = C - c;
        if (RES) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] += r[j][i];
            // (next read a few operators later: streamed, [8192, 8192]
            // bfloat16 105 -> 90 us)
            constexpr int N = 16 / sizeof(T);
#pragma unroll
            for (int n = 0; n < 8; n += N) {
                float part[N];
#pragma unroll
                for (int i = 0; i < N; ++i) part[i] = v[j][n + i];
                stream_values(sum + row * lds + c + n, left - n, part);
            }
        }
        if (NORM) {
            float g[8];
            load_values<8>(w + c, left, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sq += v[j][i] * v[j][i];
                v[j][i] *= g[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, mag_bits(v[j][i]));
    }
    top = wave_max(top);
    if (NORM) sq = wave_sum(sq);
    if (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) {
            s_max[wave] = top;
            s_sq[wave] = sq;
        }
        __syncthreads();
        top = 0;
        sq = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            top = max(top, s_max[i]);
            sq += s_sq[i];
        }
    }
    const float s = scale_of(top);
    if (tid == 0) scale[row] = NORM ? normed_scale(s, sq, C, eps) : s;
    const Quantiser quant(s);
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
        const int c = (tid + j * THREADS) * 8, left = C - c;
        if (left <= 0) continue;
        unsigned out[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            out[h] = to_bytes(quant.quotient(v[j][4 * h]), quant.quotient(v[j][4 * h + 1]),
                              quant.quotient(v[j][4 * h + 2]), quant.quotient(v[j][4 * h + 3]));
        store_bytes<8>(q + row * ldq + c, left, out);
    }
    if (NORM && s > 0.0f && !squares_hold(sq, eps)) {  // all of the row's threads or none
        __shared__ double s_part[WAVES];
        const float wide = normed_scale_wide<T, RES, THREADS>(
            x + row * ldx, RES ? res + row * ldr : nullptr, C, tid, s, eps, s_part);
        if (tid == 0) scale[row] = wide;
    }
}

// Rows too long for the registers: read twice.
template <typename T, bool RES, bool NORM>
__global__ __launch_bounds__(1024) void long_rows_q8_kernel(
    const T* __restrict__ x, long long ldx, const T* __restrict__ res, long long ldr,
    const float* __restrict__ w, int C, float eps, T* __restrict__ sum, long long lds,
    int8_t* __restrict__ q, long long ldq, float* __restrict__ scale) {
    __shared__ unsigned s_max[16];
    __shared__ float s_sq[16];
    const long long row = blockIdx.x;
    const T* xr = x + row * ldx;
    const T* rr = RES ? res + row * ldr : nullptr;
    unsigned top = 0;
    float sq = 0.0f;
    for (int c = threadIdx.x; c < C; c += 1024) {
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
    for (int i = 0; i < 16; ++i) {
        top = max(top, s_max[i]);
        sq += s_sq[i];
    }
    const float s = scale_of(top);
    if (threadIdx.x == 0) scale[row] = NORM ? normed_scale(s, sq, C, eps) : s;
    const Quantiser quant(s);
    for (int c = threadIdx.x; c < C; c += 1024) {
        float h = (float)xr[c];
        if (RES) h += (float)rr[c];
        q[row * ldq + c] =
            (int8_t)to_bytes(quant.quotient(NORM ? h * w[c] : h), 0.0f, 0.0f, 0.0f);
    }
    if (NORM && s > 0.0f && !squares_hold(sq, eps)) {
        __shared__ double s_part[16];
        const float wide = normed_scale_wide<T, RES, 1024>(xr, rr, C, threadIdx.x, s, eps, s_part);
        if (threadIdx.x == 0) scale[row] = wide;
    }
}

// 16 bytes of output a thread; THREADS of them walk a row.
template <typename T, int THREADS>
__global__ __launch_bounds__(256) void dequant_q8_kernel(const int8_t* __restrict__ q,
                                                         long long ldq,
                                                         const float* __restrict__ scale, int M,
                                                         int C, T* __restrict__ y,
                                                         long long ldy) {
    const long long row = THREADS == 64 ? blockIdx.x * 4LL + wave_id() : blockIdx.x;
    if (row >= M) return;
    const int tid = THREADS == 64 ? threadIdx.x & 63 : threadIdx.x;
    const float s = scale[row];
    constexpr int N = 16 / sizeof(T);
    for (int c = tid * N; c < C; c += THREADS * N) {
        float v[N];
        load_stored<N>(q + row * ldq + c, C - c, v);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= s;
        stream_values(y + row * ldy + c, C - c, v);
    }
}

template <typename T, bool RES, bool NORM>
hipError_t rows_q8(const void* x, long long ldx, const void* res, long long ldr, const float* w,
                   int M, int C, float eps, void* sum, long long lds, int8_t* q, long long ldq,
                   float* scale, hipStream_t stream) {
    const T* px = (const T*)x;
    const T* pr = (const T*)res;
    T* ps = (T*)sum;
#define AVAE_ROWS(THREADS, HELD)                                                                 \
    hipLaunchKernelGGL((rows_q8_kernel<T, RES, NORM, THREADS, HELD>),                            \
                       dim3((unsigned)(THREADS == 64 ? (M + 3LL) / 4 : M)),                      \
                       dim3(THREADS < 256 ? 256 : THREADS), 0, stream, px, ldx, pr, ldr, w, M, C, \
                       eps, ps, lds, q, ldq, scale)
    // A wave for a short row, which needs no barrier; a workgroup for others,
    // where fewer bytes a lane leave more waves on the CUs ([6000, 1536]
    // bfloat16 with residual: 17.2 us a wave a row, 14.3 so).
    if (C <= 512)
        AVAE_ROWS(64, 1);
    else if (C <= 2048)
        AVAE_ROWS(256, 1);
    else if (C <= 4096)
        AVAE_ROWS(256, 2);
    else if (C <= 8192)
        AVAE_ROWS(256, 4);
    else if (C <= 16384)
        AVAE_ROWS(1024, 2);
    else if (C <= 32768)
        AVAE_ROWS(1024, 4);
    else
        hipLaunchKernelGGL((long_rows_q8_kernel<T, RES, NORM>), dim3((unsigned)M), dim3(1024), 0,
                           stream, px, ldx, pr, ldr, w, C, eps, ps, lds, q, ldq, scale);
#undef AVAE_ROWS
    return hipGetLastError();
}

template <typename T>
hipError_t rows_q8(const void* x, long long ldx, const void* res, long long ldr, const float* w,
                   int M, int C, float eps, void* sum, long long lds, int8_t* q, long long ldq,
                   float* scale, hipStream_t stream) {
    if (res)
        return rows_q8<T, true, true>(x, ldx, res, ldr, w, M, C, eps, sum, lds, q, ldq, scale,
                                      stream);
    if (w)
        return rows_q8<T, false, true>(x, ldx, res, ldr, w, M, C, eps, sum, lds, q, ldq, scale,
                                       stream);
    return rows_q8<T, false, false>(x, ldx, res, ldr, w, M, C, eps, sum, lds, q, ldq, scale,
                                    stream);
}

template <typename T>
hipError_t dequant_q8(const int8_t* q, long long ldq, const float* scale, int M, int C, void* y,
                      long long ldy, hipStream_t stream) {
    if (M >= 2048 || C <= 512)
        hipLaunchKernelGGL((dequant_q8_kernel<T, 64>), dim3((unsigned)((M + 3LL) / 4)), dim3(256),
                           0, stream, q, ldq, scale, M, C, (T*)y, ldy);
    else
        hipLaunchKernelGGL((dequant_q8_kernel<T, 256>), dim3((unsigned)M), dim3(256), 0, stream, q,
                           ldq, scale, M, C, (T*)y, ldy);
    return hipGetLastError();
}

}  // namespace

namespace {

// A launch has fewer than 2^32 threads: rows go out in runs of this many.
constexpr int kRun = 1 << 21;

template <typename T>
hipError_t rows_runs(const T* x, long long ldx, const T* res, long long ldr, const float* w, int M,
                     int C, float eps, T* sum, long long lds, int8_t* q, long long ldq,
                     float* scale, hipStream_t stream) {
    hipError_t e = hipSuccess;
    for (long long m = 0; m < M && e == hipSuccess; m += kRun)
        e = rows_q8<T>(x + m * ldx, ldx, res ? res + m * ldr : nullptr, ldr, w,
                       (int)std::min<long long>(M - m, kRun), C, eps,
                       sum ? sum + m * lds : nullptr, lds, q + m * ldq, ldq, scale + m, stream);
    return e;
}

template <typename T>
hipError_t dequant_runs(const int8_t* q, long long ldq, const float* scale, int M, int C, T* y,
                        long long ldy, hipStream_t stream) {
    hipError_t e = hipSuccess;
    for (long long m = 0; m < M && e == hipSuccess; m += kRun)
        e = dequant_q8<T>(q + m * ldq, ldq, scale + m, (int)std::min<long long>(M - m, kRun), C,
                          y + m * ldy, ldy, stream);
    return e;
}

}  // namespace

hipError_t launch_rows_q8(int dtype, const void* x, long long ldx, const void* res, long long ldr,
                          const float* w, int M, int C, float eps, void* sum, long long lds,
                          int8_t* q, long long ldq, float* scale, hipStream_t stream) {
    prof_pre(stream);
    hipError_t e;
    if (dtype == AVAE_F32)
        e = rows_runs((const float*)x, ldx, (const float*)res, ldr, w, M, C, eps, (float*)sum,
                      lds, q, ldq, scale, stream);
    else if (dtype == AVAE_BF16)
        e = rows_runs((const __bf16*)x, ldx, (const __bf16*)res, ldr, w, M, C, eps, (__bf16*)sum,
                      lds, q, ldq, scale, stream);
    else
        e = rows_runs((const _Float16*)x, ldx, (const _Float16*)res, ldr, w, M, C, eps, (_Float16*)sum,
                      lds, q, ldq, scale, stream);
    const double n = (double)M * C, es = dtype == AVAE_F32 ? 4 : 2;
    prof_post(stream, "rows_q8_kernel", 6.0 * n, n * (es * (res ? 3 : 1) + 1));
    return e;
}

hipError_t launch_dequant_q8(int dtype, const int8_t* q, long long ldq, const float* scale, int M,
                             int C, void* y, long long ldy, hipStream_t stream) {
    prof_pre(stream);
    const hipError_t e =
        dtype == AVAE_F32    ? dequant_runs(q, ldq, scale, M, C, (float*)y, ldy, stream)
        : dtype == AVAE_BF16 ? dequant_runs(q, ldq, scale, M, C, (__bf16*)y, ldy, stream)
                             : dequant_runs(q, ldq, scale, M, C, (_Float16*)y, ldy, stream);
    const double n = (double)M * C;
    prof_post(stream, "dequant_q8_kernel", n, n * (1 + (dtype == AVAE_F32 ? 4 : 2)));
    return e;
}

}  // namespace avae
