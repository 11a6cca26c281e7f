// Product of 8-bit activations and weights with a scale for each row of
// either:
//   y[m, n] = act( (sum_k a[m, k] w[n, k]) * sa[m] * sw[n] + bias[n] )
// The sum is exact in int32 (|a|, |w| <= 128, K <= 131071), so its order
// never shows in the result.
#include "avae.h"
#include "avae_internal.h"
#include "q8.h"

namespace avae {
namespace {

using namespace q8;

typedef int v4i __attribute__((ext_vector_type(4)));

template <typename T, bool SILU>
__device__ inline T epilogue(int acc, float sa, float sw, float bias) {
    // fmaf keeps the scaled sum and the bias in one rounding
    float v = fmaf((float)acc * sa, sw, bias);
    if (SILU) v = v / (1.0f + __expf(-v));
    return round_to<T>(v);
}

// Any alignment, any K: a 64 x 64 tile of y per workgroup, 64 bytes of K a
// step, staged byte by byte with zeros outside the operands.
template <typename T, bool SILU>
__global__ __launch_bounds__(256) void linear_q8_any_kernel(
    const int8_t* __restrict__ a, long long lda, const float* __restrict__ sa,
    const int8_t* __restrict__ w, long long ldw, const float* __restrict__ sw,
    const float* __restrict__ bias, int M, int N, int K, T* __restrict__ y, long long ldy) {
    constexpr int LD = 80;  // 16-byte aligned rows, 16 bytes of padding
    __shared__ __align__(16) int8_t s_a[64 * LD];
    __shared__ __align__(16) int8_t s_w[64 * LD];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n0 = blockIdx.x * 64, m0 = blockIdx.y * 64;
    v4i acc[4] = {};
    for (int k0 = 0; k0 < K; k0 += 64) {
        for (int i = tid; i < 64 * 64; i += 256) {
            const int r = i >> 6, k = k0 + (i & 63);
            s_a[r * LD + (i & 63)] = (m0 + r < M && k < K) ? a[(m0 + r) * lda + k] : 0;
            s_w[r * LD + (i & 63)] = (n0 + r < N && k < K) ? w[(n0 + r) * ldw + k] : 0;
        }
        __syncthreads();
        const int at = (lane & 15) * LD + (lane >> 4) * 16;
        const v4i av = *reinterpret_cast<const v4i*>(s_a + wave * 16 * LD + at);
        for (int t = 0; t < 4; ++t) {
            const v4i wv = *reinterpret_cast<const v4i*>(s_w + t * 16 * LD + at);
            acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av, wv, acc[t], 0, 0, 0);
        }
        __syncthreads();
    }
    for (int t = 0; t < 4; ++t) {
        const int n = n0 + t * 16 + (lane & 15);
        if (n >= N) continue;
        for (int r = 0; r < 4; ++r) {
            const int m = m0 + wave * 16 + (lane >> 4) * 4 + r;
            if (m < M)
                y[m * ldy + n] =
                    epilogue<T, SILU>(acc[t][r], sa[m], sw[n], bias ? bias[n] : 0.0f);
        }
    }
}

template <typename T, bool SILU>
hipError_t linear_q8(const int8_t* a, long long lda, const float* sa, const int8_t* w,
                     long long ldw, const float* sw, const float* bias, int M, int N, int K,
                     void* y, long long ldy, hipStream_t stream) {
    hipLaunchKernelGGL((linear_q8_any_kernel<T, SILU>), dim3((N + 63) / 64, (M + 63) / 64),
                       dim3(256), 0, stream, a, lda, sa, w, ldw, sw, bias, M, N, K, (T*)y, ldy);
    return hipGetLastError();
}

}  // namespace

size_t linear_q8_workspace_bytes(int M, int N, int K) { return 0; }

hipError_t launch_linear_q8(const int8_t* a, long long lda, const float* sa, const int8_t* w,
                            long long ldw, const float* sw, const float* bias, int M, int N, int K,
                            int act, int dtype, void* y, long long ldy, void* ws,
                            hipStream_t stream) {
    prof_pre(stream);
    hipError_t e;
#define AVAE_LINEAR(T)                                                                         \
    (act ? linear_q8<T, true>(a, lda, sa, w, ldw, sw, bias, M, N, K, y, ldy, stream)           \
         : linear_q8<T, false>(a, lda, sa, w, ldw, sw, bias, M, N, K, y, ldy, stream))
    if (dtype == AVAE_F32)
        e = AVAE_LINEAR(float);
    else if (dtype == AVAE_BF16)
        e = AVAE_LINEAR(__bf16);
    else
        e = AVAE_LINEAR(_Float16);
#undef AVAE_LINEAR
    prof_post(stream, "linear_q8_kernel", 2.0 * M * N * K,
              (double)M * K + (double)N * K + (double)M * N * (dtype == AVAE_F32 ? 4 : 2));
    return e;
}

}  // namespace avae
