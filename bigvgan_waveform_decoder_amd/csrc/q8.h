// Device helpers shared by the 8-bit serving operators (q8_*.hip): element
// types, the quantiser's rounding, reductions over a wave.
//
// Element types: float, __bf16 and _Float16 hold what the caller passes as
// AVAE_F32, AVAE_BF16 and AVAE_F16.  All arithmetic is in float32.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "avae_internal.h"

namespace avae {
namespace q8 {

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
    T v[N];
};

// A float32 result in the output's type.  The value is fixed in float32
// first: a product would else be fused with its conversion to float16 and
// rounded differently there than for the other types.
template <typename T>
__device__ inline T round_to(float x) {
    if constexpr (sizeof(T) == 2) asm("" : "+v"(x));
    return (T)x;
}

// Largest magnitude by its bits: a NaN or an infinity wins over every finite
// value, so a non-finite row is seen in the maximum itself.
__device__ inline unsigned mag_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr unsigned kInfBits = 0x7f800000u;

// Scale of values whose largest magnitude is `amax_bits`: amax times float32's
// 1 / 127, within 0.57 of a last place of amax / 127, and to the bit what
// torch's `amax / 127` gives on the device (it divides by a number so); NaN if
// one of the values is not finite.
__device__ inline float scale_of(unsigned amax_bits) {
    return amax_bits >= kInfBits ? __uint_as_float(0x7fc00000u)
                                 : __uint_as_float(amax_bits) * (1.0f / 127.0f);
}

// x / scale, correctly rounded, for x in the row that the scale was taken
// from; 0 where the scale is 0 or NaN.  The quotient is x times the
// reciprocal, corrected by its own remainder (exact in one fmaf); scales so
// small or large that reciprocal or remainder would leave float32's normal
// range take the division itself.  A scale of a few of the smallest
// subnormals can be a third below its row's maximum / 127: quotients past
// 127 are held there.
struct Quantiser {
    float scale, inv;
    bool plain;

    __device__ explicit Quantiser(float s) : scale(s), inv(1.0f / s), plain(s >= 1e-30f && s <= 1e30f) {}

    __device__ float quotient(float x) const {
        if (plain) {
            const float r = x * inv;
            return fmaf(fmaf(-r, scale, x), inv, r);
        }
        return scale > 0.0f ? fminf(fmaxf(x / scale, -127.0f), 127.0f) : 0.0f;
    }
};

// Four quotients in [-127.5, 127.5) rounded to bytes.  Adding 1.5 * 2^23
// leaves the nearest whole number (ties to even) in the low bits.
__device__ inline unsigned to_bytes(float a, float b, float c, float d) {
    constexpr float kRound = 12582912.0f;
    const unsigned x = __float_as_uint(a + kRound), y = __float_as_uint(b + kRound);
    const unsigned z = __float_as_uint(c + kRound), w = __float_as_uint(d + kRound);
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(w, z, 0x0c0c0400u),
                                 __builtin_amdgcn_perm(y, x, 0x0c0c0400u), 0x05040100u);
}

// N consecutive values from any address; what lies past `left` of them is 0.
template <int N, typename T>
__device__ inline void load_values(const T* p, int left, float (&x)[N]) {
    if (left >= N) {
        T v[N];
        __builtin_memcpy(v, p, sizeof(v));
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = (float)v[i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = i < left ? (float)p[i] : 0.0f;
    }
}

template <int N, typename T>
__device__ inline void store_values(T* p, int left, const float (&x)[N]) {
    T v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = round_to<T>(x[i]);
    if (left >= N) {
        __builtin_memcpy(p, v, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) p[i] = v[i];
    }
}

// 16 bytes of outputs that the caller reads back from memory: not kept in
// the caches where the address allows the one store.
template <typename T>
__device__ inline void stream_values(T* p, int left, const float (&x)[16 / sizeof(T)]) {
    constexpr int N = 16 / sizeof(T);
    typedef unsigned u4 __attribute__((ext_vector_type(4), aligned(4)));
    if (left >= N && ((uintptr_t)p & 3) == 0) {
        T v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = round_to<T>(x[i]);
        u4 w;
        __builtin_memcpy(&w, v, 16);
        __builtin_nontemporal_store(w, reinterpret_cast<u4*>(p));
    } else {
        store_values<N>(p, left, x);
    }
}

template <int N>
__device__ inline void store_bytes(int8_t* p, int left, const unsigned (&w)[N / 4]) {
    if (left >= N) {
        __builtin_memcpy(p, w, N);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) p[i] = (int8_t)(w[i / 4] >> (8 * (i % 4)));
    }
}

// N stored values from any address as floats.
template <int N>
__device__ inline void load_stored(const int8_t* p, int left, float (&x)[N]) {
    if (left >= N) {
        int8_t v[N];
        __builtin_memcpy(v, p, N);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = (float)v[i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = i < left ? (float)p[i] : 0.0f;
    }
}

// Rows cu[b] .. cu[b+1] of sequence b and its length (not below 0: then its
// rows are tokens of no page); false if it has none, or if the offsets do not
// lie in the packed rows.
__device__ inline bool ragged_rows(const Ragged& r, int b, int& at, int& n, int& len) {
    at = r.cu[b];
    const int end = r.cu[b + 1];
    len = max(r.lens[b], 0);
    n = end - at;
    return at >= 0 && end > at && end <= r.total;
}

// The page of a table's column, or -1 if there is none: a column outside the
// table, or an entry that is no page.  In two steps, so that an entry can be
// on its way while other work goes on; the entry is read from inside the
// table whatever the column (col >= 0).
__device__ inline int page_entry(const CacheQ8& c, int b, int col) {
    return c.table[(long long)b * c.table_ld + min(col, c.table_cols - 1)];
}

__device__ inline int page_checked(const CacheQ8& c, int col, int entry) {
    return col < c.table_cols && entry >= 0 && entry < c.n_pages ? entry : -1;
}

__device__ inline int page_of(const CacheQ8& c, int b, int col) {
    return page_checked(c, col, page_entry(c, b, col));
}

// Workgroups go to the 8 XCDs in turn; this gives each XCD a contiguous range
// of the `count` tiles, so that neighbours share its L2.
__device__ inline int xcd_remap(int id, int count) {
    const int q = count >> 3, r = count & 7, xcd = id & 7, at = id >> 3;
    return xcd < r ? xcd * (q + 1) + at : r * (q + 1) + (xcd - r) * q + at;
}

// This wave's index in its workgroup, known to be the same in all its lanes.
__device__ inline int wave_id() {
    return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

__device__ inline unsigned wave_max(unsigned v) {
    for (int o = 32; o > 0; o >>= 1) v = max(v, (unsigned)__shfl_xor((int)v, o));
    return v;
}

__device__ inline float wave_sum(float v) {
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

}  // namespace q8
}  // namespace avae
