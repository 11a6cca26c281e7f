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

// Scale of values whose largest magnitude is `amax_bits`: amax / 127 rounded
// to float32; NaN if one of them is not finite.
__device__ inline float scale_of(unsigned amax_bits) {
    return amax_bits >= kInfBits ? __uint_as_float(0x7fc00000u)
                                 : __uint_as_float(amax_bits) / 127.0f;
}

// The stored value nearest x / scale (ties to even, the division correctly
// rounded).  0 where the scale is 0 or NaN.
__device__ inline int quantise(float x, float scale) {
    if (!(scale > 0.0f)) return 0;
    return (int)fminf(fmaxf(rintf(x / scale), -127.0f), 127.0f);
}

// Rows cu[b] .. cu[b+1] of sequence b; false if it has none, or if the
// offsets do not lie in the packed rows.
__device__ inline bool ragged_rows(const Ragged& r, int b, int& at, int& n, int& len) {
    at = r.cu[b];
    const int end = r.cu[b + 1];
    len = r.lens[b];
    n = end - at;
    return at >= 0 && end > at && end <= r.total && len > 0;
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
