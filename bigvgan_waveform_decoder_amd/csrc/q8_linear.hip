// Product of 8-bit activations and weights with a scale for each row of
// either:
//   y[m, n] = act( (sum_k a[m, k] w[n, k]) * sa[m] * sw[n] + bias[n] )
// The sum is exact in int32 (|a|, |w| <= 128, K <= 131071), so neither its
// order nor its split shows in the result.
//
// Both operands have K contiguous, which is what the matrix instruction
// takes (v_mfma_i32_16x16x64_i8: lane l = 16 g + i holds 16 consecutive k of
// row i at 16 g).  The weights are its A operand and the activations B, so a
// lane ends with consecutive n of one row m; with the weight rows dealt to
// the tiles in fours (row 4 T (i / 4) + 4 t + i % 4 of T tiles to tile t) it
// holds 4 T of them and stores them at once.
//
// Measured (bfloat16 output; the library's int8 product reaches 2330 TOPS at
// [8192]^3): [8192, 8192, 8192] 484 us, 2270 TOPS, bound by LDS reads and
// matrix instructions alike (1536 of LDS and 512 of staging cycles beside
// 2048 of products a step); [6000, 6144, 1536] 80-83 us, whose twelve steps a
// tile leave the outputs' writes and the SiLU of 96 values a thread a third
// of the time; [37, 1536, 6144] 11.0 us and [1, 4608, 1536] 4.0 us (an empty
// kernel takes 1.8): latency.  A wave goes through its steps in batches and a
// remainder of single ones, which wait for their loads one after the other
// (all four of a wave's steps at K = 1536 with up to 32 rows), and as built a
// batch has up to seven loads in flight, not all of its 24.
#include <algorithm>

#include "avae.h"
#include "avae_internal.h"
#include "q8.h"

namespace avae {
namespace {

using namespace q8;

typedef int v4i __attribute__((ext_vector_type(4)));

struct LinearQ8 {
    const int8_t *a, *w;
    long long lda, ldw, ldy;
    const float *sa, *sw, *bias;
    void* y;
    int M, N, K;
    int yvec;  // outputs can be stored 16 bytes at a time
};

// 16 bytes of a row from k on.  AL: the address is a multiple of 16.
// Otherwise the aligned words that hold them are read (every word holds one
// of the bytes, so none lies outside the row's memory) and shifted into
// place: a load from an odd address takes three times as long
// ([37, 1535, 6143]: 36 us against 11 aligned).
template <bool AL>
__device__ inline v4i load16(const int8_t* row, int k) {
    if (AL) return *reinterpret_cast<const v4i*>(row + k);
    const uintptr_t at = (uintptr_t)(row + k);
    const unsigned shift = (unsigned)at & 3;
    struct alignas(4) Words {
        unsigned w[4];
    };
    const Words x = *reinterpret_cast<const Words*>(at & ~(uintptr_t)3);
    const unsigned last = *reinterpret_cast<const unsigned*>((at + 15) & ~(uintptr_t)3);
    return (v4i){(int)__builtin_amdgcn_alignbyte(x.w[1], x.w[0], shift),
                 (int)__builtin_amdgcn_alignbyte(x.w[2], x.w[1], shift),
                 (int)__builtin_amdgcn_alignbyte(x.w[3], x.w[2], shift),
                 (int)__builtin_amdgcn_alignbyte(last, x.w[3], shift)};
}

// The same with zeros from K on.
__device__ inline v4i load16_tail(const int8_t* row, int k, int K) {
    v4i v;
    for (int i = 0; i < 4; ++i) {
        unsigned x = 0;
        for (int j = 0; j < 4; ++j)
            if (k + 4 * i + j < K) x |= (unsigned)(uint8_t)row[k + 4 * i + j] << (8 * j);
        v[i] = (int)x;
    }
    return v;
}

// SiLU's quick exponential is off by |v| 2^-23 of itself at most, under 2^-16
// where it is not 0: nothing to a 16-bit output.  A float32 one is computed to
// its own rounding.
template <typename T, bool SILU>
__device__ inline float epilogue(int acc, float sa, float sw, float bias) {
    const float v = fmaf((float)acc * sa, sw, bias);
    if (!SILU) return v;
    if (sizeof(T) == 4) return v / (1.0f + expf(-v));
    // (in eighths: the reciprocal of a number over 2^126 would be 0)
    return 0.125f * v * __builtin_amdgcn_rcpf(fmaf(0.125f, __expf(-v), 0.125f));
}

// Four outputs of row m from column n on: their scales, and the store.
struct Scales4 {
    float sa, sw[4], bias[4];
};

__device__ inline Scales4 scales4(const LinearQ8& p, int m, int n) {
    Scales4 s;
    s.sa = p.sa[m];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int c = min(n + r, p.N - 1);
        s.sw[r] = p.sw[c];
        s.bias[r] = p.bias ? p.bias[c] : 0.0f;
    }
    return s;
}

template <typename T, bool SILU>
__device__ inline void store4(const LinearQ8& p, int m, int n, v4i acc, const Scales4& s) {
    T* y = (T*)p.y + (long long)m * p.ldy + n;
    Pack<T, 4> out;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        out.v[r] = round_to<T>(epilogue<T, SILU>(acc[r], s.sa, s.sw[r], s.bias[r]));
    if (p.yvec) {
        *reinterpret_cast<Pack<T, 4>*>(y) = out;
    } else if (n + 4 <= p.N) {
        __builtin_memcpy(y, &out, sizeof(out));
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < p.N) y[r] = out.v[r];
    }
}

// Few rows: 16 NT weight rows by 16 MT activation rows a workgroup, K split
// over its waves, operands straight from memory to registers, the waves'
// sums joined in LDS.  The weights are read once for every 16 MT rows; the
// activations come from the L2.
template <typename T, bool SILU, bool AL, int MT, int NT>
__global__ __launch_bounds__(512) void linear_q8_rows_kernel(LinearQ8 p) {
    static_assert(MT * NT <= 8, "a wave for each pair of tiles, 8 waves at most");
    __shared__ v4i s_sum[8 * MT * NT * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int i = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * (16 * NT), m0 = blockIdx.y * (16 * MT);
    const int8_t* wr[NT];
    const int8_t* ar[MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        wr[t] = p.w + (long long)min(n0 + 4 * NT * (i >> 2) + 4 * t + (i & 3), p.N - 1) * p.ldw;
#pragma unroll
    for (int t = 0; t < MT; ++t) ar[t] = p.a + (long long)min(m0 + 16 * t + i, p.M - 1) * p.lda;
    // the outputs that this thread joins and stores, their scales fetched ahead
    const int l = threadIdx.x & 63, pair = threadIdx.x >> 6;
    const int out_m = m0 + 16 * (pair % MT) + (l & 15);
    const int out_n = n0 + 4 * NT * (l >> 4) + 4 * (pair / MT);
    const bool out = pair < NT * MT && out_m < p.M && out_n < p.N;
    Scales4 sc;
    if (out) sc = scales4(p, out_m, out_n);
    const int steps = (p.K + 63) / 64;
    const int per = ((steps + waves - 1) / waves + 1) & ~1;  // whole cache lines a wave
    const int s1 = min((wave + 1) * per, steps), full = min(s1, p.K / 64);
    int s = wave * per;
    v4i acc[NT][MT] = {};
    // steps of a batch: as many as 96 registers hold the operands of (the
    // compiler spreads their loads among the products)
    constexpr int U = 24 / (MT + NT) < 8 ? 24 / (MT + NT) : 8;
    for (; s + U <= full; s += U) {
        v4i wv[U][NT], av[U][MT];
        // a row's steps one after the other: two of them share a cache line
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int u = 0; u < U; ++u) wv[u][t] = load16<AL>(wr[t], (s + u) * 64 + 16 * g);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int u = 0; u < U; ++u) av[u][t] = load16<AL>(ar[t], (s + u) * 64 + 16 * g);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int v = 0; v < MT; ++v)
                    acc[t][v] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[u][t], av[u][v], acc[t][v],
                                                                      0, 0, 0);
    }
    for (; s < s1; ++s) {
        v4i wv[NT], av[MT];
        const int k = s * 64 + 16 * g;
        if (s < full) {
#pragma unroll
            for (int t = 0; t < NT; ++t) wv[t] = load16<AL>(wr[t], k);
#pragma unroll
            for (int t = 0; t < MT; ++t) av[t] = load16<AL>(ar[t], k);
        } else {
#pragma unroll
            for (int t = 0; t < NT; ++t) wv[t] = load16_tail(wr[t], k, p.K);
#pragma unroll
            for (int t = 0; t < MT; ++t) av[t] = load16_tail(ar[t], k, p.K);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int v = 0; v < MT; ++v)
                acc[t][v] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[t], av[v], acc[t][v], 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int v = 0; v < MT; ++v)
            s_sum[((wave * NT + t) * MT + v) * 64 + lane] = acc[t][v];
    __syncthreads();
    if (out) {
        v4i sum = s_sum[threadIdx.x];
        for (int w = 1; w < waves; ++w) sum += s_sum[w * (NT * MT * 64) + threadIdx.x];
        store4<T, SILU>(p, out_m, out_n, sum, sc);
    }
}

// Waits for this wave's memory operations, LDS DMA included (vmcnt 0; expcnt
// and lgkmcnt at their maxima): put before the barrier that publishes a
// staged buffer.
__device__ __forceinline__ void wait_dma() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// Many rows: a tile of BM x BN outputs a workgroup, 128 bytes of K a step,
// staged in two LDS buffers; each wave owns 16 MTW rows by 64 columns.
//
// A staged row is 128 bytes, its 16-byte chunks stored at chunk ^ key(row),
// so that the 16 rows that a fragment read takes at one logical chunk lie
// over all the banks.  The DMA writes LDS in lane order; the permutation is
// in the addresses that the lanes read from.
//
// DMA: rows and bases are multiples of 16 bytes; the next step's tiles come
// in by LDS DMA during the products of this one.  Otherwise they pass
// through registers.
template <typename T, bool SILU, bool DMA, int WGM, int WGN, int MTW, int KS>
__global__ __launch_bounds__(WGM* WGN * 64) void linear_q8_tile_kernel(LinearQ8 p, int m_tiles,
                                                                       int n_tiles, int group) {
    constexpr int NW = WGM * WGN, BM = WGM * MTW * 16, BN = WGN * 64;
    constexpr int JA = BM / 8 / NW, JW = BN / 8 / NW;  // 1 KB pieces a wave stages
    static_assert(JA * 8 * NW == BM && JW * 8 * NW == BN, "whole pieces");
    constexpr int PART = (BM + BN) * 128, STEP = KS * 128;
    __shared__ __align__(16) int8_t s_even[KS * PART];
    __shared__ __align__(16) int8_t s_odd[KS * PART];
    // (a wave index known to be scalar moves the staging addresses to the
    // scalar unit, ahead of each DMA: 584 against 483 us at 8192^3)
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i = lane & 15, g = lane >> 4;

    // the j-th 1 KB piece (8 staged rows) of this wave
    auto piece = [&](int j) { return j < JA ? wave + NW * j : BM / 8 + wave + NW * (j - JA); };
    int m0, n0;
    const int8_t *ab, *wb;
    int aoff[JA], woff[JW];
    // `group` row tiles sweep all column tiles together: what they stage
    // stays in the XCD's L2
    auto take = [&](int id) {
        const int tile = xcd_remap(id, m_tiles * n_tiles);
        const int span = group * n_tiles, first = tile / span * group;
        const int rows = min(group, m_tiles - first), in = tile % span;
        m0 = (first + in % rows) * BM;
        n0 = in / rows * BN;
        ab = p.a + (long long)m0 * p.lda;
        wb = p.w + (long long)n0 * p.ldw;
#pragma unroll
        for (int j = 0; j < JA; ++j) {
            const int r = 8 * (wave + NW * j) + (lane >> 3);
            aoff[j] = min(r, p.M - 1 - m0) * (int)p.lda + 16 * ((lane & 7) ^ (r & 7));
        }
#pragma unroll
        for (int j = 0; j < JW; ++j) {
            const int r = 8 * (wave + NW * j) + (lane >> 3);
            woff[j] = min(r, p.N - 1 - n0) * (int)p.ldw +
                      16 * ((lane & 7) ^ ((r & 3) | ((r >> 2) & 4)));
        }
    };
    const int wm = wave / WGN, wn = wave % WGN;
    v4i reg[DMA ? 1 : KS * (JA + JW)];

    // a whole step on its way to the buffer: begun before the products of
    // the step ahead, ended after them
    auto stage_begin = [&](int8_t* s, int k) {
#pragma unroll
        for (int q = 0; q < KS; ++q)
#pragma unroll
            for (int j = 0; j < JA + JW; ++j) {
                const bool is_w = j >= JA;
                const int8_t* from = (is_w ? wb : ab) + k + 128 * q;
                const int off = is_w ? woff[j - JA] : aoff[j];
                if constexpr (DMA)
                    __builtin_amdgcn_global_load_lds(
                        (const void*)(from + off),
                        (__attribute__((address_space(3))) void*)(s + q * PART +
                                                                  piece(j) * 1024),
                        16, 0, 0);
                else
                    __builtin_memcpy(&reg[q * (JA + JW) + j], from + off, 16);
            }
    };
    auto stage_end = [&](int8_t* s) {
        if constexpr (!DMA) {
#pragma unroll
            for (int q = 0; q < KS; ++q)
#pragma unroll
                for (int j = 0; j < JA + JW; ++j)
                    *reinterpret_cast<v4i*>(s + q * PART + piece(j) * 1024 + lane * 16) =
                        reg[q * (JA + JW) + j];
        }
    };
    // what is left of K after the last whole step, with zeros behind it
    auto stage_rest = [&](int8_t* s, int k) {
#pragma unroll 1
        for (int j = wave; j < (BM + BN) / 8; j += NW) {
            const bool is_w = j >= BM / 8;
            const int r = 8 * (is_w ? j - BM / 8 : j) + (lane >> 3);
            const int c = (lane & 7) ^ (is_w ? (r & 3) | ((r >> 2) & 4) : r & 7);
            const int8_t* row = is_w ? wb + (long long)min(r, p.N - 1 - n0) * p.ldw
                                     : ab + (long long)min(r, p.M - 1 - m0) * p.lda;
            *reinterpret_cast<v4i*>(s + j * 1024 + lane * 16) =
                k + 16 * c + 16 <= p.K ? load16<DMA>(row, k + 16 * c)
                                       : load16_tail(row, k + 16 * c, p.K);
        }
    };
    v4i acc[4][MTW];
    auto products = [&](const int8_t* s) {
        const int8_t* sa = s + (wm * MTW * 16 + i) * 128;
        const int8_t* sw = s + (BM + wn * 64 + 16 * (i >> 2) + (i & 3)) * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int ca = 16 * ((4 * h + g) ^ (i & 7));
            const int cw = 16 * ((4 * h + g) ^ ((i & 3) | (i & 4)));
            v4i wv[4], av[MTW];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                wv[t] = *reinterpret_cast<const v4i*>(sw + 4 * t * 128 + cw);
#pragma unroll
            for (int t = 0; t < MTW; ++t)
                av[t] = *reinterpret_cast<const v4i*>(sa + 16 * t * 128 + ca);
#pragma unroll
            for (int v = 0; v < MTW; ++v)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    acc[t][v] =
                        __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[t], av[v], acc[t][v], 0, 0, 0);
        }
    };

    auto publish = [&]() {
        wait_dma();
        __syncthreads();
    };
    const int whole = p.K / STEP * STEP, tiles = m_tiles * n_tiles;
    take(blockIdx.x);
    if (whole) stage_begin(s_even, 0);
    for (int id = blockIdx.x; id < tiles;) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int v = 0; v < MTW; ++v) acc[t][v] = (v4i){};
        if (whole) {
            stage_end(s_even);
            publish();
            for (int k = 0;;) {
                const bool more = k + STEP < whole;
                if (more) stage_begin(s_odd, k + STEP);
#pragma unroll
                for (int q = 0; q < KS; ++q) products(s_even + q * PART);
                if (more) stage_end(s_odd);
                publish();
                if (!more) break;
                k += 2 * STEP;
                if (k < whole) stage_begin(s_even, k);
#pragma unroll
                for (int q = 0; q < KS; ++q) products(s_odd + q * PART);
                if (k < whole) stage_end(s_even);
                publish();
                if (k >= whole) break;
            }
        }
        for (int k = whole; k < p.K; k += 128) {
            stage_rest(s_even, k);
            publish();
            products(s_even);
            __syncthreads();
        }
        // the next tile's first step comes in while this one's outputs go out
        const int m_out = m0, n_out = n0;
        id += gridDim.x;
        if (id < tiles) {
            take(id);
            if (whole) stage_begin(s_even, 0);
        }

        // 16 consecutive outputs of MTW rows
        const int n = n_out + wn * 64 + 16 * g, ends = min(max(p.N - n, 0), 16);
        float sw[16], bias[16];
        if (ends == 16) {
            __builtin_memcpy(sw, p.sw + n, sizeof(sw));
            if (p.bias) __builtin_memcpy(bias, p.bias + n, sizeof(bias));
        } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                sw[c] = c < ends ? p.sw[n + c] : 0.0f;
                bias[c] = c < ends && p.bias ? p.bias[n + c] : 0.0f;
            }
        }
        if (!p.bias)
#pragma unroll
            for (int c = 0; c < 16; ++c) bias[c] = 0.0f;
        float sa[MTW];
#pragma unroll
        for (int v = 0; v < MTW; ++v) sa[v] = p.sa[min(m_out + (wm * MTW + v) * 16 + i, p.M - 1)];
        constexpr int E = 16 / sizeof(T);
#pragma unroll
        for (int v = 0; v < MTW; ++v) {
            const int m = m_out + (wm * MTW + v) * 16 + i;
            if (m >= p.M) continue;
            T* y = (T*)p.y + (long long)m * p.ldy + n;
#pragma unroll
            for (int c = 0; c < 16; c += E) {
                Pack<T, E> out;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    out.v[e] = round_to<T>(epilogue<T, SILU>(acc[(c + e) / 4][v][(c + e) % 4], sa[v],
                                                          sw[c + e], bias[c + e]));
                if (p.yvec) {
                    // past the caches, which the operands need
                    // ([6000, 8192, 2048]: 135 -> 118 us)
                    typedef unsigned u4 __attribute__((ext_vector_type(4)));
                    if (c < ends)
                        __builtin_nontemporal_store(__builtin_bit_cast(u4, out),
                                                    reinterpret_cast<u4*>(y + c));
                } else if (c + E <= ends) {
                    __builtin_memcpy(y + c, &out, sizeof(out));
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (c + e < ends) y[c + e] = out.v[e];
                }
            }
        }
    }
}

// Rows of K bytes at any address to rows of `width` bytes, a multiple of 128,
// with zeros behind them: what the tiles are staged from by DMA.  A wave a
// row, the activations' first.
__global__ __launch_bounds__(256) void pack_q8_kernel(LinearQ8 p, int8_t* __restrict__ out,
                                                      int width) {
    for (long long row = blockIdx.x * 4LL + (threadIdx.x >> 6); row < (long long)p.M + p.N;
         row += gridDim.x * 4LL) {
        const int8_t* from = row < p.M ? p.a + row * p.lda : p.w + (row - p.M) * p.ldw;
        for (int k = (threadIdx.x & 63) * 16; k < width; k += 1024)
            *reinterpret_cast<v4i*>(out + row * width + k) =
                k + 16 <= p.K ? load16<false>(from, k) : load16_tail(from, k, p.K);
    }
}

constexpr int kCus = 256;

template <typename T, bool SILU, bool AL, int MT, int NT>
hipError_t run_rows(const LinearQ8& p, hipStream_t stream) {
    const int steps = (p.K + 63) / 64;
    const int waves = max(steps < 8 ? steps : 8, MT * NT);  // one for each pair of tiles at least
    hipLaunchKernelGGL((linear_q8_rows_kernel<T, SILU, AL, MT, NT>),
                       dim3((p.N + 16 * NT - 1) / (16 * NT), (p.M + 16 * MT - 1) / (16 * MT)),
                       dim3(64 * waves), 0, stream, p);
    return hipGetLastError();
}

template <typename T, bool SILU, bool DMA, int WGM, int WGN, int MTW, int KS>
hipError_t run_tile(const LinearQ8& p, hipStream_t stream) {
    constexpr int BM = WGM * MTW * 16, BN = WGN * 64;
    const int mt = (p.M + BM - 1) / BM, nt = (p.N + BN - 1) / BN;
    // a workgroup that has a CU to itself takes one tile after another
    const int grid = BM * BN * 2 >= 96 * 1024 ? std::min(mt * nt, kCus) : mt * nt;
    hipLaunchKernelGGL((linear_q8_tile_kernel<T, SILU, DMA, WGM, WGN, MTW, KS>), dim3(grid),
                       dim3(WGM * WGN * 64), 0, stream, p, mt, nt, 4);
    return hipGetLastError();
}

long long tiles(int M, int N, int bm, int bn) {
    return (long long)((M + bm - 1) / bm) * ((N + bn - 1) / bn);
}

// Whether the rows kernel takes a product.  It re-reads an operand for each
// 64 x 32 outputs; from more of those than CUs on, the tiles win
// ([128, 6144, 1536]: 12.5 against 8.5 us; [300, 1536, 6144], 240
// workgroups: 20.1 against 22).
bool by_rows(int M, int N) { return M <= 16 || tiles(M, N, 64, 32) <= kCus; }

// Which kernel: by the workgroups that each makes of M x N (times measured on
// [M, N, K], bfloat16 output).
template <typename T, bool SILU, bool AL>
hipError_t run(const LinearQ8& p, hipStream_t stream) {
    const auto tiles = [&](int bm, int bn) { return avae::tiles(p.M, p.N, bm, bn); };
    // (offsets inside a tile are 32 bits)
    if (by_rows(p.M, p.N) || p.lda >= (1 << 22) || p.ldw >= (1 << 22)) {
        // the largest tiles that leave at least 144 workgroups, bfloat16:
        // ([37, 1536, 6144]: 16 x 16 12.1 us, 32 x 16 11.1, 32 x 32 13.8;
        // [37, 6144, 1536]: 16 x 16 10.9, 32 x 16 9.6, 64 x 32 6.7; at the
        // limit, K = 6144: [1, 4608] 144 workgroups of 16 x 32 8.9 against
        // 9.8 of 16 x 16, [1, 4096] 128 of them 8.8 against 7.1; [64, 4608]
        // 144 of 64 x 32 19.8 against 24.4, [64, 4096] 128 19.7 against 13.9)
        if (p.M > 32 && tiles(64, 32) >= 144) return run_rows<T, SILU, AL, 4, 2>(p, stream);
        if (p.M > 16 && tiles(32, 32) >= 144) return run_rows<T, SILU, AL, 2, 2>(p, stream);
        if (p.M > 16 && tiles(32, 16) >= 144) return run_rows<T, SILU, AL, 2, 1>(p, stream);
        if (p.M <= 16 && tiles(16, 32) >= 144) return run_rows<T, SILU, AL, 1, 2>(p, stream);
        return run_rows<T, SILU, AL, 1, 1>(p, stream);
    }
    if constexpr (AL) {
        // up to two 64 x 64 tiles a CU ([1000, 1536, 1536]: 11.0 us, 64 x 128
        // 12.7; [512, 6144, 1536], three a CU: 18.9 against 15.1)
        if (tiles(64, 64) <= 2 * kCus) return run_tile<T, SILU, true, 2, 1, 2, 2>(p, stream);
        // the large tiles fill the CUs in rounds; a 64 x 128 one costs half
        // as much again for its area, but leaves no CU idle
        // ([6000, 6144, 1536]: 256 x 256 103 us, 192 x 256 87, 64 x 128 104;
        // [8192, 8192, 8192]: 476, 532, 713; [2048, 1536, 6144]: 78, 64, 38)
        const auto rounds = [&](int bm) {
            return (double)((tiles(bm, 256) + kCus - 1) / kCus) * bm * 256;
        };
        const double small = 1.5 * p.M * p.N / kCus;
        if (rounds(256) < rounds(192) && rounds(256) < small)
            return run_tile<T, SILU, true, 2, 4, 8, 1>(p, stream);
        if (rounds(192) < small) return run_tile<T, SILU, true, 2, 4, 6, 1>(p, stream);
    }
    return run_tile<T, SILU, AL, 2, 2, 2, 1>(p, stream);
}

template <typename T, bool SILU>
hipError_t linear_q8(LinearQ8 p, void* ws, hipStream_t stream) {
    const bool al = (((uintptr_t)p.a | (uintptr_t)p.w | p.lda | p.ldw) & 15) == 0;
    if (al) return run<T, SILU, true>(p, stream);
    if (linear_q8_workspace_bytes(p.M, p.N, p.K) == 0) return run<T, SILU, false>(p, stream);
    // large and not aligned: laid out anew for the DMA, which pays from the
    // first tiles on ([6000, 6143, 1535]: 104 us, 285 straight from memory)
    int8_t* rows = (int8_t*)ws;
    const int width = (p.K + 127) / 128 * 128;
    // (a launch has fewer than 2^32 threads)
    const unsigned groups = (unsigned)std::min(((long long)p.M + p.N + 3) / 4, 1LL << 22);
    hipLaunchKernelGGL(pack_q8_kernel, dim3(groups), dim3(256), 0, stream, p, rows, width);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.a = rows;
    p.w = rows + (long long)p.M * width;
    p.lda = p.ldw = p.K = width;
    return run<T, SILU, true>(p, stream);
}

}  // namespace

// Rows whose length is no multiple of 16 bytes are laid out anew where the
// product is large enough for tiles.
size_t linear_q8_workspace_bytes(int M, int N, int K) {
    if (K % 16 == 0 || by_rows(M, N)) return 0;
    return ((size_t)M + N) * ((K + 127) / 128 * 128);
}

hipError_t launch_linear_q8(const int8_t* a, long long lda, const float* sa, const int8_t* w,
                            long long ldw, const float* sw, const float* bias, int M, int N, int K,
                            int act, int dtype, void* y, long long ldy, void* ws,
                            hipStream_t stream) {
    const int es = dtype == AVAE_F32 ? 4 : 2;
    const LinearQ8 p{a,  w, lda, ldw, ldy, sa, sw, bias, y, M, N, K,
                     (N * es) % 16 == 0 && (ldy * es) % 16 == 0 && ((uintptr_t)y & 15) == 0};
    prof_pre(stream);
    hipError_t e;
    if (dtype == AVAE_F32)
        e = act ? linear_q8<float, true>(p, ws, stream) : linear_q8<float, false>(p, ws, stream);
    else if (dtype == AVAE_BF16)
        e = act ? linear_q8<__bf16, true>(p, ws, stream) : linear_q8<__bf16, false>(p, ws, stream);
    else
        e = act ? linear_q8<_Float16, true>(p, ws, stream) : linear_q8<_Float16, false>(p, ws, stream);
    prof_post(stream, "linear_q8_kernel", 2.0 * M * N * K,
              (double)M * K + (double)N * K + (double)M * N * es);
    return e;
}

}  // namespace avae
