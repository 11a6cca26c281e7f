// Attention over the 8-bit cache for a few dozen to a few hundred query rows,
// the drafts of a sequence: a part of q8_attn.h.
//
// 32 rows of one cache head a workgroup, the keys of a chunk dealt to its
// waves 32 at a time, straight from memory to the matrix cores' registers
// (v_mfma_f32_32x32x16_f16, as in the kernel for many rows): no staging and
// no barrier in the loop, so that short rows leave no wave without work.  A
// wave's next keys are asked for as soon as it has converted the present
// ones, its next values after their product.  Each wave keeps its own
// maximum, sum and output; they are joined in LDS, and chunks by the kernels
// that join.
//
// The tiles of a sequence's rows read the same keys: they go to one XCD, one
// after the other, and find them in its L2 (the memory traffic of three tiles
// is one's).
//
// One tile is bound by HBM ([16 sequences of 12000 keys, 4 heads of 128], 24
// rows: 51 us, 3.9 TB/s), more by their vector instructions, 370 for 32 rows
// and 32 keys, half of them the conversion of keys and values (96 rows 91 us:
// the vector units are busy 65%, the matrix cores 17% of the cycles; 360
// accesses of the first cache a step).  Three waves a SIMD: with the rows'
// operands in registers there are two (96 rows 110 us when this took 101); two
// tiles a wave, which share the conversion and the accesses, leave two at best
// (144 for 101): a wave's step is a chain of instructions, which more waves
// hide better than fewer instructions shorten it.  Nor do fewer accesses help:
// keys loaded line by line and turned through LDS take as long (heads of 64,
// 96 rows: 74 us either way).
#pragma once

// Waves a SIMD of the kernel below: what its registers allow (heads of 256
// nearly: 1 to 7 a lane go to scratch).
constexpr int mid_residency(int dim) { return dim > 128 ? 2 : 3; }
// Waves of its workgroups where they take all the keys of their rows: what
// fits in LDS.
constexpr int mid_wide_waves(int dim) { return dim > 128 ? 4 : 8; }

template <int N>
__device__ inline Words<(N + 3) / 4> load_bytes(const int8_t* p) {  // N bytes, N-byte aligned
    if constexpr (N == 2) {
        Words<1> r;
        r.w[0] = *reinterpret_cast<const unsigned short*>(p);
        return r;
    } else {
        return load_words<N / 4>(p);
    }
}

template <typename T, int D, typename R, int W>
__global__ __launch_bounds__(64 * W, W > kWaves ? 2 : mid_residency(D)) void attn_q8_mid_kernel(
    AttnQ8 a, CacheQ8 c, Ragged r, R x, int splits, int chunk, int tiles, float* part) {
    constexpr bool kSplit = sizeof(T) == 4;
    constexpr int KC = D / 16;  // key operands of 16 dims
    constexpr int DT = D / 32;  // output tiles; a lane's values of one key, too
    constexpr int LD = D + 4, JD = 64 + 4;
    __shared__ __align__(16) h8 s_q[(kSplit ? 2 : 1) * KC * 64];
    __shared__ __align__(16) float s_out[W * 32 * JD];
    __shared__ float s_m[W * 32], s_l[W * 32];
    const int lane = threadIdx.x & 63, wave = wave_id(), n32 = lane & 31, g = lane >> 5;
    const int pairs = r.seqs * c.heads, tile = (blockIdx.x >> 3) % tiles;
    const long long unit = (long long)((blockIdx.x >> 3) / tiles) * 8 + (blockIdx.x & 7);
    if (unit >= (long long)pairs * splits) return;
    const int split = (int)(unit / pairs), in_all = (int)(unit % pairs);
    const int b = in_all / c.heads, head = in_all % c.heads;
    int cu0, n, len;
    if (!ragged_rows(r, b, cu0, n, len)) return;
    const int group = a.q_heads / c.heads, rows = n * group, r0 = tile * 32;
    if (r0 >= rows) return;
    const Row row = row_of(a, c, x, b, head, cu0, n, len, r0 + n32);
    // the row's values, on their way while the chunk is found
    Pack<T, 16> q_raw[D / 32];
    {
        const T* q = (const T*)a.q + (long long)row.tok * a.q_tok +
                     (long long)row.q_head * a.q_head + 16 * g;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) __builtin_memcpy(q_raw[j].v, q + 32 * j, sizeof(q_raw[j].v));
    }
    if (x.pieces) chunk = best_chunk(x, c, r, lane, group, 32, splits, 32 * W);
    const Row row0 = row_of(a, c, x, b, head, cu0, n, len, r0);
    const Row row1 = row_of(a, c, x, b, head, cu0, n, len, min(r0 + 31, rows - 1));
    const int first = a.first ? max(a.first[b], 0) : 0;
    const int any_lo = a.window ? max(first, len - n + r0 / group - a.window + 1) : first;
    const int any_hi = row1.hi, pre = row1.pre;
    // every row sees the keys from row1.lo to all_hi
    const int all_hi = x.tree ? min(row0.hi, len - n) : row0.hi;
    // keys [first, pre) of all rows, then those from `base` on, counted through
    int base = any_lo < any_hi ? any_lo & ~31 : 0, in_pre = 0;
    int u_lo = chunk_start(base, split, chunk);
    int u_hi = any_lo < any_hi ? min(u_lo + chunk, any_hi) : 0;
    if (first < pre) {
        in_pre = ((pre + 31) & ~31) - (first & ~31);
        base = max(base, (pre + 31) & ~31);
        u_lo = chunk_start(0, split, chunk);
        u_hi = min(u_lo + chunk, in_pre + max(any_hi - base, 0));
    }
    auto key_at = [&](int u) {
        if (first < pre) return u < in_pre ? (first & ~31) + u : base + (u - in_pre);
        return u;
    };
    if (splits > 1 && u_lo >= u_hi) {  // a chunk without keys
        if (threadIdx.x < 32 && row.live) {
            float* pr =
                part + (((long long)row.tok * a.q_heads + row.q_head) * splits + split) * LD;
            pr[0] = neg_inf();
            pr[1] = 0.0f;
        }
        return;
    }

    // The table entries of a step, read two steps ahead of their use.
    int entry[2];
    auto look_up = [&](int u) {
        const int t = key_at(u);
        entry[0] = page_entry(c, b, t >> c.shift);
        entry[1] = page_entry(c, b, (t + 16) >> c.shift);
    };
    // Keys: lane 32 g + n has dims 32 j + 16 g .. + 15 of key n; values: dims
    // DT n .. of the keys 16 u + 8 (k / 4) + 4 g + k % 4.
    Words<4> kw[D / 32];
    Words<(DT + 3) / 4> vw[2][8];
    float ks[2], vs[2], next_ks[2], next_vs[2];
    bool there[2], next_there[2];
    long long at[2];
    auto fetch_keys = [&](int u) {
        const int t = key_at(u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k0 = t + 16 * h;
            const int page =
                page_checked(c, k0 >> c.shift, __builtin_amdgcn_readfirstlane(entry[h]));
            // a half that no row sees may lie in a page that holds anything
            next_there[h] = page >= 0 && ((k0 < any_hi && k0 + 16 > any_lo) ||
                                          (k0 < pre && k0 + 16 > first));
            at[h] = (long long)max(page, 0) * c.heads + head;
            next_ks[h] = c.k_scale[at[h]];
            next_vs[h] = c.v_scale[at[h]];
            at[h] = (at[h] * c.page + (k0 & (c.page - 1))) * D;
        }
        const int8_t* from = c.k + (n32 < 16 ? at[0] : at[1]) + (n32 & 15) * D + 16 * g;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) kw[j] = load_words<4>(from + 32 * j);
    };
    auto fetch_values = [&]() {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int8_t* from = c.v + at[u] + 4 * g * D + DT * n32;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                vw[u][k] = load_bytes<DT>(from + ((k & 3) + 8 * (k >> 2)) * D);
        }
    };
    const int u_first = u_lo + 32 * wave;
    look_up(u_first);
    fetch_keys(u_first);
    fetch_values();
    look_up(u_first + 32 * W);

    const Shape<T, R> shape(x, row);
    // The rows are the same for all waves: their operands lie in LDS, in the
    // lanes' order, and leave the registers to another wave.
    float to_log2;  // not negative: the scale's sign goes into the rows
    {
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf((float)q_raw[j].v[i]));
        top = max_halves(top);
        const int e = min(max((int)((__float_as_uint(top) >> 23) & 255) - 127, -100), 127);
        const float up = copysignf(__uint_as_float((unsigned)(127 + 14 - e) << 23), a.scale);
        to_log2 = shape.held(
            __uint_as_float((unsigned)(127 - 14 + e) << 23) *
            (x.cap > 0.0f ? shape.held(fabsf(a.scale) / x.cap) : fabsf(a.scale) * kLog2e));
        if (wave == 0) {
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                h8 high, low;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = (float)q_raw[j / 2].v[j % 2 * 8 + i] * up;
                    high[i] = (_Float16)v;
                    low[i] = (_Float16)(v - (float)high[i]);
                }
                s_q[64 * j + lane] = high;
                if (kSplit) s_q[64 * (KC + j) + lane] = low;
            }
        }
    }
    __syncthreads();

    f16v acc[DT] = {};
    float m = neg_inf(), l = 0.0f;
    // The accumulated values are in units of 2^(lg_run - 15), lg_run the
    // largest logarithm of a value scale so far (below every one at first).
    float lg_run = -140.0f;

    for (int u0 = u_first; u0 < u_hi; u0 += 32 * W) {
        const int t0 = key_at(u0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ks[h] = next_ks[h];
            vs[h] = next_vs[h];
            there[h] = next_there[h];
        }
        asm volatile("" ::: "memory");  // (the operands are read anew each step)
        f16v s = {};
#pragma unroll
        for (int j = 0; j < KC; ++j) {
            const h8 kv = to_half8(kw[j / 2].w[j % 2 * 2], kw[j / 2].w[j % 2 * 2 + 1]);
            s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kv, s_q[64 * j + lane], s, 0, 0, 0);
            if (kSplit)
                s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kv, s_q[64 * (KC + j) + lane], s, 0, 0,
                                                           0);
        }
        // (what is asked for past the last step is of no use, and harmless)
        fetch_keys(u0 + 32 * W);
        look_up(u0 + 64 * W);

        float by[2] = {shape.by(ks[0], to_log2), shape.by(ks[1], to_log2)};
        shape_scores(shape, s, by, (float)(row.pos - (t0 + 4 * g)));
        float lg_vs[2], inv_vs[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            lg_vs[u] = finite(vs[u]) ? __builtin_amdgcn_logf(vs[u]) : neg_inf();
            inv_vs[u] = __builtin_amdgcn_rcpf(vs[u]);
        }
        bool part_seen = t0 < row1.lo || t0 + 32 > all_hi;
        part_seen &= t0 < first || t0 + 32 > row0.pre;
        if (__builtin_amdgcn_readfirstlane(part_seen || !there[0] || !there[1] ||
                                           !finite(vs[0] + vs[1]))) {
            // What is hidden from a row goes into its scores, and a value
            // scale that is not finite too: so it stays with the rows that
            // see it.  Scales of keys that a row does not see are not in its
            // reference.
            const unsigned seen = keys_seen(row, x, len - n, t0);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bool good = finite(vs[u]);
#pragma unroll
                for (int j = 8 * u; j < 8 * u + 8; ++j) {
                    const float y = good ? s[j] * by[u] : nan();
                    const bool on = seen >> (4 * g) & 1u << (8 * (j >> 2) + (j & 3));
                    s[j] = there[u] && on ? y : neg_inf();
                }
                by[u] = 1.0f;
                if (!there[u] || !(seen >> (16 * u) & 0xffffu)) lg_vs[u] = neg_inf();
                // (values of a page that holds anything are still numbers)
                if (!there[u] || !good) inv_vs[u] = 0.0f;
            }
        }
        // The row's references move only when a key passes them by so much
        // that p * vs would leave float16 (2^15 at the reference).
        float top[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            top[u] = s[8 * u];
#pragma unroll
            for (int j = 1; j < 8; ++j) top[u] = fmaxf(top[u], s[8 * u + j]);
        }
        const float m_new = fmaxf(m, max_halves(fmaxf(top[0] * by[0], top[1] * by[1])));
        const float lg_new = fmaxf(lg_run, fmaxf(lg_vs[0], lg_vs[1]));
        if (__any(m_new - m + (lg_new - lg_run) > 0.99f)) {
            const float back = __builtin_amdgcn_exp2f(m - (m_new == neg_inf() ? 0.0f : m_new));
            l *= back;
            const float to = back * __builtin_amdgcn_exp2f(lg_run - lg_new);
#pragma unroll
            for (int t = 0; t < DT; ++t) acc[t] *= to;
            m = m_new;
            lg_run = lg_new;
        }
        const float m_at = m == neg_inf() ? 0.0f : m;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            // probabilities times their value scale, straight from the
            // exponent; their sum is theirs over the same factor, kept 2^15
            // times as large
            const float lift = fmaxf(lg_vs[u] + 15.0f - lg_run, -60.0f) - m_at;
            const float drop = fminf(inv_vs[u] * __builtin_amdgcn_exp2f(lg_run), 0x1p75f);
            float sum = 0.0f;
            h8 ph, pl;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float x0 = __builtin_amdgcn_exp2f(fmaf(s[8 * u + j], by[u], lift));
                const float x1 = __builtin_amdgcn_exp2f(fmaf(s[8 * u + j + 1], by[u], lift));
                sum += x0 + x1;
                const h2 hx = __builtin_convertvector(((f2){x0, x1}), h2);
                ph[j] = hx[0];
                ph[j + 1] = hx[1];
                if (kTwoParts<T>) {
                    pl[j] = (_Float16)(x0 - (float)hx[0]);
                    pl[j + 1] = (_Float16)(x1 - (float)hx[1]);
                }
            }
            l = fmaf(sum, drop, l);
#pragma unroll
            for (int w = 0; w < (DT + 3) / 4; ++w) {
                // bytes of eight keys, four dims: pairs of keys, then halves
                unsigned lo01[4], hi01[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lo01[i] = pair_lo(vw[u][2 * i].w[w], vw[u][2 * i + 1].w[w]);
                    hi01[i] = pair_hi(vw[u][2 * i].w[w], vw[u][2 * i + 1].w[w]);
                }
#pragma unroll
                for (int e = 0; e < (DT < 4 ? DT : 4); ++e) {
                    h2 y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        y[i] = to_half2(e < 2 ? lo01[i] : hi01[i],
                                        (e & 1) ? 0x04030402u : 0x04010400u);
                    const h8 vv = __builtin_bit_cast(h8, y);
                    f16v o = acc[4 * w + e];
                    o = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, ph, o, 0, 0, 0);
                    if (kTwoParts<T>) o = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, pl, o, 0, 0, 0);
                    acc[4 * w + e] = o;
                }
            }
        }
        fetch_values();
    }

    l = (l + __shfl_xor(l, 32)) * 0x1p-15f;
    if (shape.quick && shape.capped) m += shape.cap;
    if (g == 0) {
        s_m[wave * 32 + n32] = m;
        s_l[wave * 32 + n32] = l;
    }
    // the unit in two halves, since it may be below float32
    const float half = __builtin_amdgcn_exp2f(0.5f * (lg_run - 15.0f));
    // joined 64 dims at a time
#pragma unroll
    for (int d0 = 0; d0 < D; d0 += 64) {
        constexpr int N = DT < 4 ? DT : 4, EACH = 64 / DT;  // rows of the stacked output tiles
        if (d0 > 0) __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (8 * (i >> 2) / EACH != d0 / 64) continue;
            const int at = DT * (8 * (i >> 2) + 4 * g + (i & 3)) - d0;
#pragma unroll
            for (int t = 0; t < DT; t += N) {
                Pack<float, N> o;
#pragma unroll
                for (int e = 0; e < N; ++e) o.v[e] = acc[t + e][i] * half * half;
                *reinterpret_cast<Pack<float, N>*>(s_out + (wave * 32 + n32) * JD + at + t) = o;
            }
        }
        __syncthreads();
        // each thread joins four dims of a row
        for (int e = threadIdx.x; e < 32 * 16; e += 64 * W) {
            const int i = e / 16, d = e % 16 * 4;
            const Row to = row_of(a, c, x, b, head, cu0, n, len, r0 + i);
            if (!to.live) break;  // rows come in order
            float top = neg_inf(), sum = 0.0f;
            for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w * 32 + i]);
            const float base_m = top == neg_inf() ? 0.0f : top;
            f4 o = {};
            for (int w = 0; w < W; ++w) {
                const float by = chunk_weight(s_m[w * 32 + i], s_l[w * 32 + i], base_m);
                if (by == 0.0f) continue;
                sum += by * s_l[w * 32 + i];
                o += by * *reinterpret_cast<const f4*>(s_out + (w * 32 + i) * JD + d);
            }
            const long long out_row = (long long)to.tok * a.q_heads + to.q_head;
            if (splits > 1) {
                float* pr = part + (out_row * splits + split) * LD;
                *reinterpret_cast<f4*>(pr + 4 + d0 + d) = o;
                if (d0 + d == 0) {
                    pr[0] = top;
                    pr[1] = sum;
                }
            } else {
                const float by = sum == 0.0f ? 0.0f : 1.0f / sum;  // a NaN sum stays NaN
                Pack<T, 4> y;
#pragma unroll
                for (int j = 0; j < 4; ++j) y.v[j] = round_to<T>(o[j] * by);
                *reinterpret_cast<Pack<T, 4>*>((T*)a.out + out_row * D + d0 + d) = y;
                if (a.lse && d0 + d == 0) a.lse[out_row] = lse_of(top, sum);
            }
        }
    }
}
