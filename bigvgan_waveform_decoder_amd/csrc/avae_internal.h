// Internal launch interface between the C-ABI layer and the HIP kernels.
// Not installed; include/avae.h is the public boundary.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace avae {

constexpr int kFilterLen = 12;

// Resampling taps passed by value to the activation kernel (they land in
// scalar registers).  up2 holds the upsampling taps already multiplied by
// the x2 gain of the transposed convolution (exact: a power of two).
struct ActTaps {
    float up2[kFilterLen];
    float down[kFilterLen];
};

// Epilogue of the Conv1d kernel:
//   v   = conv + bias[o], then Snake(v, snake_alpha[o]) if given, (+ residual[idx])
//   out = v * out_scale (+ out[idx] if accumulate)
// residual may alias out (same element read then written by one lane).
struct ConvEpilogue {
    const float* bias;         // [Cout] or null
    const float* residual;     // [B, Cout, Tout] or null
    float out_scale;
    int accumulate;
    const float* snake_alpha;  // [Cout] or null: plain Snake after the bias
    const float* in_alpha;     // [Cin] or null: plain Snake of the input as it is staged
};

// Launch profiler (profile.cpp).  prof_pre/prof_post bracket one launch;
// they do nothing unless a profiled region is open.  Phases: 0 dec_in,
// 1 conv_pre, 2 upsamples, 3 resblocks, 4 act_post, 5 conv_post, -1 none.
enum Phase { kPhaseNone = -1, kPhaseDecIn = 0, kPhaseConvPre = 1, kPhaseUpsamples = 2,
             kPhaseResblocks = 3, kPhaseActPost = 4, kPhaseConvPost = 5 };
void prof_set_phase(int phase);
void prof_pre(hipStream_t s);
void prof_post(hipStream_t s, const char* name, double flops, double bytes);

// Host-side float64 Kaiser-sinc design (filter_design.cpp).
void design_kaiser_sinc(double cutoff, double half_width, int taps, double* out);
// Host-side float64 Hann-sinc interpolator taps; returns the tap count
// (out may be null to query it).
int design_hann_sinc(int ratio, double rolloff, double lpw, double* out);

// y is written with non-temporal stores (not kept in the caches).
hipError_t launch_act1d(const float* x, float* y, int B, int C, int T,
                        const float* log_alpha, const float* log_beta,
                        const ActTaps& taps, hipStream_t stream);

// Returns hipErrorInvalidValue if the shape needs more LDS than a block has.
hipError_t launch_conv1d(const float* x, float* y, const float* w, int B, int Cin, int Cout,
                         int T, int Tout, int K, int dilation, int pad,
                         const ConvEpilogue& ep, hipStream_t stream);

// in_alpha: [Cin] or null, plain Snake applied to the input as it is staged.
hipError_t launch_convtr1d(const float* x, float* y, const float* w, const float* bias,
                           int B, int Cin, int Cout, int Tin, int Tout, int K, int stride,
                           int pad, hipStream_t stream, const float* in_alpha = nullptr);

// Conv1d through 256-point overlap-save transforms (fftconv.hip), "same"
// padding, shapes that plan::fft_supported takes.  wp holds
// fft_conv_weight_floats(Cin, Cout) floats from launch_fft_pack; xspec and
// yspec plan::fft_spectrum_bytes(B, Cin | Cout, T, K, d) bytes each.  With
// act_log_alpha, act_log_beta and act_taps all given, the convolution's
// input is Activation1d(x) (as launch_act1d computes it), evaluated inside
// the forward transforms; else with ep.in_alpha, the plain Snake of x there.
// ep.snake_alpha applies the plain Snake after the bias, as launch_conv1d.
size_t fft_conv_weight_floats(int Cin, int Cout);
hipError_t launch_fft_pack(const float* w, float* wp, int Cin, int Cout, int K, int dilation,
                           hipStream_t s);
hipError_t launch_conv1d_fft(const float* x, float* y, const float* wp, int B, int Cin, int Cout,
                             int T, int K, int dilation, const ConvEpilogue& ep, float* xspec,
                             float* yspec, hipStream_t s, const float* act_log_alpha = nullptr,
                             const float* act_log_beta = nullptr,
                             const ActTaps* act_taps = nullptr);

// Conv1d to a single output channel ("same" padding, odd K) followed by the
// final nonlinearity (0 none, 1 tanh, 2 clamp to [-1,1]).  pre_final, if not
// null, also receives the value before the nonlinearity ([B, T]).  With
// interleave2, input rows 2b and 2b+1 are the two stereo sides of output
// row b, written interleaved: y[b][2t + side].
hipError_t launch_conv_out1(const float* x, float* y, float* pre_final, const float* w,
                            const float* bias, int B, int Cin, int T, int K, int final_act,
                            int interleave2, hipStream_t stream,
                            const float* in_alpha = nullptr);

// Plain Snake (snake.hip): y = x + sin^2(alpha_c x) / (alpha_c + 1e-9).
hipError_t launch_snake(const float* x, float* y, int B, int C, int T, const float* alpha,
                        hipStream_t stream);

// Fused AMP unit (amp_unit.hip): y = x + conv2(act2(conv1(act1(x)))) for one
// dilation step, then y * out_scale (+ y_old if accumulate).  Narrow widths
// only (amp_unit_supported); the weights come packed by
// launch_pack_unit_weights into amp_unit_packed_floats(C, K) floats.  x and y
// must not overlap.
bool amp_unit_supported(int C, int K, int dilation);
size_t amp_unit_packed_floats(int C, int K);
hipError_t launch_pack_unit_weights(const float* w, float* wt, int C, int K, hipStream_t s);
// n <= 8 weights of one (C, K) packed in one launch.
hipError_t launch_pack_unit_weights_n(const float* const* w, float* const* wt, int n, int C,
                                      int K, hipStream_t s);
hipError_t launch_amp_unit(const float* x, float* y, const float* wt1, const float* b1,
                           const float* wt2, const float* b2, const float* la1, const float* lb1,
                           const float* la2, const float* lb2, int B, int C, int T, int K,
                           int dilation, float out_scale, int accumulate, const ActTaps& taps,
                           hipStream_t stream);

// Causal log-mel (bwe.hip): x [B, T] (zero beyond T) -> out [B, n_mels,
// frames], frame f covering padded samples [f hop, f hop + L) with L - hop
// zeros on the left; basis [2 nf, L], mel [n_mels, nf].
hipError_t launch_mel_stft(const float* x, float* out, int B, int T, int frames,
                           const float* basis, int nf, int L, int hop, const float* mel,
                           int n_mels, hipStream_t stream);
// out[b, t] (t < Lout) = [clamp](resid[b, t] + skip(t)), skip the x`ratio`
// interpolation (k host taps) of x zero-extended from T to Tp samples and
// replicate-padded; resid may be null (skip alone).
hipError_t launch_bwe_combine(const float* x, const float* resid, float* out, int B, int T,
                              int Tp, int Lres, int Lout, int ratio, const float* taps_host,
                              int k, int do_clamp, hipStream_t stream);

// y[i] += x[0][i] + ... + x[n-1][i] for i < count (n <= 3): the MRF sum of
// AMP blocks that ran concurrently into separate buffers.
hipError_t launch_sum_into(float* y, float* const* x, int n, size_t count, hipStream_t stream);

// Matrix-core throughput probe (probe.hip): `blocks` workgroups of 256
// threads, each wave running `chains` (8 or 16) independent FP32 MFMA
// accumulator chains for `iters` iterations; sink gets blocks*256 floats.
hipError_t launch_mfma_probe(int chains, int blocks, int iters, float* sink, hipStream_t s);
hipError_t launch_stream_copy(const float* x, float* y, long long n4, hipStream_t s);

// y[b,c,t] = x[b,c,t] * scale[c] + shift[c]
hipError_t launch_channel_affine(const float* x, float* y, const float* scale,
                                 const float* shift, int B, int C, int T, hipStream_t stream);

// ---- 8-bit serving operators (q8_*.hip).  dtype: enum avae_dtype.

// Sets the calling thread's avae_last_error() and returns `code`.
int abi_fail(int code, const char* fmt, ...);

// The paged cache and its page table, as include/avae.h describes them.
struct CacheQ8 {
    int8_t *k, *v;            // [n_pages][heads][page][dim]
    float *k_scale, *v_scale; // [n_pages][heads]
    const int* table;         // [seqs][table_ld], page of each column
    long long table_ld;
    int table_cols;
    int n_pages, heads, page, dim;
    int shift;                // page = 1 << shift
};

// Packed rows of `seqs` sequences: rows cu[b] .. cu[b+1] are the last ones of
// sequence b, which has lens[b] tokens.
struct Ragged {
    const int *cu, *lens;
    int seqs, total, max_rows;
};

// sum, res and w may be null (no residual; no norm).
hipError_t launch_rows_q8(int dtype, const void* x, long long ldx, const void* res, long long ldr,
                          const float* w, int M, int C, float eps, void* sum, long long lds,
                          int8_t* q, long long ldq, float* scale, hipStream_t stream);
hipError_t launch_dequant_q8(int dtype, const int8_t* q, long long ldq, const float* scale, int M,
                             int C, void* y, long long ldy, hipStream_t stream);
size_t linear_q8_workspace_bytes(int M, int N, int K);
hipError_t launch_linear_q8(const int8_t* a, long long lda, const float* sa, const int8_t* w,
                            long long ldw, const float* sw, const float* bias, int M, int N, int K,
                            int act, int dtype, void* y, long long ldy, void* ws,
                            hipStream_t stream);
// Pages of a sequence that a write's launch covers: what max_rows tokens can
// touch, at any place in the first of them, and no more than the table has.
int kv_write_q8_pages(const CacheQ8& c, const Ragged& r);
hipError_t launch_kv_write_q8(int dtype, const void* k, long long k_tok, long long k_head,
                              const void* v, long long v_tok, long long v_head, const CacheQ8& c,
                              const Ragged& r, hipStream_t stream);
hipError_t launch_kv_read_q8(int dtype, const CacheQ8& c, const Ragged& r, void* k, void* v,
                             hipStream_t stream);

// What turns the heads.  positions null: a row's place in its sequence.
struct RopeQ8 {
    const float* freq;     // [half] radians a position
    int half;              // pairs that are turned
    int apart;             // half where the dims of a pair are that far apart, 0: neighbours
    float amp;
    const int* positions;  // [total]
};

// Heads x [total][heads][dim] that go to y, at their strides; weight [dim]
// null: no norm.
struct HeadsQ8 {
    const void* x;
    void* y;
    const float* weight;
    long long tok, head, y_tok, y_head;
    int heads;
};
// r.cu null: all r.total rows (positions given).
hipError_t launch_qk_norm_rope(int dtype, const HeadsQ8& q, const HeadsQ8& k, const RopeQ8& rope,
                               const Ragged& r, int dim, float eps, hipStream_t stream);
hipError_t launch_kv_write_rope_q8(int dtype, const void* k, long long k_tok, long long k_head,
                                   const void* v, long long v_tok, long long v_head,
                                   const float* weight, float eps, const RopeQ8& rope,
                                   const CacheQ8& c, const Ragged& r, hipStream_t stream);
hipError_t launch_tree_mask(const int* parents, const Ragged& r, int words, int* mask,
                            long long ld, int* positions, hipStream_t stream);

struct AttnQ8 {
    const void* q;            // [total][q_heads][dim], strides q_tok, q_head
    long long q_tok, q_head;
    void* out;                // [total][q_heads][dim]
    float* lse;               // [total][q_heads] or null
    const int* first;         // [seqs] or null: keys before it are not seen
    int q_heads, max_len, causal, window;
    float scale;
};
// prefix: tokens in view whatever the window, at most (0 without a window).
size_t attn_q8_workspace_bytes(int seqs, int total, int max_rows, int max_len, int q_heads,
                               int heads, int dim, int elem, int window, int prefix = 0,
                               bool rules = false);
// Threads of its largest launch in units of 256, over all axes: those of the
// kernel, or of the join.
long long attn_q8_workgroups(int seqs, int total, int max_rows, int max_len, int q_heads,
                             int heads, int dim, int elem, int window, int prefix = 0,
                             bool rules = false);
hipError_t launch_attn_q8(int dtype, const AttnQ8& a, const CacheQ8& c, const Ragged& r, void* ws,
                          hipStream_t stream);

// What the attention does to its scores, and which keys a row sees besides.
struct AttnRules {
    float cap;              // 0: none
    const float* slopes;    // [q_heads] or null
    const int* prefix;      // [seqs] or null
    int max_prefix;
    const unsigned* tree;   // [total][tree_words] bits at stride tree_ld, or null
    long long tree_ld;
    int tree_words;
    int pieces, span;       // set by the launch: how the keys of many rows are cut
};
hipError_t launch_attn_rules_q8(int dtype, const AttnQ8& a, const AttnRules& x, const CacheQ8& c,
                                const Ragged& r, void* ws, hipStream_t stream);
// The same for 16-bit types under caps over 256.
hipError_t launch_attn_caps_q8(int dtype, const AttnQ8& a, const AttnRules& x, const CacheQ8& c,
                               const Ragged& r, void* ws, hipStream_t stream);

}  // namespace avae
