// Attention over the 8-bit paged cache, without rules (kernels: q8_attn.h).
#include "q8_attn.h"

namespace avae {

size_t attn_q8_workspace_bytes(int seqs, int total, int max_rows, int max_len, int q_heads,
                               int heads, int dim, int elem, int window, int prefix,
                               bool rules) {
    const Cut k = cut(seqs, max_rows, max_len, q_heads, heads, dim, elem, window, prefix, rules);
    return k.splits > 1 ? (size_t)total * q_heads * k.splits * (dim + 4) * sizeof(float) : 0;
}

long long attn_q8_workgroups(int seqs, int total, int max_rows, int max_len, int q_heads,
                             int heads, int dim, int elem, int window, int prefix,
                             bool rules) {
    const Cut k = cut(seqs, max_rows, max_len, q_heads, heads, dim, elem, window, prefix, rules);
    const int wide = k.mid ? mid_wide_waves(dim) : wide_waves(dim, elem);
    const long long blocks =
        (k.mid ? mid_blocks(k, heads, seqs) : (long long)k.tiles * k.splits * heads * seqs) *
        (k.wide ? wide / kWaves : 1);
    if (k.splits == 1) return blocks;
    // a join with rules goes by the sequences, as many rows for each as one may have
    const long long rows = (long long)total * q_heads;
    const long long joined = rules ? (long long)max_rows * q_heads * seqs : rows;
    return std::max(blocks, join_by_waves(k.splits, rows) ? joined / 4 + 1 : 2 * joined);
}

hipError_t launch_attn_q8(int dtype, const AttnQ8& a, const CacheQ8& c, const Ragged& r, void* ws,
                          hipStream_t stream) {
    return launch_attn(dtype, a, NoRules{}, c, r, ws, "attn_q8_kernel", stream);
}

}  // namespace avae
