// tree_attn.h - what the two forms of the tree attention share (tree_attn.cu: CUDA cores and
// f32 throughout; tree_tc.cu: tensor cores on 16-bit operands).
#pragma once

#include <type_traits>

#include "qw_ops.h"

namespace qw {

struct TreeArgs {
    const uint8_t *k, *v;
    const __half *ks, *vs;
    int64_t seq, head, pos, sseq, shead, spos;
    const void *q;
    void *out;
    int dtype;                   // of q and out
    int64_t qseq, qnode, qhead, oseq, onode, ohead;
    const unsigned long long *mask;
    const int32_t *len, *count;
    int n_max, max_ctx, Hkv, G, S, row_tiles;
    float scale_log2;
    float *part;                 // [n_seq][Hkv][n_max * G][S][D + 2]
};

// The same with a prefix that all sequences see, in planes of its own: [head][position][dim] (prefix attention).
struct PrefixArgs : TreeArgs {
    const uint8_t *pk, *pv;
    const __half *pks, *pvs;
    int64_t phead, ppos, pshead, pspos;
    const int32_t *plen;
    int p_max, n_seq;
    int Sp, p_row_tiles, p_blocks;  // CUDA-core form: splits of the prefix, tiles of all sequences' rows, their blocks
    unsigned long long inv_rows;    // 2^32 / (n_max G) + 1: row / (n_max G) for fewer than 2^20 rows
    unsigned long long inv_g;
};
template <bool PREFIX>
using AttnArgs = typename std::conditional<PREFIX, PrefixArgs, TreeArgs>::type;

// The prefix's length, if it fits its cache; else every row is NaN.
__device__ __forceinline__ bool prefix_length(const PrefixArgs &a, int &len) {
    len = *a.plen;
    return len >= 0 && len <= a.p_max;
}

// The drafted rows that node i of sequence b sees: its mask, or without masks itself and the ones before it.
__device__ __forceinline__ unsigned long long node_mask(const TreeArgs &a, int b, int i) {
    return a.mask ? a.mask[(int64_t)b * a.n_max + i] : ~0ull >> (63 - i);
}

__device__ __forceinline__ float load_q(const TreeArgs &a, int64_t at) {
    return a.dtype == QW_DT_F32   ? reinterpret_cast<const float *>(a.q)[at]
           : a.dtype == QW_DT_F16 ? __half2float(reinterpret_cast<const __half *>(a.q)[at])
                                  : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(a.q)[at]);
}

__device__ __forceinline__ void store_out(const TreeArgs &a, int64_t at, float v) {
    if (a.dtype == QW_DT_F32) reinterpret_cast<float *>(a.out)[at] = v;
    else if (a.dtype == QW_DT_F16) reinterpret_cast<__half *>(a.out)[at] = __float2half_rn(v);
    else reinterpret_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
}

// Whether sequence b's lengths fit its cache; if not its rows come out as NaN.
__device__ __forceinline__ bool lengths(const TreeArgs &a, int b, int &len, int &n) {
    len = a.len[b];
    n = a.count ? a.count[b] : a.n_max;
    return n >= 0 && n <= a.n_max && len >= 0 && len <= a.max_ctx - n;
}

// Tensor-core form.  CTAs of a launch (one per SM of a GB300; a launch with fewer tiles takes
// fewer), positions per tile, query rows per tile.
constexpr int kTcCtas = 152;
constexpr int kTcTile = 128;
constexpr int kTcRows = 128;
constexpr size_t kTcStatusBytes = 1024;  // one status word per CTA, then the partials
static_assert(kTcCtas * 4 <= kTcStatusBytes, "status words");

size_t tree_tc_scratch_bytes(int rows, int head_dim);
cudaError_t launch_tree_tc(const TreeArgs &a, const qw_kv_view &kv, int max_len, void *scratch, cudaStream_t st,
                           bool chained);
size_t prefix_tc_scratch_bytes(int64_t rows, int head_dim);
cudaError_t launch_prefix_tc(const PrefixArgs &a, const qw_kv_view &prefix, const qw_kv_view &kv, int max_len, int max_prefix,
                             void *scratch, cudaStream_t st, bool chained);

}  // namespace qw
