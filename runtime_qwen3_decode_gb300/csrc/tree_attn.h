// tree_attn.h - what the two forms of the tree attention share (tree_attn.cu: CUDA cores and
// f32 throughout; tree_tc.cu: tensor cores on 16-bit operands).
#pragma once

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

}  // namespace qw
