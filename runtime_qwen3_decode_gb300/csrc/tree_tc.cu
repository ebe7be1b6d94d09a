// tree_tc.cu - the tensor-core form of the attention of drafted-token trees (tree_tc.cuh): its merge and launches.
#include "tree_tc.cuh"

namespace qw {
namespace {

// Merge of the items that were cut: thread = (row, four dims) of one (row tile, KV head, sequence).
// The partials lie row-fastest, so a warp's loads are runs of neighbours, and the loads of
// kMergeBatch partials are in flight at once: this kernel is nothing but their latency.  What
// does not depend on the partials comes before the wait for them, and small blocks without
// shared memory find room beside the attention's, so that they are there when it ends.
// Also fills the rows of sequences that do not fit with NaN, and every row if a CTA gave up.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_tc_merge_kernel(const Tree p, int ctas) {
    const TreeArgs &a = p.a;
    const int nrt_max = (a.n_max * a.G + kTcRows - 1) / kTcRows;
    const int rt = blockIdx.x % nrt_max, h = blockIdx.x / nrt_max, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31;
    int len, n;
    const bool fits = lengths(a, b, len, n);
    const int rows = (fits ? n : a.n_max) * a.G, r0 = rt * kTcRows;
    const int nr = min(kTcRows, rows - r0);
    const int e = blockIdx.z * kMergeThreads + tid, rl = nr > 0 ? e % nr : 0, dq = nr > 0 ? e / nr : D, r = r0 + rl;
    long long before = 0, total = 0;
    for (int i = lane; i < p.n_seq; i += 32) {
        const long long w = seq_work(p, i);
        total += w;
        if (i < b) before += w;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    const int nrt = (n * a.G + kTcRows - 1) / kTcRows, tiles = seq_tiles(len + n);
    int c0 = 0, c1 = 0;
    if (fits && n > 0) {
        // owner of tile t: the largest c with T c / C <= t
        const long long t0 = before + ((long long)h * nrt + rt) * tiles, t1 = t0 + tiles;
        c0 = (int)(total < (1 << 24) ? ((unsigned)(t0 + 1) * (unsigned)ctas - 1) / (unsigned)total : ((t0 + 1) * ctas - 1) / total);
        c1 = (int)(total < (1 << 24) ? ((unsigned)t1 * (unsigned)ctas - 1) / (unsigned)total : (t1 * ctas - 1) / total);
    }
    chain_wait();
    int gave_up = 0;  // read here, looked at behind the partials' loads
#pragma unroll
    for (int i = 0; i < (kTcCtas + 31) / 32; ++i) gave_up |= p.status[min(lane + 32 * i, ctas - 1)];
    const int64_t at = b * a.oseq + (int64_t)p.node_of(r) * a.onode + (int64_t)(h * a.G + r - p.node_of(r) * a.G) * a.ohead + 4 * dq;
    if (dq >= D / 4) c1 = c0;
    float num[4] = {0.f, 0.f, 0.f, 0.f}, den = 0.f, mx;
    add_partials<D>(p, ctas, total, c0, c1, rl, dq, num, den, mx);
    gave_up = __any_sync(0xffffffffu, gave_up);
    if (dq >= D / 4) return;
    if (!fits || gave_up) {
        for (int i = 0; i < 4; ++i) store_out(a, at + i, nanf(""));
        return;
    }
    if (c0 == c1) return;  // finished by its one CTA
    if (den == 0.f) den = 1.f;  // a row that sees nothing: 0
#pragma unroll
    for (int k = 0; k < 4; ++k) num[k] /= den;
    uint2 o;
    if (a.dtype == QW_DT_F16) o = make_uint2(pack2<false>(num[0], num[1]), pack2<false>(num[2], num[3]));
    else o = make_uint2(pack2<true>(num[0], num[1]), pack2<true>(num[2], num[3]));
    *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(a.out) + at) = o;
}

template <int D>
cudaError_t launch_tree_dim(const Tree &p, const qw_kv_view &kv, int ctas, cudaStream_t st, bool chained) {
    const cudaError_t e = launch_dim<D>(p, kv, nullptr, ctas, st, chained);
    if (e != cudaSuccess) return e;
    const int nrt = (p.a.n_max * p.a.G + kTcRows - 1) / kTcRows;
    const int units = std::min(kTcRows, p.a.n_max * p.a.G) * (D / 4);
    return launch_k(true, tree_tc_merge_kernel<D>, dim3(nrt * p.a.Hkv, p.n_seq, (units + kMergeThreads - 1) / kMergeThreads),
                    dim3(kMergeThreads), 0, st, p, ctas);
}

}  // namespace

size_t tree_tc_scratch_bytes(int rows, int head_dim) {
    return kTcStatusBytes + (size_t)2 * kTcCtas * (head_dim + 2) * slot_rows(rows) * 4;
}

cudaError_t launch_tree_tc(const TreeArgs &a, const qw_kv_view &kv, int max_len, void *scratch, cudaStream_t st,
                           bool chained) {
    Tree p{};
    p.a = a;
    p.n_seq = kv.n_seq;
    p.rows_max = slot_rows(a.n_max * a.G);
    p.inv_g = (1ull << 32) / a.G + 1;
    p.status = (int *)scratch;
    p.part = (float *)((uint8_t *)scratch + kTcStatusBytes);
    const int nrt = (a.n_max * a.G + kTcRows - 1) / kTcRows;
    const long long tiles = (long long)kv.n_seq * kv.n_kv_heads * nrt * ((max_len + a.n_max + kTcTile - 1) / kTcTile);
    const int ctas = (int)std::min<long long>(kTcCtas, tiles);
    return kv.head_dim == 128 ? launch_tree_dim<128>(p, kv, ctas, st, chained) : launch_tree_dim<64>(p, kv, ctas, st, chained);
}

}  // namespace qw
