// prefix_tc.cu - the tensor-core form of the attention of a batch that shares a prefix (tree_tc.cuh): its merge and launches.
#include "tree_tc.cuh"

namespace qw {
namespace {

// Merge of the items that were cut: as in tree_tc.cu, (row, four dims) of one (row tile, KV head), but with SHARES threads in as many warps
// for each, which take every SHARES-th partial: with one row tile an item has some 20 of them, and the kernel is the latency of their
// loads (8 KV heads behind a prefix of 32768: 3.9 us with four threads, 7.2 with one; 64 row tiles, whose items are hardly cut,
// 100 us more).  Also fills the rows of sequences that do not fit with NaN, and every row if the prefix does not or a CTA gave up.
template <int D, int SHARES>
__global__ void __launch_bounds__(kMergeThreads) prefix_tc_merge_kernel(const Prefix p, int ctas) {
    const PrefixArgs &a = p.a;
    const int rt = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    const int nr = min(kTcRows, row_count(p) - rt * kTcRows);
    constexpr int UNITS = kMergeThreads / SHARES;
    __shared__ float part[SHARES][UNITS][6];  // a thread's sums and their reference
    const int share = tid / UNITS, unit = tid % UNITS;
    const int e = blockIdx.z * UNITS + unit, rl = e % nr, dq = e / nr;
    int b, node, g, len, n, plen;
    p.place(rt * kTcRows + rl, b, node, g);
    const bool fits = lengths(a, b, len, n) && prefix_length(a, plen);
    const int64_t at = b * a.oseq + (int64_t)node * a.onode + (int64_t)(h * a.G + g) * a.ohead + 4 * dq;
    chain_wait();
    const int nrt = row_tiles(p);
    const long long first = p.starts[rt], tiles = p.starts[rt + 1] - first, whole = p.starts[nrt];
    const bool by_item = p.starts[nrt + 1] != 0;
    const long long total = by_item ? ctas : whole * a.Hkv;  // no share is empty where items have CTAs of their own
    int gave_up = 0;
#pragma unroll
    for (int i = 0; i < (kTcCtas + 31) / 32; ++i) gave_up |= p.status[min(lane + 32 * i, ctas - 1)];
    int c0 = 0, c1 = 0;
    if (by_item && dq < D / 4) {
        const int k = (int)tiles / a.Hkv;
        if (k > 0) c0 = (int)first + h * k, c1 = c0 + k - 1;
    } else if (tiles > 0 && dq < D / 4) {
        // owner of tile t: the largest c with T c / C <= t
        const long long t0 = first * a.Hkv + h * tiles, t1 = t0 + tiles;
        c0 = (int)(total < (1 << 24) ? ((unsigned)(t0 + 1) * (unsigned)ctas - 1) / (unsigned)total : ((t0 + 1) * ctas - 1) / total);
        c1 = (int)(total < (1 << 24) ? ((unsigned)t1 * (unsigned)ctas - 1) / (unsigned)total : (t1 * ctas - 1) / total);
    }
    const bool there = fits && node < n;
    float num[4] = {0.f, 0.f, 0.f, 0.f}, den = 0.f, mx = -INFINITY;
    if (there) add_partials<D>(p, ctas, total, c0, c1, rl, dq, num, den, mx, share, SHARES);
    gave_up = __any_sync(0xffffffffu, gave_up);
    if constexpr (SHARES > 1) {
        float *mine = part[share][unit];
        mine[0] = mx, mine[1] = den;
#pragma unroll
        for (int k = 0; k < 4; ++k) mine[2 + k] = num[k];
        __syncthreads();
        if (share == 0) {
            float top = mx;
#pragma unroll
            for (int i = 1; i < SHARES; ++i) top = fmaxf(top, part[i][unit][0]);
            den = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) num[k] = 0.f;
#pragma unroll
            for (int i = 0; i < SHARES; ++i) {
                const float *x = part[i][unit];
                if (x[0] == -INFINITY && x[1] == 0.f) continue;  // nothing seen
                const float w = exp2f(x[0] - top);
                den += x[1] * w;
#pragma unroll
                for (int k = 0; k < 4; ++k) num[k] += x[2 + k] * w;
            }
        }
    }
    if (share != 0 || dq >= D / 4 || (fits && !there)) return;
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
cudaError_t launch_prefix_dim(const Prefix &p, const qw_kv_view &prefix, const qw_kv_view &kv, int ctas, cudaStream_t st, bool chained) {
    const cudaError_t e = launch_dim<D>(p, kv, &prefix, ctas, st, chained);
    if (e != cudaSuccess) return e;
    const int rows = p.n_seq * p.a.n_max * p.a.G, nrt = (rows + kTcRows - 1) / kTcRows, units = std::min(kTcRows, rows) * (D / 4);
    auto merge = [&](auto kernel, int per_block) {
        return launch_k(true, kernel, dim3(nrt, p.a.Hkv, (units + per_block - 1) / per_block), dim3(kMergeThreads), 0, st, p, ctas);
    };
    return nrt * p.a.Hkv * 12 <= ctas ? merge(prefix_tc_merge_kernel<D, 4>, kMergeThreads / 4) : merge(prefix_tc_merge_kernel<D, 1>, kMergeThreads);
}

// Positions of a tile.  Operands of two terms fill the shared memory with one tile of 128, but two of 64, so that one is converted
// while the other is used (us, 128 : 64, 8 KV heads, one fp16 node a sequence, over f32 rows: 8 sequences of 300 behind 4096 28 : 25, 32
// of 512 behind 32768 145 : 104, 64 of 4096 357 : 357).  Over 8-bit rows, which convert faster, what a tile takes whatever it
// holds counts more: a tile of 128 of the prefix, whose rows are all live, gains some 0.8 us, one of a single sequence, whose rows are
// mostly others', loses 0.6, and the first tile is ready some 3 us earlier (256 sequences behind 32768 283 : 241, 16 of 5 nodes
// and 500 behind 2048 39 : 34, 64 of 1024 97 : 112, 64 of 4096 302 : 367).
int tile_log2(int format, int dtype, long long prefix_tiles, long long own_tiles) {
    const bool two = format == QW_KV_F32 || (format == QW_KV_INT8_G32 && dtype == QW_DT_F16);
    if (!two) return 7;
    return format == QW_KV_F32 || 3 * own_tiles <= 4 * prefix_tiles + 15 * kTcCtas ? 6 : 7;
}

size_t starts_bytes(int64_t rows) { return (((rows + kTcRows - 1) / kTcRows + 2) * 8 + 255) / 256 * 256; }

}  // namespace

size_t prefix_tc_scratch_bytes(int64_t rows, int head_dim) {
    return starts_bytes(rows) + tree_tc_scratch_bytes((int)std::min<int64_t>(rows, kTcRows), head_dim);
}

cudaError_t launch_prefix_tc(const PrefixArgs &a, const qw_kv_view &prefix, const qw_kv_view &kv, int max_len, int max_prefix,
                             void *scratch, cudaStream_t st, bool chained) {
    Prefix p{};
    const int rows = kv.n_seq * a.n_max * a.G;
    p.a = a;
    p.n_seq = kv.n_seq;
    p.rows_max = slot_rows(rows);
    p.inv_g = a.inv_g;
    p.starts = (long long *)scratch;
    uint8_t *rest = (uint8_t *)scratch + starts_bytes(rows);
    p.status = (int *)rest;
    p.part = (float *)(rest + kTcStatusBytes);
    const long long nrt = (rows + kTcRows - 1) / kTcRows;
    auto tiles = [&](int log2, long long positions) { return (long long)kv.n_kv_heads * ((positions + (1 << log2) - 1) >> log2); };
    p.tile_log2 = tile_log2(kv.format, a.dtype, nrt * tiles(7, max_prefix), kv.n_seq * tiles(7, max_len + a.n_max));
    const long long all = nrt * tiles(p.tile_log2, max_prefix) + kv.n_seq * tiles(p.tile_log2, max_len + a.n_max);
    const int ctas = (int)std::min<long long>(kTcCtas, all);
    return kv.head_dim == 128 ? launch_prefix_dim<128>(p, prefix, kv, ctas, st, chained)
                              : launch_prefix_dim<64>(p, prefix, kv, ctas, st, chained);
}

}  // namespace qw
