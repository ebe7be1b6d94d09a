// tree_attn.cu - attention of the nodes of drafted-token trees over their sequences' caches.
//
// Sequence b holds len[b] cached positions and, behind them, the rows of count[b] drafted
// nodes.  Node i sees every cached position and the drafted rows whose bits are set in
// mask[b][i] (its ancestors and itself).  For query head h of node i, with the KV head
// h / G and the scores in the log2 domain:
//   s_j = scale log2(e) q . k_j            over the positions j that node i sees
//   out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),   m = max_j s_j
// and 0 where node i sees nothing.  One node with its own bit set is the attention of an
// ordinary decode step.
//
// The positions of a sequence are split over CTAs, each with its own running maximum, sum
// and f32 accumulator (an online softmax), and the splits are merged in order by a second
// kernel, so the result does not depend on timing.
#include <algorithm>
#include <cmath>

#include "tc.cuh"
#include "tree_attn.h"

namespace qw {
namespace {

constexpr int kTile = 64;       // positions per tile
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Where row r of a KV head's queries lies in out.
__device__ __forceinline__ int64_t out_row(const TreeArgs &a, int b, int h, int r) {
    return b * a.oseq + (int64_t)(r / a.G) * a.onode + (int64_t)(h * a.G + r % a.G) * a.ohead;
}

// The split's positions: equal shares of whole tiles.
__device__ __forceinline__ void split_range(int total, int S, int s, int &p0, int &p1) {
    const int tiles = (total + kTile - 1) / kTile;
    const int per = tiles / S, more = tiles % S;
    p0 = min(total, (s * per + min(s, more)) * kTile);
    p1 = min(total, ((s + 1) * per + min(s + 1, more)) * kTile);
}

// CUDA-core form: f32 arithmetic throughout, for f32 queries over every kind of cache and for small calls.  A CTA takes
// RT query rows (row r = node r / G, head r % G of the KV head's group) and one split of the
// positions.  Per tile of 64 positions: K and V rows as they lie in the cache into registers (the next
// tile's while this one is worked on; the first tile's before anything else, as the latency of
// the first loads is most of a short call), widened to f32 in shared memory; scores with
// one position per thread and the query rows broadcast; the online softmax with one warp per
// row; P V with four dims per lane and up to four rows per warp, the other warps taking other rows or
// other positions, so that a V row is read from shared memory once per four rows (eight rows per
// warp read less but left one CTA per SM: 800 us for 64 nodes over 32768 positions instead of 670).  With few rows it is bound by the latency of that chain or by the
// cache's bytes, with many by shared memory: 512 flops per row, position and KV head, in pairs
// (FFMA2), whose operands keep its reads at 87% of their rate; tiles of up to 32 rows share them.
// One token of 8 sequences over f32 caches of up to 512: 9 us (floor 3); 8 nodes over 32768 f32
// positions: 123 us (40); 64 nodes over 32768 8-bit positions: 680 us (11).
template <typename KV, int D, int RT>
__global__ void __launch_bounds__(kThreads, 2) tree_kernel(const TreeArgs a) {
    constexpr int KS = D + 4;                       // padded K row: quarter warps read 8 banks groups
    constexpr int LPR = D / 4;                      // lanes per V row
    constexpr int KPW = 32 / LPR;                   // positions a warp takes at once in P V
    constexpr int RW = RT < 4 ? RT : 4;             // rows per warp in P V
    constexpr int KW = kWarps / (RT / RW);          // warps that share them, each with its positions
    constexpr int RS = RT < 4 ? 1 : RT / 4;         // rows per thread in the scores
    constexpr int E = 16 / sizeof(KV), LPT = kTile * (D / E) / kThreads;  // elements per load; loads per thread and plane
    extern __shared__ __align__(16) float smf[];
    float *sk = smf, *sv = sk + kTile * KS, *sq = sv + kTile * D, *sp = sq + RT * D;
    float *red = smf;                               // at the end, over K and V: [RT][KW * KPW parts][D]
    static_assert(RT * KW * KPW * D <= kTile * (KS + D), "the parts fit over K and V");
    __shared__ float salpha[RT], sm[RT], sl[RT];
    __shared__ unsigned long long smask[RT];
    tc::chain_wait();
    tc::chain_release();
    const int b = blockIdx.z, h = blockIdx.y / a.row_tiles, rt = blockIdx.y % a.row_tiles, s = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int len, n;
    const bool fits = lengths(a, b, len, n);
    const int r0 = rt * RT, rows = n * a.G;
    if (!fits) {  // without a merge kernel behind it this one fills the rows
        for (int i = tid; a.S == 1 && i < RT * D; i += kThreads)
            if (r0 + i / D < a.n_max * a.G) store_out(a, out_row(a, b, h, r0 + i / D) + i % D, nanf(""));
        return;
    }
    if (r0 >= rows) return;
    const int total = len + n;
    int p0, p1;
    split_range(total, a.S, s, p0, p1);
    const KV *kb = reinterpret_cast<const KV *>(a.k) + b * a.seq + h * a.head;
    const KV *vb = reinterpret_cast<const KV *>(a.v) + b * a.seq + h * a.head;
    uint4 raw[2][LPT];
    __half scale[2][sizeof(KV) == 1 ? LPT : 1];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int plane = 0; plane < 2; ++plane)
#pragma unroll
            for (int i = 0; i < LPT; ++i) {
                const int x = tid + kThreads * i, c = x % (D / E), pos = t0 + x / (D / E);
                raw[plane][i] = make_uint4(0u, 0u, 0u, 0u);
                if constexpr (sizeof(KV) == 1) scale[plane][i] = __half(0);
                if (pos >= p1) continue;
                raw[plane][i] = *reinterpret_cast<const uint4 *>((plane ? vb : kb) + (int64_t)pos * a.pos + E * c);
                if constexpr (sizeof(KV) == 1)
                    scale[plane][i] = ((plane ? a.vs : a.ks) + b * a.sseq + h * a.shead + (int64_t)pos * a.spos)[E * c / kQGroup];
            }
    };
    fetch(p0);
    for (int i = tid; i < RT * D; i += kThreads) {
        const int r = r0 + i / D;
        sq[i] = r < rows ? load_q(a, b * a.qseq + (int64_t)(r / a.G) * a.qnode +
                                         (int64_t)(h * a.G + r % a.G) * a.qhead + i % D) * a.scale_log2
                         : 0.f;
    }
    if (tid < RT) {
        sm[tid] = -INFINITY;
        sl[tid] = 0.f;
        smask[tid] = r0 + tid < rows ? a.mask[(int64_t)b * a.n_max + (r0 + tid) / a.G] : 0ull;
    }
    float2 acc[RW][2];
#pragma unroll
    for (int i = 0; i < RW; ++i) acc[i][0] = acc[i][1] = make_float2(0.f, 0.f);
    for (int t0 = p0; t0 < p1; t0 += kTile) {
        __syncthreads();
#pragma unroll
        for (int plane = 0; plane < 2; ++plane)
#pragma unroll
            for (int i = 0; i < LPT; ++i) {
                const int x = tid + kThreads * i, c = x % (D / E), j = x / (D / E);
                float *dst = plane ? sv + j * D + E * c : sk + j * KS + E * c;
                const KV *e = reinterpret_cast<const KV *>(&raw[plane][i]);
#pragma unroll
                for (int k = 0; k < E; k += 4) {
                    float4 f;
                    if constexpr (sizeof(KV) == 1) {
                        const float sc = __half2float(scale[plane][i]);
                        f = make_float4((float)e[k] * sc, (float)e[k + 1] * sc, (float)e[k + 2] * sc, (float)e[k + 3] * sc);
                    } else {
                        f = make_float4(elem_to_f(e[k]), elem_to_f(e[k + 1]), elem_to_f(e[k + 2]), elem_to_f(e[k + 3]));
                    }
                    *reinterpret_cast<float4 *>(dst + k) = f;
                }
            }
        if (t0 + kTile < p1) fetch(t0 + kTile);
        __syncthreads();
        // scores: thread = (position tid % 64, rows tid / 64 + 4 i)
        {
            const int j = tid & 63, rg = tid >> 6;
            float2 d[RS];
#pragma unroll
            for (int i = 0; i < RS; ++i) d[i] = make_float2(0.f, 0.f);
            if (RT >= 4 || rg < RT) {
#pragma unroll 4
                for (int c = 0; c < D; c += 4) {
                    const float4 k = *reinterpret_cast<const float4 *>(sk + j * KS + c);
#pragma unroll
                    for (int i = 0; i < RS; ++i) {
                        const float4 q = *reinterpret_cast<const float4 *>(sq + (rg + 4 * i) * D + c);
                        d[i] = __ffma2_rn(make_float2(q.x, q.y), make_float2(k.x, k.y), d[i]);
                        d[i] = __ffma2_rn(make_float2(q.z, q.w), make_float2(k.z, k.w), d[i]);
                    }
                }
                const int p = t0 + j;
#pragma unroll
                for (int i = 0; i < RS; ++i) {
                    const int r = rg + 4 * i;
                    const bool sees = p < len || (p < total && ((smask[r] >> (p - len)) & 1ull));
                    sp[r * kTile + j] = p < p1 && sees ? d[i].x + d[i].y : -INFINITY;
                }
            }
        }
        __syncthreads();
        // online softmax: one warp per row
        for (int r = warp; r < RT; r += kWarps) {
            const float x0 = sp[r * kTile + lane], x1 = sp[r * kTile + 32 + lane];
            float m = fmaxf(x0, x1);
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float old = sm[r], mn = fmaxf(old, m);
            // a row that has seen nothing yet keeps m = -inf: every weight 0
            const float e0 = x0 == -INFINITY ? 0.f : exp2f(x0 - mn), e1 = x1 == -INFINITY ? 0.f : exp2f(x1 - mn);
            float l = e0 + e1;
#pragma unroll
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            sp[r * kTile + lane] = e0;
            sp[r * kTile + 32 + lane] = e1;
            if (lane == 0) {
                const float al = old == -INFINITY ? 0.f : exp2f(old - mn);
                salpha[r] = al;
                sl[r] = sl[r] * al + l;
                sm[r] = mn;
            }
        }
        __syncthreads();
        // P V: warp -> rows; a position that a row does not see adds nothing, whatever its V holds
        {
            const int jl = lane / LPR, c = 4 * (lane % LPR);
            const int row0 = warp / KW * RW, jw = warp % KW;
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const float al = salpha[row0 + i];
#pragma unroll
                for (int e = 0; e < 2; ++e) acc[i][e] = __fmul2_rn(acc[i][e], make_float2(al, al));
            }
            const bool tail = t0 + kTile > len;
            // four positions' weights per read: they are most of this loop's shared-memory traffic
            constexpr int STEP = KW * KPW;
#pragma unroll 2
            for (int j0 = 4 * (jw * KPW + jl); j0 < kTile; j0 += 4 * STEP) {
                float4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const float4 *>(sv + (j0 + k) * D + c);
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    const float4 w = *reinterpret_cast<const float4 *>(sp + (row0 + i) * kTile + j0);
                    const float p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (tail && p[k] == 0.f) continue;
                        acc[i][0] = __ffma2_rn(make_float2(p[k], p[k]), make_float2(v[k].x, v[k].y), acc[i][0]);
                        acc[i][1] = __ffma2_rn(make_float2(p[k], p[k]), make_float2(v[k].z, v[k].w), acc[i][1]);
                    }
                }
            }
        }
    }
    // the parts of a row (KW warps x KPW lane groups) added in order
    {
        constexpr int PARTS = KW * KPW;
        const int jl = lane / LPR, c = 4 * (lane % LPR);
        const int row0 = warp / KW * RW, jw = warp % KW;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RW; ++i)
            *reinterpret_cast<float4 *>(red + ((row0 + i) * PARTS + jw * KPW + jl) * D + c) =
                make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
        __syncthreads();
        for (int i = tid; i < RT * D; i += kThreads) {
            const int rl = i / D, d = i % D, r = r0 + rl;
            if (r >= rows) continue;
            float o = 0.f;
#pragma unroll
            for (int k = 0; k < PARTS; ++k) o += red[(rl * PARTS + k) * D + d];
            if (a.S == 1) {  // the only split: nothing to merge
                store_out(a, out_row(a, b, h, r) + d, sl[rl] == 0.f ? 0.f : o / sl[rl]);
                continue;
            }
            float *dst = a.part + ((((int64_t)b * a.Hkv + h) * a.n_max * a.G + r) * a.S + s) * (D + 2);
            dst[d] = o;
            if (d == 0) {
                dst[D] = sm[rl];
                dst[D + 1] = sl[rl];
            }
        }
    }
}

// One query row per CTA: out = sum_s acc_s 2^(m_s - M) / sum_s l_s 2^(m_s - M), in order.  The partials
// of kBatch splits are loaded at once: the kernel is their latency.
constexpr int kBatch = 8;

template <int D>
__global__ void __launch_bounds__(D) tree_merge_kernel(const TreeArgs a) {
    const int r = blockIdx.x, h = blockIdx.y, b = blockIdx.z, d = threadIdx.x;
    int len, n;
    const bool fits = lengths(a, b, len, n);
    const int64_t at = out_row(a, b, h, r) + d;
    const float *src = a.part + (((int64_t)b * a.Hkv + h) * a.n_max * a.G + r) * a.S * (D + 2);
    tc::chain_wait();
    if (fits && r >= n * a.G) return;
    if (!fits) {
        store_out(a, at, nanf(""));
        return;
    }
    float mx = -INFINITY, num = 0.f, den = 0.f;
    for (int s = 0; s < a.S; s += kBatch) {
        float m[kBatch], l[kBatch], v[kBatch], top = mx;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float *ps = src + (int64_t)(s + i) * (D + 2);
            const bool is = s + i < a.S;
            m[i] = is ? ps[D] : -INFINITY;
            l[i] = is ? ps[D + 1] : 0.f;
            v[i] = is ? ps[d] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) top = fmaxf(top, m[i]);
        const float old = mx == -INFINITY ? 0.f : exp2f(mx - top);
        mx = top;
        num *= old;
        den *= old;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (m[i] == -INFINITY && l[i] == 0.f) continue;  // the split showed the row nothing
            const float w = exp2f(m[i] - mx);
            num += v[i] * w;
            den += l[i] * w;
        }
    }
    store_out(a, at, den == 0.f ? 0.f : num / den);
}

int rows_per_tile(int rows) { return rows <= 2 ? 2 : rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

// Splits: up to four CTAs for every SM (three of them fit at 16 rows of 128 dims, and in a ragged batch
// some have nothing to do), none shorter than a tile.
int splits(int n_seq, int Hkv, int row_tiles, int rt, int total) {
    const int tiles = (total + kTile - 1) / kTile;
    const int64_t base = (int64_t)n_seq * Hkv * row_tiles;
    const int64_t want = (4 * 152 + base - 1) / base;
    if (tiles <= 2 && rt <= 4) return 1;  // a second tile costs less than the merge's launch
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, tiles));
}

// Whether a call with 16-bit queries is better off on the CUDA cores: they need no set-up of barriers,
// tensor memory and conversions, but time grows with every tile of 64 positions.  Measured, us,
// CUDA cores against tensor cores, 8 KV heads of two query heads of 128 dims.  Two rows (one node), fp16
// queries: one sequence over 64 8-bit positions 7 : 11, 8 sequences over 512 (576 tiles) 14 : 23, over 1024 (1088)
// 24 : 26; bf16 beside bf16 6 : 9, 13 : 17 and 21 : 18, but one sequence over 4096 (520) 17 : 14.  Eight rows:
// one sequence over 1024 8-bit positions (136) 10 : 14, over 4096 (520) 25 : 21; bf16 10 : 12 and 23 : 14.  Sixteen
// rows, 8-bit: over 512 (72) 12 : 14, over 2048 (264) 18 : 16; bf16 11 : 12 and 17 : 14.  f32 rows cost the
// conversion most and the CUDA cores nothing: up to four rows always (8 sequences of one node over 4096:
// 64 : 91), up to eight until 608 tiles (8 sequences of four nodes over 512, 576 tiles: 20 : 25; over 1024: 36 : 33).
// bf16 queries over f32 rows measure as fp16 ones.
bool small_call(const qw_kv_view &kv, const qw_tree_attention_args &t) {
    const int64_t tiles = (int64_t)kv.n_seq * kv.n_kv_heads * ((t.max_len + t.n_max + kTile - 1) / kTile);
    const int rows = t.n_max * (t.n_heads / kv.n_kv_heads);
    const bool direct = t.dtype == QW_DT_BF16 && kv.format == QW_KV_BF16;
    const bool f32 = kv.format == QW_KV_F32;
    if (rows <= 4) return f32 || tiles <= 4 * 152;
    if (rows <= 8) return tiles <= (direct ? 1 : f32 ? 4 : 2) * 152;
    return rows <= 16 && !direct && tiles <= 152;
}

template <typename KV, int D, int RT>
cudaError_t launch_tile(const TreeArgs &a, int n_seq, cudaStream_t st, bool chained) {
    constexpr int smem = (kTile * (D + 4) + kTile * D + RT * D + RT * kTile) * 4;
    cudaError_t e = allow_smem<tree_kernel<KV, D, RT>>(smem);
    if (e != cudaSuccess) return e;
    return launch_k(chained, tree_kernel<KV, D, RT>, dim3(a.S, a.Hkv * a.row_tiles, n_seq), dim3(kThreads), smem, st, a);
}

template <typename KV, int D>
cudaError_t launch_rt(const TreeArgs &a, int n_seq, int rt, cudaStream_t st, bool ch) {
    cudaError_t e = rt == 2   ? launch_tile<KV, D, 2>(a, n_seq, st, ch)
                    : rt == 4 ? launch_tile<KV, D, 4>(a, n_seq, st, ch)
                    : rt == 8 ? launch_tile<KV, D, 8>(a, n_seq, st, ch)
                    : rt == 16 ? launch_tile<KV, D, 16>(a, n_seq, st, ch)
                               : launch_tile<KV, D, 32>(a, n_seq, st, ch);
    if (e != cudaSuccess || a.S == 1) return e;
    return launch_k(true, tree_merge_kernel<D>, dim3(a.n_max * a.G, a.Hkv, n_seq), dim3(D), 0, st, a);
}

}  // namespace

size_t tree_attn_scratch_bytes(int n_seq, int n_kv_heads, int n_max, int n_heads, int head_dim, int max_len) {
    const int G = n_heads / n_kv_heads, rows = n_max * G, rt = rows_per_tile(rows);
    const int S = splits(n_seq, n_kv_heads, (rows + rt - 1) / rt, rt, max_len + n_max);
    const size_t cores = ((size_t)n_seq * n_kv_heads * rows * S * (head_dim + 2) * 4 + 255) / 256 * 256;
    return std::max(cores, tree_tc_scratch_bytes(rows, head_dim));
}

cudaError_t launch_tree_attn(const qw_kv_view &kv, const qw_tree_attention_args &t, void *scratch, cudaStream_t st,
                             bool chained) {
    if (kv.n_seq == 0 || t.n_max == 0) return cudaSuccess;
    TreeArgs a{};
    a.k = (const uint8_t *)kv.k;
    a.v = (const uint8_t *)kv.v;
    a.ks = (const __half *)kv.k_scale;
    a.vs = (const __half *)kv.v_scale;
    a.seq = kv.seq_stride, a.head = kv.head_stride, a.pos = kv.pos_stride;
    a.sseq = kv.scale_seq_stride, a.shead = kv.scale_head_stride, a.spos = kv.scale_pos_stride;
    a.q = t.q;
    a.out = t.out;
    a.dtype = t.dtype;
    a.qseq = t.q_seq_stride, a.qnode = t.q_node_stride, a.qhead = t.q_head_stride;
    a.oseq = t.out_seq_stride, a.onode = t.out_node_stride, a.ohead = t.out_head_stride;
    a.mask = (const unsigned long long *)t.mask;
    a.len = t.len;
    a.count = t.count;
    a.n_max = t.n_max;
    a.max_ctx = kv.max_ctx;
    a.Hkv = kv.n_kv_heads;
    a.G = t.n_heads / kv.n_kv_heads;
    a.scale_log2 = t.scale * kOpsLog2e;
    a.part = (float *)scratch;
    if (t.dtype != QW_DT_F32 && !small_call(kv, t)) return launch_tree_tc(a, kv, t.max_len, scratch, st, chained);
    const int rows = t.n_max * a.G, rt = rows_per_tile(rows);
    a.row_tiles = (rows + rt - 1) / rt;
    a.S = splits(kv.n_seq, kv.n_kv_heads, a.row_tiles, rt, t.max_len + t.n_max);
    const int D = kv.head_dim;
    if (kv.format == QW_KV_F32)
        return D == 128 ? launch_rt<float, 128>(a, kv.n_seq, rt, st, chained) : launch_rt<float, 64>(a, kv.n_seq, rt, st, chained);
    if (kv.format == QW_KV_BF16)
        return D == 128 ? launch_rt<__nv_bfloat16, 128>(a, kv.n_seq, rt, st, chained)
                        : launch_rt<__nv_bfloat16, 64>(a, kv.n_seq, rt, st, chained);
    return D == 128 ? launch_rt<int8_t, 128>(a, kv.n_seq, rt, st, chained) : launch_rt<int8_t, 64>(a, kv.n_seq, rt, st, chained);
}

}  // namespace qw
