// kvcache.cu - rows of a K/V cache written (and quantised on the way) and read back.
//
// A cache of n_seq sequences holds, per KV head and position, one K and one V row of
// head_dim elements: f32, bf16, or int8 codes with one fp16 scale per 32 elements (the
// Q8_0 block of "Scalar-Native Qwen3 Reference Runtime As The Numerical Authority",
// section 3, codes and scales in separate planes).  Both kernels are copies with a
// conversion: bound by the bytes of the source rows and of the written rows.  A thread
// moves eight elements of a row, so a warp's accesses are contiguous runs of 256 bytes or
// more, and a 32-element group is four adjacent lanes: its maximum takes two shuffles.
#include "qw_ops.h"

namespace qw {
namespace {

constexpr int kRowThreads = 256;

struct RowArgs {
    uint8_t *k, *v;           // the cache
    __half *ks, *vs;
    int64_t seq, head, pos;   // its strides (elements), and the scales'
    int64_t sseq, shead, spos;
    uint8_t *rk, *rv;         // the rows
    int64_t rseq, rhead, rrow;
    const int32_t *start, *count;
    int heads, n_max, max_ctx;
};

// T: the rows' element type; KV: float, __nv_bfloat16, or int8_t for the 8-bit format.
// blockIdx.y = sequence, blockIdx.z = K or V; the sequence's heads * n_max rows are cut into
// blocks of U passes of kRowThreads / (D / 8) rows.  A thread issues the loads of its U rows
// before it uses any.
template <typename T, typename KV, int D, int U, bool READ>
__global__ void __launch_bounds__(kRowThreads) kv_rows_kernel(const RowArgs a) {
    constexpr int TPR = D / 8;  // threads per row
    constexpr int RPB = kRowThreads / TPR;
    const int c = threadIdx.x % TPR, b = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const int s0 = a.start[b], n = a.count ? a.count[b] : a.n_max;
    // a sequence whose rows would leave the cache is not touched
    const bool fits = n >= 0 && n <= a.n_max && s0 >= 0 && s0 <= a.max_ctx - n;
    const uint32_t rows = (uint32_t)a.heads * (uint32_t)a.n_max;
    T *row[U];
    KV *cache[U];
    __half *sc[U];
    bool live[U];
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t x = (blockIdx.x * U + u) * RPB + threadIdx.x / TPR;
        const uint32_t h = x / (uint32_t)a.n_max, i = x - h * (uint32_t)a.n_max;
        live[u] = fits && x < rows && (int)i < n;
        const int64_t at = live[u] ? (int64_t)s0 + i : 0;
        row[u] = reinterpret_cast<T *>(is_v ? a.rv : a.rk) + b * a.rseq + h * a.rhead + i * a.rrow + 8 * c;
        cache[u] = reinterpret_cast<KV *>(is_v ? a.v : a.k) + b * a.seq + h * a.head + at * a.pos + 8 * c;
        if constexpr (sizeof(KV) == 1) sc[u] = (is_v ? a.vs : a.ks) + b * a.sseq + h * a.shead + at * a.spos + c / 4;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[u][k] = 0.f;
        if (!live[u]) continue;
        if constexpr (!READ) load8(row[u], v[u]);
        else if constexpr (sizeof(KV) == 1) load8_q8(cache[u], __half2float(*sc[u]), v[u]);
        else load8(cache[u], v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if constexpr (READ) {
            if (live[u]) store8(row[u], v[u]);
        } else if constexpr (sizeof(KV) == 1) {
            __half scale;
            const uint2 q = quant8(v[u], scale);  // whole warp: a group's lanes share live
            if (live[u]) {
                *reinterpret_cast<uint2 *>(cache[u]) = q;
                if (c % 4 == 0) *sc[u] = scale;
            }
        } else if (live[u]) {
            store8(cache[u], v[u]);
        }
    }
}

template <typename T, typename KV, int D, int U, bool READ>
cudaError_t launch_u(const RowArgs &a, int n_seq, cudaStream_t st) {
    constexpr int per = U * kRowThreads / (D / 8);
    const long long rows = (long long)a.heads * a.n_max;
    return launch_k(false, kv_rows_kernel<T, KV, D, U, READ>, dim3((unsigned)((rows + per - 1) / per), n_seq, 2),
                    dim3(kRowThreads), 0, st, a);
}

// Four rows per thread where that still leaves blocks for every SM (32768 rows of 8 heads read back
// as bf16: see the file's head); one row for the few rows of a decode step.
template <typename T, typename KV, bool READ>
cudaError_t launch_rows(const RowArgs &a, int n_seq, int D, cudaStream_t st) {
    const long long rows = (long long)a.heads * a.n_max * n_seq;
    const bool many = rows * 2 * (D / 8) >= 4LL * 2 * 152 * kRowThreads;
    if (D == 128)
        return many ? launch_u<T, KV, 128, 4, READ>(a, n_seq, st) : launch_u<T, KV, 128, 1, READ>(a, n_seq, st);
    return many ? launch_u<T, KV, 64, 4, READ>(a, n_seq, st) : launch_u<T, KV, 64, 1, READ>(a, n_seq, st);
}

template <typename T, bool READ>
cudaError_t launch_rows_kv(const RowArgs &a, const qw_kv_view &kv, cudaStream_t st) {
    const int n = kv.n_seq, D = kv.head_dim;
    return kv.format == QW_KV_F32    ? launch_rows<T, float, READ>(a, n, D, st)
           : kv.format == QW_KV_BF16 ? launch_rows<T, __nv_bfloat16, READ>(a, n, D, st)
                                     : launch_rows<T, int8_t, READ>(a, n, D, st);
}

template <bool READ>
cudaError_t launch_any(const qw_kv_view &kv, const qw_kv_rows &r, const int32_t *start, const int32_t *count,
                       cudaStream_t st) {
    RowArgs a{};
    a.k = (uint8_t *)kv.k;
    a.v = (uint8_t *)kv.v;
    a.ks = (__half *)kv.k_scale;
    a.vs = (__half *)kv.v_scale;
    a.seq = kv.seq_stride, a.head = kv.head_stride, a.pos = kv.pos_stride;
    a.sseq = kv.scale_seq_stride, a.shead = kv.scale_head_stride, a.spos = kv.scale_pos_stride;
    a.rk = (uint8_t *)r.k;
    a.rv = (uint8_t *)r.v;
    a.rseq = r.seq_stride, a.rhead = r.head_stride, a.rrow = r.row_stride;
    a.start = start;
    a.count = count;
    a.heads = kv.n_kv_heads;
    a.n_max = r.n_max;
    a.max_ctx = kv.max_ctx;
    if (r.n_max == 0) return cudaSuccess;
    return r.dtype == QW_DT_F32   ? launch_rows_kv<float, READ>(a, kv, st)
           : r.dtype == QW_DT_F16 ? launch_rows_kv<__half, READ>(a, kv, st)
                                  : launch_rows_kv<__nv_bfloat16, READ>(a, kv, st);
}

}  // namespace

cudaError_t launch_kv_append(const qw_kv_view &kv, const qw_kv_rows &src, const int32_t *start, const int32_t *count,
                             cudaStream_t st) {
    return launch_any<false>(kv, src, start, count, st);
}

cudaError_t launch_kv_read(const qw_kv_view &kv, const qw_kv_rows &dst, const int32_t *start, const int32_t *count,
                           cudaStream_t st) {
    return launch_any<true>(kv, dst, start, count, st);
}

}  // namespace qw
