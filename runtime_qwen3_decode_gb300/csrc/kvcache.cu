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
    long long rows;           // n_seq * heads * n_max
};

// T: the rows' element type; KV: float, __nv_bfloat16, or int8_t for the 8-bit format.
// A thread's row is one of the 2 * rows (K rows, then V rows); D / 8 threads share it.
template <typename T, typename KV, int D, bool READ>
__global__ void __launch_bounds__(kRowThreads) kv_rows_kernel(const RowArgs a) {
    constexpr int TPR = D / 8;  // threads per row
    constexpr int RPB = kRowThreads / TPR;
    const int c = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * RPB;
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < 2 * a.rows; r0 += step) {
        long long r = r0 + threadIdx.x / TPR;
        bool live = r < 2 * a.rows;
        const bool is_v = r >= a.rows;
        if (is_v) r -= a.rows;
        if (!live) r = 0;
        const int i = (int)(r % a.n_max);
        const long long bh = r / a.n_max;
        const int h = (int)(bh % a.heads), b = (int)(bh / a.heads);
        const int s0 = a.start[b], n = a.count ? a.count[b] : a.n_max;
        // a sequence whose rows would leave the cache is not touched
        live = live && i < n && n <= a.n_max && s0 >= 0 && s0 <= a.max_ctx - n;
        const int64_t at = b * a.seq + h * a.head + (int64_t)(live ? s0 + i : 0) * a.pos + 8 * c;
        T *row = reinterpret_cast<T *>(is_v ? a.rv : a.rk) + b * a.rseq + h * a.rhead + i * a.rrow + 8 * c;
        KV *cache = reinterpret_cast<KV *>(is_v ? a.v : a.k) + at;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if constexpr (sizeof(KV) == 1) {
            __half *sc = (is_v ? a.vs : a.ks) + b * a.sseq + h * a.shead + (int64_t)(live ? s0 + i : 0) * a.spos + c / 4;
            if constexpr (READ) {
                if (live) {
                    load8_q8(cache, __half2float(*sc), v);
                    store8(row, v);
                }
            } else {
                if (live) load8(row, v);
                __half scale;
                const uint2 u = quant8(v, scale);  // whole warp: the group's lanes share live
                if (live) {
                    *reinterpret_cast<uint2 *>(cache) = u;
                    if (c % 4 == 0) *sc = scale;
                }
            }
        } else if (live) {
            if constexpr (READ) {
                load8(cache, v);
                store8(row, v);
            } else {
                load8(row, v);
                store8(cache, v);
            }
        }
    }
}

template <typename T, typename KV, bool READ>
cudaError_t launch_rows(const RowArgs &a, int D, cudaStream_t st) {
    const long long per = kRowThreads / (D / 8);
    const long long blocks = (2 * a.rows + per - 1) / per;
    const dim3 grid((unsigned)(blocks < 152 * 8 * 8 ? blocks : 152 * 8 * 8));
    return D == 128 ? launch_k(false, kv_rows_kernel<T, KV, 128, READ>, grid, dim3(kRowThreads), 0, st, a)
                    : launch_k(false, kv_rows_kernel<T, KV, 64, READ>, grid, dim3(kRowThreads), 0, st, a);
}

template <typename T, bool READ>
cudaError_t launch_rows_kv(const RowArgs &a, int format, int D, cudaStream_t st) {
    return format == QW_KV_F32    ? launch_rows<T, float, READ>(a, D, st)
           : format == QW_KV_BF16 ? launch_rows<T, __nv_bfloat16, READ>(a, D, st)
                                  : launch_rows<T, int8_t, READ>(a, D, st);
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
    a.rows = (long long)kv.n_seq * kv.n_kv_heads * r.n_max;
    if (a.rows == 0) return cudaSuccess;
    return r.dtype == QW_DT_F32   ? launch_rows_kv<float, READ>(a, kv.format, kv.head_dim, st)
           : r.dtype == QW_DT_F16 ? launch_rows_kv<__half, READ>(a, kv.format, kv.head_dim, st)
                                  : launch_rows_kv<__nv_bfloat16, READ>(a, kv.format, kv.head_dim, st);
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
