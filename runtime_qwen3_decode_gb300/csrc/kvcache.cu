// kvcache.cu - rows of a K/V cache written (and quantised on the way) and read back.
//
// A cache of n_seq sequences holds, per KV head and position, one K and one V row of
// head_dim elements: f32, bf16, or int8 codes with one fp16 scale per 32 elements (the
// Q8_0 block of "Scalar-Native Qwen3 Reference Runtime As The Numerical Authority",
// section 3, codes and scales in separate planes).  Both kernels are copies with a
// conversion: bound by the bytes of the source rows and of the written rows.  A lane moves 16
// bytes of a row, so every access of a warp is one contiguous run on both sides, and a
// 32-element group is 4 (16-bit rows) or 8 (f32) adjacent lanes: its maximum takes two or
// three shuffles.
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

// E consecutive elements as they lie in memory.  Rows begin on 16-byte boundaries and no more, so eight
// f32 elements (32 bytes) are two accesses of 16: a type aligned to 32 would let the compiler make
// one access of 32 of them, which faults on a row that begins between two such boundaries.
template <typename T, int E>
struct alignas(sizeof(T) * E < 16 ? sizeof(T) * E : 16) Pack {
    T e[E];
};
static_assert(alignof(Pack<float, 8>) == 16, "rows are aligned to 16 bytes");

// The 8-bit form of a 32-element group held by 32 / E adjacent lanes, E elements each: d = amax /
// 127 in f32, code = a / d rounded half away from zero (the Q8_0 block's quantiser), scale =
// fp16(d).  A NaN or an infinity anywhere in the group makes the scale NaN, so that the group
// reads back as NaN instead of as some finite value.  Whole warps call it.
template <int E>
__device__ __forceinline__ Pack<int8_t, E> quantise(const float (&v)[E], __half &scale) {
    float amax = 0.f, probe = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        amax = fmaxf(amax, fabsf(v[i]));
        probe = fmaf(v[i], 0.f, probe);  // 0 unless a value is not finite, then NaN
    }
#pragma unroll
    for (int o = 1; o < kQGroup / E; o <<= 1) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        probe += __shfl_xor_sync(0xffffffffu, probe, o);
    }
    const float d = amax / 127.0f;
    Pack<int8_t, E> c;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float r = d > 0.f ? fminf(fmaxf(roundf(v[i] / d), -127.f), 127.f) : 0.f;
        c.e[i] = (int8_t)(int)r;
    }
    scale = __float2half_rn(d + probe);
    return c;
}

// T: the rows' element type; KV: float, __nv_bfloat16, or int8_t for the 8-bit format.
// blockIdx.x = (head, block of U * kRowThreads / (D / E) rows), blockIdx.y = sequence, blockIdx.z = K
// or V: one division per block (a division per row, in 64 bits, was most of the time).  A lane's U
// rows are all loaded before one is written; the rest of the latency is left to the many small
// blocks of an SM.  32768 rows of 8 heads of 128 read back as bf16: 40 us, 5.2 TB/s, 77% of the
// measured copy rate (blocks that looped over rows with the next ones prefetched needed more
// registers and took 73); 2048 f32 rows of 8 heads appended: 11 us under the profiler, one wave.
template <typename T, typename KV, int D, int U, bool READ>
__global__ void __launch_bounds__(kRowThreads) kv_rows_kernel(const RowArgs a, int blocks) {
    constexpr int E = 16 / sizeof(T);
    constexpr int TPR = D / E;  // lanes per row
    constexpr int RPB = kRowThreads / TPR;
    using Src = typename std::conditional<READ, KV, T>::type;
    const int c = threadIdx.x % TPR, b = blockIdx.y, h = blockIdx.x / blocks;
    const int i0 = (blockIdx.x - h * blocks) * RPB * U + threadIdx.x / TPR;
    const bool is_v = blockIdx.z != 0;
    const int s0 = a.start[b], n = a.count ? a.count[b] : a.n_max;
    // a sequence whose rows would leave the cache is not touched
    if (n <= 0 || n > a.n_max || s0 < 0 || s0 > a.max_ctx - n) return;
    T *row = reinterpret_cast<T *>(is_v ? a.rv : a.rk) + b * a.rseq + h * a.rhead + i0 * a.rrow + E * c;
    KV *cache = reinterpret_cast<KV *>(is_v ? a.v : a.k) + b * a.seq + h * a.head + ((int64_t)s0 + i0) * a.pos + E * c;
    __half *sc = (is_v ? a.vs : a.ks) + b * a.sseq + h * a.shead + ((int64_t)s0 + i0) * a.spos + E * c / kQGroup;
    Pack<Src, E> x[U];
    __half scale[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (i0 + u * RPB >= n) continue;
        if constexpr (READ) x[u] = *reinterpret_cast<const Pack<Src, E> *>(cache + u * RPB * a.pos);
        else x[u] = *reinterpret_cast<const Pack<Src, E> *>(row + u * RPB * a.rrow);
        if constexpr (READ && sizeof(KV) == 1) scale[u] = sc[u * RPB * a.spos];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool live = i0 + u * RPB < n;
        float v[E];
#pragma unroll
        for (int k = 0; k < E; ++k) {
            if constexpr (sizeof(Src) == 1) v[k] = live ? (float)x[u].e[k] * __half2float(scale[u]) : 0.f;
            else v[k] = live ? elem_to_f(x[u].e[k]) : 0.f;
        }
        if constexpr (READ) {
            Pack<T, E> o;
#pragma unroll
            for (int k = 0; k < E; ++k) o.e[k] = elem_from_f<T>(v[k]);
            if (live) *reinterpret_cast<Pack<T, E> *>(row + u * RPB * a.rrow) = o;
        } else if constexpr (sizeof(KV) == 1) {
            __half s;
            const Pack<int8_t, E> q = quantise<E>(v, s);
            if (live) {
                *reinterpret_cast<Pack<int8_t, E> *>(cache + u * RPB * a.pos) = q;
                if (c % (kQGroup / E) == 0) sc[u * RPB * a.spos] = s;
            }
        } else {
            Pack<KV, E> o;
#pragma unroll
            for (int k = 0; k < E; ++k) o.e[k] = elem_from_f<KV>(v[k]);
            if (live) *reinterpret_cast<Pack<KV, E> *>(cache + u * RPB * a.pos) = o;
        }
    }
}

template <typename T, typename KV, int D, int U, bool READ>
cudaError_t launch_u(const RowArgs &a, int n_seq, cudaStream_t st) {
    constexpr int per = U * kRowThreads / (D * (int)sizeof(T) / 16);  // rows per block
    const int blocks = (a.n_max + per - 1) / per;
    return launch_k(false, kv_rows_kernel<T, KV, D, U, READ>, dim3((unsigned)(blocks * a.heads), n_seq, 2),
                    dim3(kRowThreads), 0, st, a, blocks);
}

// Four rows per lane where they fill a block; one for the few rows of a decode step or a tree.
template <typename T, typename KV, bool READ>
cudaError_t launch_rows(const RowArgs &a, int n_seq, int D, cudaStream_t st) {
    const bool many = a.n_max >= 4 * kRowThreads / (D * (int)sizeof(T) / 16);
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
