// logits.cu - logits made ready for sampling: penalties for repeated tokens, biases and
// grammar masks, for many rows at once (the sequences of a batch, the nodes of a tree).
//
// For row r and token t, with c = how often r's history range and drafted path name t:
//   x = logits[r][t]
//   c > 0:  x = x > 0 ? x / rep : x * rep;  x -= presence + frequency * c
//   x += the row's biases for t, added in list order
//   the row has a mask and t's bit is clear:  x = -inf
// in f32, rounded once to the output's type.
//
// One pass over the logits; the bound is their bytes, read once and written once.  A CTA
// takes one row's chunk of kTok tokens: each thread issues its loads first, then the CTA
// scans the row's history, path and bias lists (a few KB that every chunk of the row reads
// again from L2) and keeps what falls in the chunk in shared memory, as a dense count and a
// dense bias per token, and then finishes its values.  Counts are whole numbers, so the
// order of their atomics does not matter; a bias named more than once is summed by the
// list's first entry alone, in order, so results do not depend on timing.
#include "qw_ops.h"

namespace qw {
namespace {

constexpr int kVecs = 4;          // vectors of four tokens per thread
constexpr uint32_t kNamed = 1u << 31, kTwice = 1u << 30, kCount = kTwice - 1;

template <typename T>
__device__ __forceinline__ void load4(const T *p, float (&v)[4]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = elem_to_f(e[i]);
    }
}

template <typename T>
__device__ __forceinline__ void store4(T *p, const float (&v)[4]) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        uint2 u;
        T *e = reinterpret_cast<T *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = elem_from_f<T>(v[i]);
        *reinterpret_cast<uint2 *>(p) = u;
    }
}

// [begin, end) of a row's list, kept inside the array; empty without a list.
__device__ __forceinline__ int2 list_range(const int32_t *range, int r, int n) {
    return range ? make_int2(max(range[2 * r], 0), min(range[2 * r + 1], n)) : make_int2(0, 0);
}

// THREADS * 16 tokens per CTA.  VEC: rows start on vector boundaries; SPARSE: there are
// lists to look at.  Whatever does not depend on something else is loaded first: the chain of
// a CTA is lists -> counts -> values, and its length, not the bytes, was the time.
template <typename T, int THREADS, bool VEC, bool SPARSE>
__global__ void __launch_bounds__(THREADS) logits_kernel(const qw_process_logits_args a) {
    constexpr int kTok = THREADS * 4 * kVecs, kAhead = 4;
    extern __shared__ __align__(16) uint32_t sm[];  // [kTok] counts and flags, [kTok] biases of the flagged
    uint32_t *cnt = sm;
    float *add = reinterpret_cast<float *>(sm + kTok);
    const int r = blockIdx.y, base = blockIdx.x * kTok, V = a.vocab, tid = threadIdx.x;
    const T *src = reinterpret_cast<const T *>(a.logits) + (int64_t)r * a.row_stride;
    T *dst = reinterpret_cast<T *>(a.out) + (int64_t)r * a.out_row_stride;
    const int which = a.mask ? (a.mask_index ? a.mask_index[r] : r) : -1;
    int2 hist = make_int2(0, 0), bias = make_int2(0, 0);
    float rep = 1.f, pres = 0.f, freq = 0.f;
    if constexpr (SPARSE) {
        if (a.penalties) {
            rep = a.penalties[3 * r], pres = a.penalties[3 * r + 1], freq = a.penalties[3 * r + 2];
            if (a.history) hist = list_range(a.history_range, r, a.n_history);
        }
        if (a.bias) bias = list_range(a.bias_range, r, a.n_bias);
    }
    float v[kVecs][4];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int t = base + 4 * (tid + THREADS * j);
        if (VEC && t + 4 <= V) {
            load4(src + t, v[j]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // without vectors a warp still reads runs of 32 neighbours
                const int s = VEC ? t + i : base + 4 * THREADS * j + THREADS * i + tid;
                v[j][i] = s < V ? elem_to_f(src[s]) : 0.f;
            }
        }
    }
    if constexpr (SPARSE) {
        uint4 *z = reinterpret_cast<uint4 *>(sm);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) z[tid + THREADS * i] = make_uint4(0u, 0u, 0u, 0u);
    }
    // the mask: a vector of four tokens lies in one word
    const bool none = which >= a.n_masks && a.mask;  // an index past the masks: nothing is allowed
    const uint32_t *mask = which >= 0 && !none ? a.mask + (int64_t)which * ((V + 31) / 32) : nullptr;
    uint32_t word[kVecs];
    if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int t = base + 4 * (tid + THREADS * j);
            word[j] = mask && t < V ? mask[t >> 5] >> (t & 31) : none ? 0u : ~0u;
        }
    }
    if constexpr (SPARSE) {
        // a token outside the vocabulary falls in no chunk, or behind the row's end
        auto count = [&](int32_t id) {
            const uint32_t t = (uint32_t)id - (uint32_t)base;
            if (t < (uint32_t)kTok) atomicAdd(cnt + t, 1u);
        };
        int32_t id0 = -1, own = -1;
        if (bias.x + tid < bias.y) id0 = a.bias_ids[bias.x + tid];
        if (a.penalties && a.path && tid < a.path_len) own = a.path[(int64_t)r * a.path_len + tid];
        int32_t ids[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = hist.x + tid + THREADS * k;
            ids[k] = i < hist.y ? a.history[i] : -1;
        }
        __syncthreads();
        count(own);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) count(ids[k]);
        for (int i = hist.x + tid + THREADS * kAhead; i < hist.y; i += THREADS) count(a.history[i]);
        if (a.penalties && a.path)
            for (int i = tid + THREADS; i < a.path_len; i += THREADS) count(a.path[(int64_t)r * a.path_len + i]);
        if (a.bias) {
            for (int i = bias.x + tid; i < bias.y; i += THREADS) {
                const uint32_t t = (uint32_t)(i == bias.x + tid ? id0 : a.bias_ids[i]) - (uint32_t)base;
                if (t < (uint32_t)kTok && (atomicOr(cnt + t, kNamed) & kNamed)) atomicOr(cnt + t, kTwice);
            }
            __syncthreads();
            for (int i = bias.x + tid; i < bias.y; i += THREADS) {
                const int32_t id = i == bias.x + tid ? id0 : a.bias_ids[i];
                const uint32_t t = (uint32_t)id - (uint32_t)base;
                if (t >= (uint32_t)kTok) continue;
                float sum = a.bias[i];
                if (cnt[t] & kTwice) {
                    bool first = true;
                    for (int k = bias.x; k < i && first; ++k) first = a.bias_ids[k] != id;
                    if (!first) continue;
                    for (int k = i + 1; k < bias.y; ++k)
                        if (a.bias_ids[k] == id) sum += a.bias[k];
                }
                add[t] = sum;
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int t0 = base + 4 * (tid + THREADS * j);
        if (VEC && t0 >= V) break;
        uint4 c4 = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (SPARSE && VEC) c4 = reinterpret_cast<const uint4 *>(cnt)[tid + THREADS * j];
        const uint32_t cw[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = VEC ? t0 + i : base + 4 * THREADS * j + THREADS * i + tid;
            float x = v[j][i];
            if constexpr (SPARSE) {
                const uint32_t c = VEC ? cw[i] : cnt[t - base];
                if (c & kCount) {
                    x = x > 0.f ? x / rep : x * rep;
                    x -= pres + freq * (float)(c & kCount);
                }
                if (c & kNamed) x += add[t - base];
            }
            bool ok;
            if constexpr (VEC) ok = (word[j] >> i) & 1u;
            else ok = !none && (!mask || t >= V || ((mask[t >> 5] >> (t & 31)) & 1u));
            x = ok ? x : -INFINITY;
            v[j][i] = x;
            if (!VEC && t < V) dst[t] = elem_from_f<T>(x);
        }
        if constexpr (VEC) {
            if (t0 + 4 <= V) {
                store4(dst + t0, v[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (t0 + i < V) dst[t0 + i] = elem_from_f<T>(v[j][i]);
            }
        }
    }
}

template <typename T, int THREADS, bool VEC>
cudaError_t launch_t(const qw_process_logits_args &a, cudaStream_t st) {
    constexpr int kTok = THREADS * 4 * kVecs;
    const dim3 grid((a.vocab + kTok - 1) / kTok, a.n_rows);
    if ((a.penalties && (a.history || a.path)) || a.bias) {
        constexpr int smem = 2 * kTok * 4;
        if (smem > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(logits_kernel<T, THREADS, VEC, true>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
        }
        return launch_k(false, logits_kernel<T, THREADS, VEC, true>, grid, dim3(THREADS), smem, st, a);
    }
    return launch_k(false, logits_kernel<T, THREADS, VEC, false>, grid, dim3(THREADS), 0, st, a);
}

template <typename T>
cudaError_t launch_vec(const qw_process_logits_args &a, cudaStream_t st) {
    const size_t unit = 4 * sizeof(T);
    const bool vec = !((uintptr_t)a.logits % unit) && !((uintptr_t)a.out % unit) && a.row_stride % 4 == 0 &&
                     a.out_row_stride % 4 == 0;
    const bool small = (long long)a.n_rows * ((a.vocab + 8191) / 8192) < 3 * 152;
    if (vec) return small ? launch_t<T, 128, true>(a, st) : launch_t<T, 512, true>(a, st);
    return small ? launch_t<T, 128, false>(a, st) : launch_t<T, 512, false>(a, st);
}

}  // namespace

cudaError_t launch_process_logits(const qw_process_logits_args &a, cudaStream_t st) {
    return a.dtype == QW_DT_F32   ? launch_vec<float>(a, st)
           : a.dtype == QW_DT_F16 ? launch_vec<__half>(a, st)
                                  : launch_vec<__nv_bfloat16>(a, st);
}

}  // namespace qw
