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
// takes a few consecutive chunks of a row.  The row's lists (a few KB) stay in registers;
// for each chunk the CTA keeps what falls in it in shared memory, as a dense count and a
// dense bias per token, while the chunk's logits are on their way: the loads of the next
// chunk are issued as soon as this one's values are out.  (One chunk per CTA spent most of
// its time waiting in turn for the lists and for the logits: 256 x 151936 f32 took 91 us; now 75,
// 4.1 TB/s, 61% of the measured copy rate.)
// Counts are whole numbers, so the order of their atomics does not matter; the biases of a token that
// is named more than once are added to its logit by the list's first entry alone, in order,
// so results do not depend on timing.
#include "qw_ops.h"

namespace qw {
namespace {

constexpr int kVecs = 4;           // vectors of four tokens per thread
constexpr int kIds = 4, kBias = 1;  // list entries that a thread keeps in registers; longer lists are read again
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

// [begin, end) of a row's list, both kept inside the array; empty without a list.
__device__ __forceinline__ int2 list_range(const int32_t *range, int r, int n) {
    return range ? make_int2(min(max(range[2 * r], 0), n), min(range[2 * r + 1], n)) : make_int2(0, 0);
}

enum { ROWS_ANY, ROWS_ALIKE, ROWS_ALIGNED };

// ROWS: aligned, every row begins on a vector boundary; alike, a row of logits and its output lie
// alike to vector boundaries, `pad` elements behind one (an odd vocabulary puts every row
// elsewhere): vectors begin there, and the first and last are cut; any, no vectors.  SPARSE: there are
// lists to look at.  (The masks of cut vectors straddle words: treating aligned rows alike
// took 94 us for 256 x 151936 f32 instead of 69.)
template <typename T, int kThreads, int ROWS, bool SPARSE>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logits_kernel(const qw_process_logits_args a, int chunks) {
    constexpr bool VEC = ROWS != ROWS_ANY;
    constexpr int kTok = kThreads * 4 * kVecs;
    // [kTok] counts and flags; of the flagged: first list entry, and the bias or (named twice) the biased logit
    extern __shared__ __align__(16) uint32_t sm[];
    uint32_t *cnt = sm, *entry = sm + kTok;
    float *add = reinterpret_cast<float *>(sm + 2 * kTok);
    const int r = blockIdx.y, V = a.vocab, tid = threadIdx.x;
    const T *src = reinterpret_cast<const T *>(a.logits) + (int64_t)r * a.row_stride;
    T *dst = reinterpret_cast<T *>(a.out) + (int64_t)r * a.out_row_stride;
    const int pad = ROWS == ROWS_ALIKE ? (int)((uintptr_t)src / sizeof(T)) & 3 : 0;
    const int end = min((int)((blockIdx.x + 1) * chunks * kTok) - pad, V);
    const int which = a.mask ? (a.mask_index ? a.mask_index[r] : r) : -1;
    const bool none = a.mask && which >= a.n_masks;  // an index past the masks: nothing is allowed
    const uint32_t *mask = which >= 0 && !none ? a.mask + (int64_t)which * ((V + 31) / 32) : nullptr;
    int2 hist = make_int2(0, 0), bias = make_int2(0, 0);
    float rep = 1.f, pres = 0.f, freq = 0.f;
    if constexpr (SPARSE) {
        if (a.penalties) {
            rep = a.penalties[3 * r], pres = a.penalties[3 * r + 1], freq = a.penalties[3 * r + 2];
            if (a.history) hist = list_range(a.history_range, r, a.n_history);
        }
        if (a.bias) bias = list_range(a.bias_range, r, a.n_bias);
    }
    auto penalised = [&](float x, uint32_t c) {
        if (c & kCount) {
            x = x > 0.f ? x / rep : x * rep;
            x -= pres + freq * (float)(c & kCount);
        }
        return x;
    };
    float v[kVecs][4];
    uint32_t word[kVecs];  // the vector's mask bits
    auto load = [&](int base) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int t = base + 4 * (tid + kThreads * j);
            if (VEC && t >= 0 && t + 4 <= V) {
                load4(src + t, v[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // without vectors a warp still reads runs of 32 neighbours
                    const int s = VEC ? t + i : base + 4 * kThreads * j + kThreads * i + tid;
                    v[j][i] = s >= 0 && s < V ? elem_to_f(src[s]) : 0.f;
                }
            }
            if constexpr (ROWS == ROWS_ALIGNED) {
                word[j] = mask && t < V ? mask[t >> 5] >> (t & 31) : none ? 0u : ~0u;
            } else if constexpr (VEC) {
                word[j] = none ? 0u : ~0u;
                if (mask && t < V) {  // four bits from bit t on, of a word and perhaps the next; t may be -3 .. -1
                    const uint32_t lo = t >= 0 ? mask[t >> 5] : 0u;
                    const uint32_t hi = (t & 31) > 28 && ((t + 3) >> 5) < (V + 31) / 32 ? mask[(t + 3) >> 5] : 0u;
                    word[j] = __funnelshift_r(lo, hi, t & 31);
                }
            }
        }
    };
    int base = blockIdx.x * chunks * kTok - pad;
    load(base);
    int32_t ids[kIds], bid[kBias], own = -1;
    float bval[kBias];
    if constexpr (SPARSE) {
#pragma unroll
        for (int k = 0; k < kIds; ++k) {
            const int i = hist.x + tid + kThreads * k;
            ids[k] = i < hist.y ? a.history[i] : -1;
        }
#pragma unroll
        for (int k = 0; k < kBias; ++k) {
            const int i = bias.x + tid + kThreads * k;
            bid[k] = i < bias.y ? a.bias_ids[i] : -1;
            bval[k] = i < bias.y ? a.bias[i] : 0.f;
        }
        if (a.penalties && a.path && tid < a.path_len) own = a.path[(int64_t)r * a.path_len + tid];
        uint4 *z = reinterpret_cast<uint4 *>(cnt);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            z[tid + kThreads * i] = make_uint4(0u, 0u, 0u, 0u);
            if (a.bias) z[tid + kThreads * (i + kVecs)] = make_uint4(~0u, ~0u, ~0u, ~0u);
        }
        __syncthreads();
    }
    for (; base < end; base += kTok) {
        if constexpr (SPARSE) {
            // a token outside the vocabulary falls in no chunk, or behind or before the row (an id of -1 to -3 in
            // the cut front of the first vector): what is computed for it is not stored
            auto count = [&](int32_t id) {
                const uint32_t t = (uint32_t)id - (uint32_t)base;
                if (t < (uint32_t)kTok) atomicAdd(cnt + t, 1u);
            };
            auto name = [&](int i, int32_t id) {
                const uint32_t t = (uint32_t)id - (uint32_t)base;
                if (t >= (uint32_t)kTok) return;
                if (atomicOr(cnt + t, kNamed) & kNamed) atomicOr(cnt + t, kTwice);
                atomicMin(entry + t, (uint32_t)i);
            };
            // entry i of the list: the first mention of a token does the work of all.  Its logit is still in src, in
            // place too: this chunk is written behind the barrier below.
            auto settle = [&](int i, int32_t id, float x) {
                const uint32_t t = (uint32_t)id - (uint32_t)base;
                if (t >= (uint32_t)kTok || entry[t] != (uint32_t)i) return;
                const uint32_t c = cnt[t];
                if ((c & kTwice) && (uint32_t)id < (uint32_t)V) {
                    x += penalised(elem_to_f(src[id]), c);
#pragma unroll 8
                    for (int k = i + 1; k < bias.y; ++k) {
                        const int32_t other = a.bias_ids[k];
                        if (other == id) x += a.bias[k];
                    }
                }
                add[t] = x;
            };
            count(own);
#pragma unroll
            for (int k = 0; k < kIds; ++k) count(ids[k]);
            for (int i = hist.x + tid + kThreads * kIds; i < hist.y; i += kThreads) count(a.history[i]);
            if (a.penalties && a.path)
                for (int i = tid + kThreads; i < a.path_len; i += kThreads) count(a.path[(int64_t)r * a.path_len + i]);
            if (a.bias) {
#pragma unroll
                for (int k = 0; k < kBias; ++k) name(bias.x + tid + kThreads * k, bid[k]);
                for (int i = bias.x + tid + kThreads * kBias; i < bias.y; i += kThreads) name(i, a.bias_ids[i]);
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kBias; ++k) settle(bias.x + tid + kThreads * k, bid[k], bval[k]);
                for (int i = bias.x + tid + kThreads * kBias; i < bias.y; i += kThreads) settle(i, a.bias_ids[i], a.bias[i]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int l0 = 4 * (tid + kThreads * j), t0 = base + l0;
            // most vectors hold no listed token
            auto listed = [&](float x, uint32_t c, int l) {
                x = penalised(x, c);
                if (c & kNamed) {
                    x = c & kTwice ? add[l] : x + add[l];
                    entry[l] = ~0u;  // for the next chunk
                }
                return x;
            };
            if constexpr (VEC) {
                if constexpr (SPARSE) {
                    uint4 *c4 = reinterpret_cast<uint4 *>(cnt + l0);
                    const uint4 c = *c4;
                    if (c.x | c.y | c.z | c.w) {
                        *c4 = make_uint4(0u, 0u, 0u, 0u);  // for the next chunk
                        if (c.x) v[j][0] = listed(v[j][0], c.x, l0);
                        if (c.y) v[j][1] = listed(v[j][1], c.y, l0 + 1);
                        if (c.z) v[j][2] = listed(v[j][2], c.z, l0 + 2);
                        if (c.w) v[j][3] = listed(v[j][3], c.w, l0 + 3);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j][i] = (word[j] >> i) & 1u ? v[j][i] : -INFINITY;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int l = 4 * kThreads * j + kThreads * i + tid, t = base + l;
                    float x = v[j][i];
                    if constexpr (SPARSE) {
                        const uint32_t c = cnt[l];
                        if (c) {
                            cnt[l] = 0u;
                            x = listed(x, c, l);
                        }
                    }
                    const bool ok = !none && (!mask || t >= V || ((mask[t >> 5] >> (t & 31)) & 1u));
                    if (t < V) dst[t] = elem_from_f<T>(ok ? x : -INFINITY);
                }
            }
            if constexpr (VEC) {
                if (t0 >= 0 && t0 + 4 <= V) {
                    store4(dst + t0, v[j]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t0 + i >= 0 && t0 + i < V) dst[t0 + i] = elem_from_f<T>(v[j][i]);
                }
            }
        }
        if (base + kTok < end) {
            load(base + kTok);
            if constexpr (SPARSE) __syncthreads();
        }
    }
}

template <typename T, int kThreads, int ROWS>
cudaError_t launch_n(const qw_process_logits_args &a, int chunks, cudaStream_t st) {
    constexpr int kTok = kThreads * 4 * kVecs, smem = 3 * kTok * 4;
    const int all = (a.vocab + (ROWS == ROWS_ALIKE ? 3 : 0) + kTok - 1) / kTok;  // a row may begin up to three elements into a vector
    const dim3 grid((all + chunks - 1) / chunks, a.n_rows);
    if ((a.penalties && (a.history || a.path)) || a.bias) {
        const cudaError_t e = allow_smem<logits_kernel<T, kThreads, ROWS, true>>(smem);
        if (e != cudaSuccess) return e;
        return launch_k(false, logits_kernel<T, kThreads, ROWS, true>, grid, dim3(kThreads), smem, st, a, chunks);
    }
    return launch_k(false, logits_kernel<T, kThreads, ROWS, false>, grid, dim3(kThreads), 0, st, a, chunks);
}

// Many tokens: chunks of 8192, several per CTA (each list entry is looked at once per chunk); few: chunks
// of 2048, one per CTA, so that every SM gets some.
template <typename T, int ROWS>
cudaError_t launch_t(const qw_process_logits_args &a, cudaStream_t st) {
    const long long large = (long long)a.n_rows * ((a.vocab + 8191) / 8192);
    if (large < 3 * 152) return launch_n<T, 128, ROWS>(a, 1, st);
    return launch_n<T, 512, ROWS>(a, large >= 4LL * 4 * 152 ? 4 : large >= 2LL * 4 * 152 ? 2 : 1, st);
}

template <typename T>
cudaError_t launch_vec(const qw_process_logits_args &a, cudaStream_t st) {
    const size_t unit = 4 * sizeof(T);
    const bool one = a.n_rows == 1;
    if ((uintptr_t)a.logits % unit == 0 && (uintptr_t)a.out % unit == 0 &&
        (one || (a.row_stride % 4 == 0 && a.out_row_stride % 4 == 0)))
        return launch_t<T, ROWS_ALIGNED>(a, st);
    if (((uintptr_t)a.logits - (uintptr_t)a.out) % unit == 0 && (one || (a.row_stride - a.out_row_stride) % 4 == 0))
        return launch_t<T, ROWS_ALIKE>(a, st);
    return launch_t<T, ROWS_ANY>(a, st);
}

}  // namespace

cudaError_t launch_process_logits(const qw_process_logits_args &a, cudaStream_t st) {
    return a.dtype == QW_DT_F32   ? launch_vec<float>(a, st)
           : a.dtype == QW_DT_F16 ? launch_vec<__half>(a, st)
                                  : launch_vec<__nv_bfloat16>(a, st);
}

}  // namespace qw
