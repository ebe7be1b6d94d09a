// sample_rows.cu - the next token of many rows of logits, drawn with given random numbers.
//
// Per row, with the tokens in order of falling logit x (ties by rising id; NaN and -inf are no
// candidates) and the weights w = e^((x - max) / T):
//   n_k = top_k (or all), Z = sum of the first n_k weights
//   n_p = the least j with w_1 + ... + w_j >= top_p Z     (top_p < 1)
//   n_m = how many have w >= min_p w_1
//   n   = min(n_k, n_p, n_m), S = w_1 + ... + w_n, token = the first j with w_1 + ... + w_j > u S
// T = 0 takes token 1.
//
// Nothing is sorted but the few tokens that stay in question.  A row belongs to the CTAs of one cluster,
// each with a piece of it in shared memory:
//   1. the greatest (logit, id) of the row;
//   2. every token's weight, added up per octave below the greatest: how many tokens and how much weight
//      each octave holds tells which of them the borders (top_k, top_p, min_p) fall in;
//   3. the tokens down to that octave, if they are at most kList, are gathered in the first CTA, sorted and
//      run through the definition.  Otherwise each border is looked for by itself: the octave's range of (logit, id)
//      keys is cut in kBins parts, counted and weighed again until what is left fits the list.
//
// Weights are whole numbers, 2^wb for the weight 1 (wb >= 38, 44 at a vocabulary of 151,936), so that their
// sums are exact: they do not depend on the order of addition, on the number of CTAs or on timing, and a
// border that is met exactly is met.  A weight itself is off by about 3e-10 (weigh()): where it is decided by a
// running sum which token is drawn, f32 weights (6e-8, and 4e-7 from the product with 1 / T) would move a border
// past a token of weight 1e-6 in every tenth row.
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "qw_ops.h"

namespace cg = cooperative_groups;

namespace qw {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 16;
constexpr int kList = 2048;
constexpr int kMaxCluster = 8;
constexpr int kCountBit = 52;     // of a thread's bin: its sum of weights below, its count above
constexpr int kMantBits = 37;     // of a weight's mantissa
constexpr int kSteps = 64;        // of the table of 2^(i / 64)
static_assert(kWarps == kBins, "one warp adds up one bin");

using u64 = unsigned long long;

struct Table {
    u64 fix[kSteps];  // 2^(i / 64) in units of 2^-37
};
struct Step {
    u64 fix;          // the same
    float f;          // and in f32
    unsigned pad;
};

struct SampleArgs {
    const void *logits;
    int64_t stride;
    int V, per, id_bits, wb;      // per: tokens per CTA of the cluster
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens, *kept;
    float *probs;
};

__device__ __forceinline__ uint32_t ord_bits(float v) {
    const uint32_t u = __float_as_uint(v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float ord_value(uint32_t e) {
    return __uint_as_float((e & 0x80000000u) ? (e & 0x7fffffffu) : ~e);
}

// NaN is -inf, -0 is +0, +inf the greatest finite number.
__device__ __forceinline__ float canonical(float x) {
    x = x == x ? fminf(x, FLT_MAX) : -INFINITY;
    return x + 0.f;
}

// What is the same for all tokens of a row.
struct Row {
    float chi, clo;   // log2(e) / T in two terms
    float top;        // the greatest logit
    int oct;          // octave of the greatest logit's weight
    bool far;         // x log2(e) / T leaves the range of the short form
    int wb;
};

constexpr float kMagic = 196608.f;  // 1.5 x 2^17: adding it rounds to multiples of 2^-6

// z = x log2(e) / T (far: (x - top) log2(e) / T) as q / 64 + r, |r| <= 1/128, r right to about 2^-31.  q does not fall as x rises.
// Products and sums that must not be contracted are spelt out.
__device__ __forceinline__ void split(const Row &w, float x, int &q, float &r) {
    float p, e;
    if (!w.far) {
        p = __fmul_rn(x, w.chi);
        e = __fmaf_rn(x, w.clo, __fmaf_rn(x, w.chi, -p));
    } else {
        const float s = __fsub_rn(x, w.top), b = __fsub_rn(s, x);
        const float rest = __fadd_rn(__fsub_rn(x, __fsub_rn(s, b)), __fsub_rn(-w.top, b));  // x - top = s + rest
        p = fmaxf(__fmul_rn(s, w.chi), -4096.f);
        e = __fmaf_rn(s, w.clo, __fmaf_rn(s, w.chi, -p));
        e = p > -4096.f ? __fmaf_rn(rest, w.chi, e) : 0.f;
    }
    p = fmaxf(p, -65000.f);
    const float t = __fadd_rn(p, kMagic);
    q = __float_as_int(t) - __float_as_int(kMagic);
    r = __fadd_rn(__fsub_rn(p, __fsub_rn(t, kMagic)), e);
}

// Octaves below the greatest weight, and the weight in units of 2^-wb: 2^(q / 64) from the table, times 2^r - 1 by
// its series to r^3 (the rest is 4e-11), which is small (0.0055) and so right to 3e-10 in f32.
__device__ __forceinline__ u64 weigh(const Row &w, const Step *step, float x, int &oct) {
    int q;
    float r;
    split(w, x, q, r);
    oct = w.oct - (q >> 6);
    if (oct > 63) return 0ull;
    const Step m = step[q & (kSteps - 1)];
    const float up = r * fmaf(r, fmaf(r, 0.05550411f, 0.24022651f), 0.69314718f);   // ln2, ln2^2 / 2, ln2^3 / 6
    const u64 mant = m.fix + (long long)__float2int_rn(m.f * up);
    const u64 wide = mant << (w.wb - kMantBits - 1);
    return oct ? (wide + (1ull << (oct - 1))) >> oct : wide;
}

__device__ __forceinline__ u64 key_of(float x, int id, int id_bits) {
    return ((u64)ord_bits(x) << id_bits) | (((1ull << id_bits) - 1ull) - (u64)id);
}

__device__ __forceinline__ u64 shfl_xor64(u64 v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

// ceil and floor of p Z for 0 <= p < 1, exact (p has 24 bits)
__device__ __forceinline__ u64 times(float p, u64 Z, bool up) {
    const u64 f = __float2ull_rz(p * 18446744073709551616.f);
    return __umul64hi(f, Z) + (up && f * Z != 0ull ? 1ull : 0ull);
}

struct Total {
    u64 w;
    unsigned n, pad;
};

// A token's key, and the number and weight of the tokens down to it.
struct Border {
    u64 key, w;
    unsigned n, pad;
};

struct Shared {
    Step step[kSteps];
    Total xch[2][kMaxCluster][kBins];   // a pass's bins of every CTA of the cluster
    Total total[kBins];                 // and their sums
    Total cum[kBins];                   // of the octaves: each with the ones above it
    u64 best[kMaxCluster];              // greatest key of every CTA
    u64 warp_best[kWarps];
    u64 list[kList];
    u64 scan[kWarps];
    unsigned listed;
    int first[3];                       // places in the sorted list
    Border found;                       // of a search
    float cut;                          // the least logit that min_p keeps
};

template <typename T, bool RES>
struct Piece {
    const T *src;         // the row
    const float *kept;    // its piece in shared memory, canonical
    int begin, end;       // tokens of this CTA
    __device__ __forceinline__ float at(int i) const {
        if constexpr (RES) return kept[i - begin];
        else return canonical(elem_to_f(src[i]));
    }
};

// One pass: every token that `bin` gives a bin in [0, kBins) is counted and weighed there; sh.total has the cluster's sums.
template <typename P, typename F>
__device__ void tally(const P &piece, Shared &sh, u64 *bins, cg::cluster_group &cl, int &turn, F bin) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
#pragma unroll
    for (int b = 0; b < kBins; ++b) bins[b * kThreads + tid] = 0ull;
    for (int i = piece.begin + tid; i < piece.end; i += kThreads) {
        u64 w;
        const int b = bin(piece.at(i), i, w);
        if (b >= 0) bins[b * kThreads + tid] += (1ull << kCountBit) + w;
    }
    __syncthreads();
    u64 w = 0;
    unsigned n = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        const u64 v = bins[warp * kThreads + lane + 32 * i];
        w += v & ((1ull << kCountBit) - 1ull);
        n += (unsigned)(v >> kCountBit);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        w += shfl_xor64(w, o);
        n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    const unsigned ctas = cl.num_blocks(), me = cl.block_rank();
    if (lane < ctas) *cl.map_shared_rank(&sh.xch[turn][me][warp], lane) = Total{w, n, 0u};
    if (ctas > 1) cl.sync();
    else __syncthreads();
    if (tid < kBins) {
        Total t{0ull, 0u, 0u};
        for (unsigned c = 0; c < ctas; ++c) {
            t.w += sh.xch[turn][c][tid].w;
            t.n += sh.xch[turn][c][tid].n;
        }
        sh.total[tid] = t;
    }
    turn ^= 1;  // a CTA that is ahead writes the other half
    __syncthreads();
}

// Descending bitonic sort of the list, n a power of two.
__device__ void sort_list(u64 *k, int n) {
    for (int size = 2; size <= n; size <<= 1)
        for (int stride = size >> 1; stride > 0; stride >>= 1) {
            __syncthreads();
            for (int i = threadIdx.x; i < n / 2; i += kThreads) {
                const int lo = 2 * i - (i & (stride - 1)), hi = lo + stride;
                const u64 a = k[lo], b = k[hi];
                if ((a < b) == ((lo & size) == 0)) {
                    k[lo] = b;
                    k[hi] = a;
                }
            }
        }
    __syncthreads();
}

// The tokens that `take` names go to the first CTA's list (sh.listed of them, at most kList), where they are sorted, with the running
// sums of their weights in cum, from `above` on.  False in the other CTAs.
template <typename P, typename F>
__device__ bool gather(const P &piece, Shared &sh, u64 *cum, cg::cluster_group &cl, const Row &row, int id_bits, u64 above, F take) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const unsigned ctas = cl.num_blocks();
    u64 *list = cl.map_shared_rank(sh.list, 0);
    unsigned *listed = cl.map_shared_rank(&sh.listed, 0);
    for (int i0 = piece.begin + 32 * warp; i0 < piece.end; i0 += kThreads) {
        const int i = i0 + lane;
        const float x = i < piece.end ? piece.at(i) : -INFINITY;
        const bool mine = x > -INFINITY && take(x, i);
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (!who) continue;
        unsigned base = 0;
        if (lane == 0) base = atomicAdd(listed, (unsigned)__popc(who));
        base = __shfl_sync(0xffffffffu, base, 0) + __popc(who & ((1u << lane) - 1u));
        if (mine && base < kList) list[base] = key_of(x, i, id_bits);
    }
    if (ctas > 1) cl.sync();
    else __syncthreads();
    if (cl.block_rank() != 0) return false;
    const int n = min((int)sh.listed, kList);
    int pow2 = 32;
    while (pow2 < n) pow2 <<= 1;
    for (int i = n + tid; i < pow2; i += kThreads) sh.list[i] = 0ull;
    sort_list(sh.list, pow2);
    // running sums: each thread takes a few neighbours
    const int each = (n + kThreads - 1) / kThreads;
    u64 mine[kList / kThreads], sum = 0;
    int oct;
    for (int j = 0; j < each; ++j) {
        const int i = tid * each + j;
        mine[j] = i < n ? weigh(row, sh.step, ord_value((uint32_t)(sh.list[i] >> id_bits)), oct) : 0ull;
        sum += mine[j];
    }
    u64 upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sh.scan[warp] = upto;
    __syncthreads();
    u64 run = above + upto - sum;
    for (int k = 0; k < warp; ++k) run += sh.scan[k];
    for (int j = 0; j < each; ++j) {
        run += mine[j];
        if (tid * each + j < n) cum[tid * each + j] = run;
    }
    __syncthreads();
    return true;
}

// First place of the sorted list for which `is` holds, n if none does.
template <typename F>
__device__ int first_of(Shared &sh, int n, int slot, F is) {
    if (threadIdx.x == 0) sh.first[slot] = n;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads)
        if (is(i)) {
            atomicMin(&sh.first[slot], i);
            break;
        }
    __syncthreads();
    return sh.first[slot];
}

// W / S, both up to 2^63, in f32
__device__ __forceinline__ float ratio(u64 W, u64 S) {
    const float w = __ull2float_rz(W), s = __ull2float_rz(S);
    const float wl = (float)(W - (u64)w), sl = (float)(S - (u64)s);
    const float q = w / s;
    return q + (fmaf(-q, s, w) + fmaf(-q, sl, wl)) / s;
}

template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) sample_rows_kernel(const __grid_constant__ SampleArgs a,
                                                               const __grid_constant__ Table table) {
    extern __shared__ __align__(16) uint8_t smem_sample[];
    Shared &sh = *reinterpret_cast<Shared *>(smem_sample);
    u64 *bins = reinterpret_cast<u64 *>(smem_sample + (sizeof(Shared) + 15) / 16 * 16);
    float *sx = reinterpret_cast<float *>(bins + kBins * kThreads);
    cg::cluster_group cl = cg::this_cluster();
    const unsigned ctas = cl.num_blocks(), me = cl.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = blockIdx.x / ctas;
    if (ctas > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");

    const float T_ = a.temperature ? a.temperature[r] : 1.f, u = a.u[r];
    const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f;
    const int top_k = a.top_k ? a.top_k[r] : 0;
    const bool greedy = T_ == 0.f;
    const bool valid = greedy || (T_ >= 1e-6f && T_ <= 1e6f && top_p > 0.f && top_p <= 1.f && min_p >= 0.f && min_p <= 1.f &&
                                  u >= 0.f && u < 1.f);
    if (tid < kSteps) sh.step[tid] = Step{table.fix[tid], (float)table.fix[tid], 0u};
    if (tid == 0) sh.listed = 0;

    // the row's piece, and its greatest key
    Piece<T, RES> piece;
    piece.src = reinterpret_cast<const T *>(a.logits) + (int64_t)r * a.stride;
    piece.begin = min(a.V, (int)me * a.per);
    piece.end = min(a.V, piece.begin + a.per);
    piece.kept = sx;
    u64 best = 0;
    {
        constexpr int E = 16 / sizeof(T);
        const T *p = piece.src + piece.begin;
        const int n = piece.end - piece.begin;
        const int head = min(n, (int)((16u - (unsigned)((uintptr_t)p & 15u)) & 15u) / (int)sizeof(T));
        const int vecs = (n - head) / E;
        float mx = -INFINITY;
        int at = 0;
        auto take = [&](int i, float v) {
            const float x = canonical(v);
            if constexpr (RES) sx[i] = x;
            if (x > mx || (x == mx && i < at)) mx = x, at = i;
        };
        const uint4 *pv = reinterpret_cast<const uint4 *>(p + head);
        constexpr int U = 4;
        for (int v0 = tid; v0 < vecs; v0 += U * kThreads) {
            uint4 raw[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (v0 + k * kThreads < vecs) raw[k] = __ldg(pv + v0 + k * kThreads);
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (v0 + k * kThreads < vecs) {
                    const T *e = reinterpret_cast<const T *>(&raw[k]);
#pragma unroll
                    for (int j = 0; j < E; ++j) take(head + (v0 + k * kThreads) * E + j, elem_to_f(e[j]));
                }
        }
        for (int i = tid; i < head; i += kThreads) take(i, elem_to_f(p[i]));
        for (int i = head + vecs * E + tid; i < n; i += kThreads) take(i, elem_to_f(p[i]));
        if (mx > -INFINITY) best = key_of(mx, piece.begin + at, a.id_bits);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) best = max(best, shfl_xor64(best, o));
    if (lane == 0) sh.warp_best[warp] = best;
    __syncthreads();
    best = 0;
    for (int k = 0; k < kWarps; ++k) best = max(best, sh.warp_best[k]);
    if (ctas > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster is there
        if (tid < ctas) *cl.map_shared_rank(&sh.best[me], tid) = best;
        cl.sync();
        for (unsigned c = 0; c < ctas; ++c) best = max(best, sh.best[c]);
    }
    const u64 id_mask = (1ull << a.id_bits) - 1ull;
    auto answer = [&](int token, float prob, int kept) {
        a.tokens[r] = token;
        if (a.probs) a.probs[r] = prob;
        if (a.kept) a.kept[r] = kept;
    };
    if (!valid || best == 0 || greedy) {
        if (me == 0 && tid == 0) {
            if (!valid || best == 0) answer(-1, 0.f, 0);
            else answer((int)(id_mask - (best & id_mask)), 1.f, 1);
        }
        return;
    }

    Row row;
    row.top = ord_value((uint32_t)(best >> a.id_bits));
    row.wb = a.wb;
    // log2(e) in two terms, divided by T in two terms
    row.chi = __fdiv_rn(1.44269502f, T_);
    row.clo = __fdiv_rn(__fadd_rn(__fmaf_rn(-row.chi, T_, 1.44269502f), 1.92596299e-8f), T_);
    row.far = !(fabsf(row.top * row.chi) < 60000.f);
    {
        int q;
        float f;
        split(row, row.top, q, f);
        row.oct = q >> 6;
    }
    // logits below this are less than min_p of the greatest
    float cut = -INFINITY;
    if (min_p > 0.f) {
        if (tid == 0) {
            const double m = (double)row.top + (double)T_ * log((double)min_p);
            float f = (float)m;
            if ((double)f < m) f = nextafterf(f, INFINITY);
            sh.cut = f;
        }
        __syncthreads();
        cut = sh.cut;
    }

    int turn = 0;
    auto octave = [&](int oct) { return min(oct, kBins - 1); };
    tally(piece, sh, bins, cl, turn, [&](float x, int, u64 &w) {
        if (x == -INFINITY) return -1;
        int oct;
        w = weigh(row, sh.step, x, oct);
        return octave(oct);
    });
    if (tid < kBins) {
        Total t{0ull, 0u, 0u};
        for (int b = 0; b <= tid; ++b) {
            t.w += sh.total[b].w;
            t.n += sh.total[b].n;
        }
        sh.cum[tid] = t;
    }
    __syncthreads();
    const Total whole = sh.cum[kBins - 1];
    const bool has_k = top_k > 0 && (unsigned)top_k < whole.n, has_p = top_p < 1.f;
    int oct_m = kBins - 1;  // octave of the least logit that min_p keeps
    if (min_p > 0.f) {
        int q;
        float f;
        split(row, cut, q, f);
        oct_m = octave(row.oct - (q >> 6));
    }
    // the octave in which the count, or the weight, reaches a number
    auto first_n = [&](unsigned n) {
        int b = 0;
        while (b < kBins - 1 && sh.cum[b].n < n) ++b;
        return b;
    };
    auto first_w = [&](u64 w) {
        int b = 0;
        while (b < kBins - 1 && sh.cum[b].w < w) ++b;
        return b;
    };
    // the last octave that can matter
    int last = has_k ? first_n((unsigned)top_k) : kBins - 1;
    if (has_p) {
        if (!has_k) last = min(first_w(times(top_p, whole.w, true)), oct_m);
    } else {
        last = min(last, oct_m);
    }

    if (sh.cum[last].n <= kList) {
        if (!gather(piece, sh, bins, cl, row, a.id_bits, 0ull, [&](float x, int) {
                int q;
                float f;
                split(row, x, q, f);
                return octave(row.oct - (q >> 6)) <= last;
            }))
            return;
        const u64 *run = bins;
        int n = (int)sh.listed;
        u64 Z = whole.w;
        if (has_k) {
            n = min(n, top_k);
            Z = run[n - 1];
        }
        if (has_p) {
            const u64 goal = times(top_p, Z, true);
            n = min(n, 1 + first_of(sh, n, 0, [&](int i) { return run[i] >= goal; }));
        }
        if (min_p > 0.f) n = first_of(sh, n, 1, [&](int i) { return ord_value((uint32_t)(sh.list[i] >> a.id_bits)) < cut; });
        const u64 S = run[n - 1], goal = times(u, S, false) + 1ull;
        const int j = min(n - 1, first_of(sh, n, 2, [&](int i) { return run[i] >= goal; }));
        if (tid == 0) answer((int)(id_mask - (sh.list[j] & id_mask)), ratio(run[j] - (j ? run[j - 1] : 0ull), S), n);
        return;
    }

    // Each border by itself: the token at which the count, or the weight, of those down to it reaches `goal`.
    auto search = [&](bool by_count, u64 goal) {
        const int oct = by_count ? first_n((unsigned)goal) : first_w(goal);
        Total above = oct ? sh.cum[oct - 1] : Total{0ull, 0u, 0u};
        unsigned inside = sh.cum[oct].n - above.n;
        // the octave's keys [lo, end), with room for the roundings of its ends
        u64 lo, end;
        {
            const float base = row.far ? row.top : 0.f;
            auto edge = [&](int q) { return base + (float)q * (1.f / kSteps) / row.chi; };
            float hi = edge((row.oct - oct + 1) * kSteps + 1), low = edge((row.oct - oct) * kSteps - 1);
            hi += (fabsf(hi) + fabsf(base)) * 1e-6f;
            low -= (fabsf(low) + fabsf(base)) * 1e-6f;
            if (!(hi < row.top)) hi = row.top;
            if (oct == kBins - 1 || !(low > -FLT_MAX)) low = -FLT_MAX;
            lo = (u64)ord_bits(canonical(low)) << a.id_bits;
            end = ((u64)ord_bits(canonical(hi)) + 1ull) << a.id_bits;
        }
        auto in_range = [&](float x, int i, u64 &key) {
            int q;
            float f;
            split(row, x, q, f);
            key = key_of(x, i, a.id_bits);
            return octave(row.oct - (q >> 6)) == oct && key >= lo && key < end;
        };
        while (inside > kList) {  // shorter by four bits each time; a single key is one token
            int shift = 0;
            while ((end - lo - 1ull) >> shift >= (u64)kBins) ++shift;
            tally(piece, sh, bins, cl, turn, [&](float x, int i, u64 &w) {
                u64 key;
                if (x == -INFINITY || !in_range(x, i, key)) return -1;
                int o;
                w = weigh(row, sh.step, x, o);
                return kBins - 1 - (int)((key - lo) >> shift);  // the greatest keys first
            });
            int b = 0;
            for (; b < kBins - 1; ++b) {
                const Total t = sh.total[b];
                if ((by_count ? (u64)(above.n + t.n) : above.w + t.w) >= goal) break;
                above.w += t.w;
                above.n += t.n;
            }
            inside = sh.total[b].n;
            lo += (u64)(kBins - 1 - b) << shift;
            end = min(end, lo + (1ull << shift));
            __syncthreads();
        }
        if (gather(piece, sh, bins, cl, row, a.id_bits, above.w, [&](float x, int i) {
                u64 key;
                return in_range(x, i, key);
            })) {
            const int n = (int)sh.listed;
            int j = by_count ? (int)(goal - above.n) - 1 : first_of(sh, n, 0, [&](int i) { return bins[i] >= goal; });
            j = max(0, min(j, n - 1));
            if (tid < ctas) *cl.map_shared_rank(&sh.found, tid) = Border{sh.list[j], bins[j], above.n + (unsigned)j + 1u, 0u};
            __syncthreads();
            if (tid == 0) sh.listed = 0;
        }
        if (ctas > 1) cl.sync();
        else __syncthreads();
        const Border f = sh.found;
        __syncthreads();
        return f;
    };
    Border kept{0ull, whole.w, whole.n, 0u};
    if (has_k) kept = search(true, (u64)top_k);
    if (has_p) kept = search(false, max(1ull, times(top_p, kept.w, true)));
    if (min_p > 0.f) {
        tally(piece, sh, bins, cl, turn, [&](float x, int i, u64 &w) {
            if (x == -INFINITY || x < cut || key_of(x, i, a.id_bits) < kept.key) return -1;
            int o;
            w = weigh(row, sh.step, x, o);
            return 0;
        });
        kept.w = sh.total[0].w;
        kept.n = sh.total[0].n;
        __syncthreads();
    }
    const Border drawn = search(false, times(u, kept.w, false) + 1ull);
    if (me == 0 && tid == 0) {
        int o;
        const u64 w = weigh(row, sh.step, ord_value((uint32_t)(drawn.key >> a.id_bits)), o);
        answer((int)(id_mask - (drawn.key & id_mask)), ratio(w, kept.w), (int)kept.n);
    }
}

template <typename T, bool RES>
cudaError_t launch_rows(const SampleArgs &a, const Table &t, int rows, int ctas, size_t smem, cudaStream_t st) {
    cudaError_t e = allow_smem<sample_rows_kernel<T, RES>>(227 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows * ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_rows_kernel<T, RES>, a, t);
}

const Table &table() {
    static const Table t = [] {
        Table x;
        for (int i = 0; i < kSteps; ++i) x.fix[i] = (u64)std::llround(std::ldexp(std::exp2((double)i / kSteps), kMantBits));
        return x;
    }();
    return t;
}

int bits_for(int64_t n) {  // least b with n <= 2^b
    int b = 0;
    while ((1ll << b) < n) ++b;
    return b;
}

}  // namespace

cudaError_t launch_sample_rows(const qw_sample_rows_args &q, cudaStream_t st) {
    const size_t fixed = (sizeof(Shared) + 15) / 16 * 16 + (size_t)kBins * kThreads * 8;
    const size_t room = 227 * 1024 - fixed;
    int ctas = 1;
    auto per = [&] { return (int)(((int64_t)q.vocab + ctas - 1) / ctas + 7) / 8 * 8; };
    while (ctas < kMaxCluster && per() > 4096 && ((int64_t)q.n_rows * ctas < 152 || (size_t)per() * 4 > room / 2)) ctas *= 2;
    SampleArgs a{};
    a.logits = q.logits;
    a.stride = q.row_stride;
    a.V = q.vocab;
    a.per = per();
    a.id_bits = bits_for(q.vocab);
    a.wb = std::min(62 - a.id_bits, kCountBit - 1 - bits_for((a.per + kThreads - 1) / kThreads));
    a.u = q.u, a.temperature = q.temperature, a.top_p = q.top_p, a.min_p = q.min_p, a.top_k = q.top_k;
    a.tokens = q.tokens, a.kept = q.kept, a.probs = q.probs;
    const bool res = (size_t)a.per * 4 <= room;
    const size_t smem = fixed + (res ? (size_t)a.per * 4 : 0);
    const Table &t = table();
    if (q.dtype == QW_DT_F32) return res ? launch_rows<float, true>(a, t, q.n_rows, ctas, smem, st) : launch_rows<float, false>(a, t, q.n_rows, ctas, smem, st);
    if (q.dtype == QW_DT_F16) return res ? launch_rows<__half, true>(a, t, q.n_rows, ctas, smem, st) : launch_rows<__half, false>(a, t, q.n_rows, ctas, smem, st);
    return res ? launch_rows<__nv_bfloat16, true>(a, t, q.n_rows, ctas, smem, st)
               : launch_rows<__nv_bfloat16, false>(a, t, q.n_rows, ctas, smem, st);
}

}  // namespace qw
