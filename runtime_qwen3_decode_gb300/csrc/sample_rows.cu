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
//   1. the greatest logit of the row;
//   2. every token counted (and, where weights matter, weighed) by the octaves of weight that it lies below the greatest (two
//      or half of one to a part), the last of B parts taking the rest: that tells which of them the lowest border falls in;
//   3. that part is cut in B again, by logits about the place where the border should be and at last by (logit, id) keys,
//      until the tokens down to the border are few: the first CTA gathers and sorts them and runs the definition on them.
//   4. Where more tokens are kept, each border (top_k, top_p, the draw) is looked for by itself, and only the part
//      that it falls in is sorted, by every CTA.
//   1b. top_k up to kMostShort, and min_p alone, list their tokens without a pass (8 rows of 151,936 12.3 us instead of 20.0).
// top_k needs counts alone: its passes weigh nothing.
//
// Bound by the number of instructions where passes weigh whole rows (47 a token), else by the time that a pass takes
// whatever it holds: some 3 us for its bins, the cluster's exchange and the search for the next zone's ends.  256 rows of
// 151,936 with mixed settings 258 us (HBM floor 23), 8 drawn from nearly everything 46, 8 of usual settings 12.3.
//
// Weights are whole numbers, 2^wb for the weight 1 (wb by the vocabulary: 44 at 151,936, never below 38), so that their
// sums are exact: they do not depend on the order of addition, on the number of CTAs, on the other rows or on timing, and a
// border that is met exactly is met.  A weight itself is off by 2.4e-9 of itself (weigh()) and half a unit at most: where it is
// decided by a running sum which token is drawn, f32 weights (6e-8, and 4e-7 from the product with 1 / T) would move a border
// past a token of weight 1e-6 in every tenth row.  Half units can all have one sign, V 2^-(wb + 1) together: 4.3e-9 at 151,936
// tokens, where u and top_p have steps of 6e-8, but 3e-5 at 2^24, as 64-bit sums leave no room for smaller units.
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "qw_ops.h"

namespace cg = cooperative_groups;

namespace qw {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
// Parts of a pass's zone, B in what follows: every thread has a bin of its own for each, 2 or 8 KB a warp.  32 up to two CTAs for
// every SM, which saves passes but leaves one CTA to an SM (us with 32 and with 8, rows of 151,936: 8 drawn from nearly everything 47
// and 68, 32 of mixed settings 62 and 67); else 8, so that two CTAs share an SM (64 bf16 ones 96 and 74, 256 347 and 261).
constexpr int kFewBins = 8, kManyBins = 32;
constexpr int kKeys = 4;              // sorted keys of a thread
constexpr int kList = kKeys * kThreads;  // tokens that are sorted at once, in one CTA
constexpr int kMostShort = 1200;     // top_k up to which the short way is tried
constexpr int kPart = kThreads;            // of a part that one border is looked for in, in every CTA
constexpr int kShort = 512, kNear = 128; // a border's tokens are cut down to this many, or to this many about it
constexpr int kMaxCluster = 8;
constexpr int kCountBit = 51;     // of a thread's bin: its sum of weights below, its count (up to 4096) above
constexpr int kMantBits = 36;     // of a weight's mantissa behind its point
constexpr int kSteps = 32;        // of the table of 2^(i / 32)

using u64 = unsigned long long;

// 2^(i / 32) in units of 2^-31, and in f32 in units of 2^-36: two words that each lie in a bank of their own for every i,
// so that 32 lanes read them at once whatever their i (16-byte entries of 64 steps took 12 turns a read).
struct Table {
    unsigned fix[kSteps];
    float f[kSteps];
};

struct SampleArgs {
    const void *logits;
    int64_t stride;
    int V, per, id_bits, wb;      // per: tokens per CTA of the cluster, a multiple of 8
    int rows, sorted;             // sorted: rows that take long first
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens, *kept;
    float *probs;
};

// Order numbers: a float's bits as a whole number that rises with its value, one step a float.  -0 and +0 share one: with a
// number for each, a zone that ended between them held every +0 where tokens are compared as floats, and only the tokens below where
// they are compared by keys.
__device__ __forceinline__ uint32_t ord_bits(float v) {
    const uint32_t u = __float_as_uint(v);
    return (u & 0x80000000u) ? 0u - u : (u | 0x80000000u);
}
__device__ __forceinline__ float ord_value(uint32_t e) {
    return __uint_as_float((e & 0x80000000u) ? (e & 0x7fffffffu) : 0u - e);
}

// NaN is -inf, -0 is +0, +inf the greatest finite number.
__device__ __forceinline__ float canonical(float x) {
    return fminf(fmaxf(x, -INFINITY), FLT_MAX) + 0.f;
}

// What is the same for all tokens of a row.
struct Row {
    float chi, clo;   // log2(e) / T in two terms
    float top;        // the greatest logit
    int oct;          // octave of the greatest logit's weight
    bool far;         // x log2(e) / T leaves the range of the short form
    int wb;
};

constexpr float kMagic = 393216.f;  // 1.5 x 2^18: adding it rounds to multiples of 2^-5

// z = x log2(e) / T (far: (x - top) log2(e) / T) of two logits as q / 32 + r, |r| <= 1/64, r right to about 2^-31.  q does not
// fall as x rises.  Products and sums that must not be contracted are spelt out; in pairs, as the passes are bound by the
// number of their instructions.
__device__ __forceinline__ void split2(const Row &w, float2 x, int (&q)[2], float2 &r) {
    const float2 chi = make_float2(w.chi, w.chi), clo = make_float2(w.clo, w.clo), magic = make_float2(kMagic, kMagic);
    const float2 minus = make_float2(-kMagic, -kMagic);
    auto neg = [](float2 v) { return make_float2(-v.x, -v.y); };
    float2 p, e;
    if (!w.far) {
        p = __fmul2_rn(x, chi);
        e = __ffma2_rn(x, clo, __ffma2_rn(x, chi, neg(p)));
    } else {
        const float2 top = make_float2(-w.top, -w.top);
        const float2 s = __fadd2_rn(x, top), b = __fadd2_rn(s, neg(x));
        const float2 rest = __fadd2_rn(__fadd2_rn(x, neg(__fadd2_rn(s, neg(b)))), __fadd2_rn(top, neg(b)));  // x - top = s + rest
        p = __fmul2_rn(s, chi);
        p = make_float2(fmaxf(p.x, -4096.f), fmaxf(p.y, -4096.f));
        e = __ffma2_rn(rest, chi, __ffma2_rn(s, clo, __ffma2_rn(s, chi, neg(p))));
        e = make_float2(p.x > -4096.f ? e.x : 0.f, p.y > -4096.f ? e.y : 0.f);
    }
    p = make_float2(fmaxf(p.x, -65000.f), fmaxf(p.y, -65000.f));
    const float2 t = __fadd2_rn(p, magic);
    q[0] = __float_as_int(t.x) - __float_as_int(kMagic);
    q[1] = __float_as_int(t.y) - __float_as_int(kMagic);
    r = __fadd2_rn(__fadd2_rn(p, neg(__fadd2_rn(t, minus))), e);
}

// Two weights in units of 2^-wb: 2^(q / 32) from the table, times 2^r - 1 by its series to r^4, which is small (0.011) and so
// right to 2.4e-9 in f32: r to 2^-31, the series to 2^-31, the table's f32 and its product with the series to 2^-24 of 0.011
// each; the table's whole number to 2^-32.  These errors do not add up over many tokens: they have either sign.  Rounding to a unit
// is off by half of one more.
__device__ __forceinline__ void weigh2(const Row &w, const Table &t, float2 x, u64 (&out)[2]) {
    int q[2];
    float2 r;
    split2(w, x, q, r);
    auto both = [](float v) { return make_float2(v, v); };
    // ln2, ln2^2 / 2, ln2^3 / 6, ln2^4 / 24
    const float2 up = __fmul2_rn(r, __ffma2_rn(r, __ffma2_rn(r, __ffma2_rn(r, both(0.0096181291f), both(0.055504109f)), both(0.24022651f)),
                                               both(0.69314718f)));
    const float2 part = __fmul2_rn(make_float2(t.f[q[0] & (kSteps - 1)], t.f[q[1] & (kSteps - 1)]), up);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        // in units of 2^-63, then shifted to 2^-(wb + 1) and rounded to 2^-wb; shr gives 0 for shifts of 64 and more
        const u64 mant = ((u64)t.fix[q[k] & (kSteps - 1)] << 32) +
                         (u64)((long long)__float2int_rn(k ? part.y : part.x) * (1ll << (63 - kMantBits)));
        u64 half;
        asm("shr.u64 %0, %1, %2;" : "=l"(half) : "l"(mant), "r"((unsigned)(62 - w.wb + w.oct - (q[k] >> 5))));
        out[k] = (half + 1ull) >> 1;
    }
}
__device__ __forceinline__ u64 weigh(const Row &w, const Table &t, float x) {
    u64 v[2];
    weigh2(w, t, make_float2(x, x), v);
    return v[0];
}

__device__ __forceinline__ u64 key_of(float x, int id, int id_bits) {
    return ((u64)ord_bits(x) << id_bits) | (u64)(((1u << id_bits) - 1u) & ~(unsigned)id);
}

__device__ __forceinline__ u64 shfl_xor64(u64 v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

// ceil and floor of p Z for 0 <= p < 1, exact (p has 24 bits)
__device__ __forceinline__ u64 times(float p, u64 Z, bool up) {
    const u64 f = __float2ull_rz(p * 18446744073709551616.f);
    return __umul64hi(f, Z) + (up && f * Z != 0ull ? 1ull : 0ull);
}

// Weight and number of some tokens; `low`: how many of them the CTAs before this one have.
struct Total {
    u64 w;
    unsigned n, low;
};

template <int B>
struct Shared {
    Table table;
    u64 xch_w[2][kMaxCluster][B];       // a pass's bins of every CTA of the cluster
    unsigned xch_n[2][kMaxCluster][B];
    Total total[B];                     // and their sums, each with the ones above it
    Total cum[B];                       // the same of the octaves
    float top[kMaxCluster], least[kMaxCluster];  // greatest and least logit of every CTA
    float group[kThreads];                       // greatest logits of kThreads parts of the row
    unsigned count[kMaxCluster];                 // tokens in every CTA's part of the short list
    int first_id[kMaxCluster];                   // temperature 0: its first token with the greatest logit
    float warp_top[kWarps], warp_least[kWarps];
    u64 scan[kWarps];
    unsigned listed, edge[2];
    int first[3];
    float near;                         // see below
    float cut;                          // the least logit that min_p keeps
    float at;                           // the logit from which on tokens are listed
};

// In the place of the passes' bins: a list is written by other CTAs when this one has summed its bins, and read
// before it clears them.  Two lists of parts in turn: a CTA that is ahead writes the next one.
struct Parts {
    u64 list[2][kPart], buf[2][kPart];
};
template <int B>
constexpr int kBinBytes = B * kThreads * 8;
static_assert(sizeof(Parts) <= kBinBytes<kFewBins> && kList * 8 <= kBinBytes<kFewBins>, "fits over the bins");

// How a pass cuts its tokens in B parts, the greatest first: by logit, top - x in units of 1 / inv (the first and the
// last part take the rest), or by key, (key - lo) >> shift.
template <int B>
struct Cut {
    bool by_value;
    float top, inv;
    u64 lo;
    int shift;
    // the whole part of (top - x) inv, cut at 0 and B - 1, by adding 2^23 rounding down
    __device__ __forceinline__ int slot(float x) const {
        return __float_as_int(__fadd_rd(fminf(fmaxf((top - x) * inv, 0.f), B - 1.f), 8388608.f)) & (B - 1);
    }
};

// The keys [lo, end) in question, how many tokens they are, and what lies above them.
struct Zone {
    u64 lo, end;
    Total above, inside;
};

template <typename T, bool RES>
struct Piece {
    const T *src;         // the row
    const float *kept;    // its piece in shared memory, canonical, padded to a multiple of four with -inf
    int begin, end;       // tokens of this CTA
    __device__ __forceinline__ int quads() const { return (end - begin + 3) >> 2; }
    __device__ __forceinline__ float4 at(int quad) const {
        if constexpr (RES) {
            return reinterpret_cast<const float4 *>(kept)[quad];
        } else {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = begin + 4 * quad + k;
                v[k] = i < end ? canonical(elem_to_f(src[i])) : -INFINITY;
            }
            return make_float4(v[0], v[1], v[2], v[3]);
        }
    }
    __device__ __forceinline__ float one(int i) const { return RES ? kept[i] : canonical(elem_to_f(src[begin + i])); }
};

// One pass: every token of the zone is counted in the part of it that the cut gives, and weighed if asked; sh.total has
// the cluster's sums.  Each thread has bins of its own.  ROW: the zone has no upper end and is cut by logits.
template <int B, bool WEIGHED, bool ROW, typename P>
__device__ __forceinline__ void tally(const P &piece, Shared<B> &sh, const Row &row, u64 *bins, cg::cluster_group &cl, int turn,
                                      const Zone &z, const Cut<B> &c, int id_bits) {
    const u64 id_mask = (1ull << id_bits) - 1ull;
    const float xl = ord_value((unsigned)(z.lo >> id_bits)), xh = ord_value((unsigned)((z.end - 1ull) >> id_bits));
    const int last = (int)(id_mask - (z.lo & id_mask)), first = (int)(id_mask - ((z.end - 1ull) & id_mask));
    const bool ties = ((z.lo | z.end) & id_mask) != 0ull;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr u64 kSum = (1ull << kCountBit) - 1ull;
#pragma unroll
    for (int b = 0; b < B; ++b) bins[b * kThreads + tid] = 0ull;
    const int quads = piece.quads();
    if constexpr (ROW) {
        // No branch but the one past four tokens outside: the others' numbers are 0 and go to the last bin.
        for (int g = tid; g < quads; g += kThreads) {
            const float4 v = piece.at(g);
            const float x[4] = {v.x, v.y, v.z, v.w};
            bool is[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) is[k] = x[k] >= xl;
            if (ties) {  // the zone's end is between tokens of one logit
#pragma unroll
                for (int k = 0; k < 4; ++k) is[k] &= !((x[k] == xl) & (piece.begin + 4 * g + k > last));
            }
            if (!(is[0] | is[1] | is[2] | is[3])) continue;
            u64 w[4] = {0ull, 0ull, 0ull, 0ull};
            if constexpr (WEIGHED) {
                u64 a[2], c[2];
                weigh2(row, sh.table, make_float2(x[0], x[1]), a);
                weigh2(row, sh.table, make_float2(x[2], x[3]), c);
                w[0] = a[0], w[1] = a[1], w[2] = c[0], w[3] = c[1];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) bins[(is[k] ? c.slot(x[k]) : B - 1) * kThreads + tid] += is[k] ? w[k] + (1ull << kCountBit) : 0ull;
        }
    } else {
        // A part of a part is a tenth of the row, but nearly every warp has some of it in any 32 quads: a thread marks its tokens
        // first, 64 at a time, and then weighs the marked ones, two by two.
        for (int g0 = tid; g0 < quads; g0 += 16 * kThreads) {
            u64 marks = 0ull;
            for (int i = 0, g = g0; i < 16 && g < quads; ++i, g += kThreads) {
                const float4 v = piece.at(g);
                const float x[4] = {v.x, v.y, v.z, v.w};
                unsigned m = 0u;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    bool is = (x[k] >= xl) & (x[k] <= xh);
                    if (ties) {
                        const int id = piece.begin + 4 * g + k;
                        is &= !((x[k] == xl) & (id > last)) & !((x[k] == xh) & (id < first));
                    }
                    m |= is ? 1u << k : 0u;
                }
                marks |= (u64)m << (4 * i);
            }
            while (marks) {
                int at[2];
                float x[2];
                const bool both = (marks & (marks - 1ull)) != 0ull;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (k == 1 && !both) {
                        at[1] = at[0];
                        break;
                    }
                    const int m = __ffsll((long long)marks) - 1;
                    marks &= marks - 1ull;
                    at[k] = 4 * (g0 + (m >> 2) * kThreads) + (m & 3);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) x[k] = piece.one(at[k]);
                u64 w[2] = {0ull, 0ull};
                if constexpr (WEIGHED) weigh2(row, sh.table, make_float2(x[0], x[1]), w);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (k == 1 && !both) break;
                    const int bin = c.by_value ? c.slot(x[k])
                                               : B - 1 - (int)((key_of(x[k], piece.begin + at[k], id_bits) - z.lo) >> c.shift);
                    bins[bin * kThreads + tid] += w[k] + (1ull << kCountBit);
                }
            }
        }
    }
    // 32 lanes' sums, the weights' in three words of 27 bits, which leave room for them
    auto add = [&](u64 &w, unsigned &n) {
        n = __reduce_add_sync(0xffffffffu, n);
        if constexpr (!WEIGHED) return;
        constexpr unsigned kWord = (1u << 27) - 1u;
        const unsigned a = __reduce_add_sync(0xffffffffu, (unsigned)w & kWord), b = __reduce_add_sync(0xffffffffu, (unsigned)(w >> 27) & kWord),
                       c = __reduce_add_sync(0xffffffffu, (unsigned)(w >> 54));
        w = (u64)a + ((u64)b << 27) + ((u64)c << 54);
    };
    __syncthreads();
    const unsigned ctas = cl.num_blocks(), me = cl.block_rank();
    for (int bin = warp; bin < B; bin += kWarps) {
        u64 w = 0;
        unsigned n = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            const u64 v = bins[bin * kThreads + lane + 32 * i];
            w += v & kSum;
            n += (unsigned)(v >> kCountBit);
        }
        add(w, n);
        if (lane < ctas) {
            *cl.map_shared_rank(&sh.xch_w[turn][me][bin], lane) = w;
            *cl.map_shared_rank(&sh.xch_n[turn][me][bin], lane) = n;
        }
    }
    if (ctas > 1) cl.sync();
    else __syncthreads();
    if (warp == 0) {
        Total t{0ull, 0u, 0u};
        if (lane < B)
            for (unsigned c = 0; c < ctas; ++c) {
                const unsigned n = sh.xch_n[turn][c][lane];
                t.w += sh.xch_w[turn][c][lane];
                t.n += n;
                if (c < me) t.low += n;
            }
#pragma unroll
        for (int o = 1; o < B; o <<= 1) {
            const u64 w = __shfl_up_sync(0xffffffffu, t.w, o);
            const unsigned n = __shfl_up_sync(0xffffffffu, t.n, o), low = __shfl_up_sync(0xffffffffu, t.low, o);
            if (lane >= o) t.w += w, t.n += n, t.low += low;
        }
        if (lane < B) sh.total[lane] = t;
    }
    __syncthreads();
}

// The least order number of [low, high] for which slot() is at most j (high + 1: none).  One warp: the 32 places about where it
// should be, which hold it but where logits lie close to 0; then by halves.
template <int B>
__device__ unsigned edge_of(const Cut<B> &c, int j, unsigned low, unsigned high) {
    const unsigned lane = threadIdx.x & 31;
    unsigned no = low, yes = high + 1u;  // below `no` it is not, from `yes` on it is
    const unsigned guess = min(max(ord_bits(c.top - __fdividef((float)(j + 1), c.inv)), low), high);
    const unsigned from = guess - min(guess - low, 16u), o = from + lane;
    const unsigned is = __ballot_sync(0xffffffffu, o <= high && c.slot(ord_value(o)) <= j);
    const unsigned in = __ballot_sync(0xffffffffu, o <= high);
    if (is) yes = from + __ffs(is) - 1;
    if (in & ~is) no = from + 32 - __clz(in & ~is);
    while (no < yes) {
        const unsigned m = no + (yes - no) / 2;
        if (c.slot(ord_value(m)) <= j) yes = m;
        else no = m + 1u;
    }
    return yes;
}

// Descending bitonic sort of n keys, K neighbours per thread, exchanged in registers, between lanes by shuffles and
// between warps through two buffers in turn.
template <int K>
__device__ __forceinline__ void sort_keys(u64 (&key)[K], u64 *buf, u64 *other_buf, int n) {
    const int tid = threadIdx.x;
    int pow2 = 32;
    while (pow2 < n) pow2 <<= 1;
    for (int size = 2; size <= pow2; size <<= 1)
        for (int stride = size >> 1; stride > 0; stride >>= 1) {
            if (stride < K) {
#pragma unroll
                for (int s = 1; s < K; s <<= 1) {
                    if (s != stride) continue;
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        if (k & s) continue;
                        const bool down = ((K * tid + k) & size) == 0;
                        const u64 a = key[k], b = key[k | s];
                        const bool swap = (b > a) == down;
                        key[k] = swap ? b : a;
                        key[k | s] = swap ? a : b;
                    }
                }
                continue;
            }
            const int far = stride / K;  // in threads
            const bool greater = ((K * tid & size) == 0) == ((tid & far) == 0);
            if (far >= 32) {
#pragma unroll
                for (int k = 0; k < K; ++k) buf[k * kThreads + tid] = key[k];
                __syncthreads();
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const u64 other = buf[k * kThreads + (tid ^ far)];
                    key[k] = (other > key[k]) == greater ? other : key[k];
                }
                u64 *t = buf;
                buf = other_buf;
                other_buf = t;
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const u64 other = shfl_xor64(key[k], far);
                    key[k] = (other > key[k]) == greater ? other : key[k];
                }
            }
        }
}

// W / S, both up to 2^63, in f32
__device__ __forceinline__ float ratio(u64 W, u64 S) {
    const float w = __ull2float_rz(W), s = __ull2float_rz(S);
    const float wl = (float)(W - (u64)w), sl = (float)(S - (u64)s);
    const float q = w / s;
    return q + (fmaf(-q, s, w) + fmaf(-q, sl, wl)) / s;
}

// Whether a row takes more than the short way (see below).
__device__ __forceinline__ bool takes_long(const SampleArgs &a, int r) {
    const int k = a.top_k ? a.top_k[r] : 0;
    if ((a.temperature && a.temperature[r] == 0.f) || (k > 0 && k <= kMostShort)) return false;
    return k > 0 || !a.min_p || !(a.min_p[r] > 0.f) || (a.top_p && a.top_p[r] < 1.f);
}

// The row of cluster c, the ones that take long first, so that none of them begins when the others are done.  All threads.
template <int B>
__device__ int row_of(const SampleArgs &a, Shared<B> &sh, int c) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int longs = 0;
    for (int r0 = 0; r0 < a.rows; r0 += kThreads) longs += __syncthreads_count(r0 + tid < a.rows && takes_long(a, r0 + tid));
    const bool want = c < longs;
    int left = want ? c : c - longs;
    for (int r0 = 0; r0 < a.rows; r0 += kThreads) {
        const bool is = r0 + tid < a.rows && takes_long(a, r0 + tid) == want;
        const unsigned who = __ballot_sync(0xffffffffu, is);
        if (lane == 0) sh.scan[warp] = __popc(who);
        const int n = __syncthreads_count(is);
        if (left < n) {
            int before = __popc(who & ((1u << lane) - 1u));
            for (int k = 0; k < warp; ++k) before += (int)sh.scan[k];
            if (is && before == left) sh.first[0] = r0 + tid;
            __syncthreads();
            return sh.first[0];
        }
        left -= n;
    }
    return c;
}

template <typename T, bool RES, int B>
__global__ void __launch_bounds__(kThreads, B == kFewBins ? 2 : 1) sample_rows_kernel(const __grid_constant__ SampleArgs a,
                                                                  const __grid_constant__ Table table) {
    extern __shared__ __align__(16) uint8_t smem_sample[];
    Shared<B> &sh = *reinterpret_cast<Shared<B> *>(smem_sample);
    u64 *bins = reinterpret_cast<u64 *>(smem_sample + (sizeof(Shared<B>) + 15) / 16 * 16);
    float *sx = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(bins) + kBinBytes<B>);
    cg::cluster_group cl = cg::this_cluster();
    const unsigned ctas = cl.num_blocks(), me = cl.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (ctas > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    int r = blockIdx.x / ctas;
    if (a.sorted) r = row_of(a, sh, r);

    const float T_ = a.temperature ? a.temperature[r] : 1.f, u = a.u[r];
    const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f;
    const int top_k = a.top_k ? a.top_k[r] : 0;
    const bool greedy = T_ == 0.f;
    const bool valid = greedy || (T_ >= 1e-6f && T_ <= 1e6f && top_p > 0.f && top_p <= 1.f && min_p >= 0.f && min_p <= 1.f &&
                                  u >= 0.f && u < 1.f);
    if (tid < kSteps) sh.table.fix[tid] = table.fix[tid], sh.table.f[tid] = table.f[tid];

    // 1. the row's piece, its greatest and its least logit
    Piece<T, RES> piece;
    piece.src = reinterpret_cast<const T *>(a.logits) + (int64_t)r * a.stride;
    piece.begin = min(a.V, (int)me * a.per);
    piece.end = min(a.V, piece.begin + a.per);
    piece.kept = sx;
    float top = -INFINITY, least = INFINITY;
    {
        constexpr int E = 16 / sizeof(T);
        const T *p = piece.src + piece.begin;
        const int n = piece.end - piece.begin;
        const int head = min(n, (int)((16u - (unsigned)((uintptr_t)p & 15u)) & 15u) / (int)sizeof(T));
        const int vecs = (n - head) / E;
        auto take = [&](int i, float v) {
            const float x = canonical(v);
            if constexpr (RES) sx[i] = x;
            top = fmaxf(top, x);
            least = x > -INFINITY ? fminf(least, x) : least;
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
        if constexpr (RES)
            if (tid < 3 && n + tid < (n + 3) / 4 * 4) sx[n + tid] = -INFINITY;
    }
    float group = top;  // of `ctas` neighbouring threads: kThreads groups in the cluster
    for (unsigned o = 1; o < ctas; o <<= 1) group = fmaxf(group, __shfl_xor_sync(0xffffffffu, group, o));
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
    }
    if (lane == 0) sh.warp_top[warp] = top, sh.warp_least[warp] = least;
    __syncthreads();
    for (int k = 0; k < kWarps; ++k) {
        top = fmaxf(top, sh.warp_top[k]);
        least = fminf(least, sh.warp_least[k]);
    }
    if (ctas > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster is there
        if (tid < ctas) {
            *cl.map_shared_rank(&sh.top[me], tid) = top;
            *cl.map_shared_rank(&sh.least[me], tid) = least;
        }
        *cl.map_shared_rank(&sh.group[me * (kThreads / ctas) + tid / ctas], tid % ctas) = group;
        cl.sync();
        for (unsigned c = 0; c < ctas; ++c) {
            top = fmaxf(top, sh.top[c]);
            least = fminf(least, sh.least[c]);
        }
    }
    if (ctas == 1) {
        sh.group[tid] = group;
        __syncthreads();
    }
    auto answer = [&](int token, float prob, int kept) {
        a.tokens[r] = token;
        if (a.probs) a.probs[r] = prob;
        if (a.kept) a.kept[r] = kept;
    };
    if (!valid || top == -INFINITY) {
        if (me == 0 && tid == 0) answer(-1, 0.f, 0);
        return;
    }
    if (greedy) {  // the first token with the greatest logit
        if (tid == 0) sh.edge[0] = a.V;
        __syncthreads();
        int id = a.V;
        for (int g = tid; g < piece.quads(); g += kThreads) {
            const float4 v = piece.at(g);
            const int k = v.x == top ? 0 : v.y == top ? 1 : v.z == top ? 2 : v.w == top ? 3 : a.V;
            id = min(id, piece.begin + 4 * g + k);
            if (k < 4) break;
        }
        id = __reduce_min_sync(0xffffffffu, id);
        if (lane == 0 && id < a.V) atomicMin(&sh.edge[0], (unsigned)id);
        __syncthreads();
        if (tid == 0) cl.map_shared_rank(sh.first_id, 0)[me] = (int)sh.edge[0];
        if (ctas > 1) cl.sync();
        else __syncthreads();
        if (me == 0 && tid == 0) {
            for (unsigned c = 0; c < ctas; ++c) id = min(id, sh.first_id[c]);
            answer(id, 1.f, 1);
        }
        return;
    }

    const u64 id_mask = (1ull << a.id_bits) - 1ull;
    Row row;
    row.top = top;
    row.wb = a.wb;
    // log2(e) in two terms, divided by T in two terms
    row.chi = __fdiv_rn(1.44269502f, T_);
    row.clo = __fdiv_rn(__fadd_rn(__fmaf_rn(-row.chi, T_, 1.44269502f), 1.92596299e-8f), T_);
    row.far = !(fabsf(row.top * row.chi) < 60000.f);
    {
        int q[2];
        float2 f;
        split2(row, make_float2(row.top, row.top), q, f);
        row.oct = q[0] >> 5;
    }
    // logits below this are less than min_p of the greatest
    float cut = -FLT_MAX;
    if (min_p > 0.f) {
        if (tid == 0) {
            const double m = (double)row.top + (double)T_ * log((double)min_p);
            float f = (float)m;
            if ((double)f < m) f = nextafterf(f, INFINITY);
            sh.cut = f;
        }
        __syncthreads();
        cut = fmaxf(cut, sh.cut);
    }
    const bool has_p = top_p < 1.f;
    // 2. octaves are no narrower than a few of the greatest logit's last places
    Cut<B> octaves{};
    octaves.by_value = true;
    octaves.top = row.top;
    octaves.inv = 1.f / fmaxf(fmaxf(T_ * (0.69314718f * 16.f / B), fabsf(row.top) * 1e-6f), 1e-30f);
    // The whole row: the tokens with keys from `bottom` on.  Without top_p, what min_p leaves out counts for nothing else; with it
    // the weights that it takes its part of do.
    Zone rows{(u64)ord_bits(fmaxf(least, has_p ? -FLT_MAX : cut)) << a.id_bits, ((u64)ord_bits(row.top) + 1ull) << a.id_bits, {}, {}};

    // 1b. A short way for top_k alone, and for min_p alone: the tokens from some logit on, listed at once.  For min_p that is
    // `cut`; for top_k it is taken from the order of the greatest logits of kThreads parts of the row: if tokens are spread
    // evenly, g of them leave a share of e^(-g / kThreads) of the parts without one.  Aimed at a few more than
    // top_k; where there are fewer after all, or more than fit, the long way is taken.
    const unsigned seg = kList / ctas;  // of the list, for each CTA
    unsigned listed = 0;
    const float floor = fmaxf(least, has_p ? -FLT_MAX : cut);
    if ((top_k > 0 && top_k <= kMostShort) || (top_k <= 0 && !has_p && min_p > 0.f)) {
        float from = floor;
        if (top_k > 0) {
            const float aim = (float)top_k + 3.f * sqrtf((float)top_k) + 8.f;
            const int m = min(kThreads - 1, (int)((float)kThreads * (1.f - __expf(-aim / kThreads))));
            // About the m-th greatest, by halves of the order numbers: a value that m + 1 groups or a few more reach (few where nearly all
            // groups do, as each then stands for many tokens).
            if (warp == 0) {
                float v[kThreads / 32];
#pragma unroll
                for (int i = 0; i < kThreads / 32; ++i) v[i] = sh.group[lane + 32 * i];
                unsigned yes = ord_bits(floor), no = ord_bits(row.top) + 1u;
                while (no - yes > 1u) {
                    const unsigned mid = yes + (no - yes) / 2;
                    const float at = ord_value(mid);
                    int n = 0;
#pragma unroll
                    for (int i = 0; i < kThreads / 32; ++i) n += v[i] >= at ? 1 : 0;
                    n = __reduce_add_sync(0xffffffffu, n);
                    if (n > m) yes = mid;
                    else no = mid;
                    if (n > m && n <= m + 1 + min(m, kThreads - m) / 8) break;
                }
                if (lane == 0) sh.at = ord_value(yes);
            }
        }
        if (tid == 0) sh.listed = 0;
        __syncthreads();
        if (top_k > 0) from = fmaxf(from, sh.at);
        u64 *list = cl.map_shared_rank(bins, 0) + me * seg;
        const int quads = piece.quads();
        for (int g = tid; g < quads; g += kThreads) {
            const float4 v = piece.at(g);
            if (!(fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) >= from)) continue;
            const float x[4] = {v.x, v.y, v.z, v.w};
            for (int k = 0; k < 4; ++k) {
                if (!(x[k] >= from)) continue;
                const unsigned at = atomicAdd(&sh.listed, 1u);
                if (at < seg) list[at] = key_of(x[k], piece.begin + 4 * g + k, a.id_bits);
            }
        }
        __syncthreads();
        if (tid < ctas) cl.map_shared_rank(sh.count, tid)[me] = sh.listed;
        if (ctas > 1) cl.sync();
        else __syncthreads();
        bool fit = true;
        for (unsigned i = 0; i < ctas; ++i) {
            listed += sh.count[i];
            fit &= sh.count[i] <= seg;
        }
        if (!fit || (listed < (unsigned)max(top_k, 0) && from > floor)) listed = 0;
    }

    // The row's way through passes and lists, in one loop so that each of them stands in the code once.
    // stage 0: top_k, by counts.  1: top_p, by weights.  2: the draw.  `seek`: a border is looked for, at which the count or the
    // weight of the tokens down to it reaches goal.
    int stage = top_k > 0 ? 0 : 1, side = 0, turn = 0;
    enum { kOctaves, kNarrow, kMinP, kNone } pass = kOctaves;
    bool seek = false, from_octaves = true;
    float near = -1.f;  // of the octave that was entered: the share of its width above the border; -1: not known; -2: cut by keys
    u64 goal = 0;
    Total whole{}, kept{};
    Zone z = rows;
    Cut<B> c = octaves;
    for (;;) {
        bool all = listed != 0;
        u64 *list = bins;
        unsigned room = kList;
        int n = (int)listed;
        if (all) {  // by the short way
            seek = (unsigned)top_k < listed && top_k > 0;
            whole.n = listed;
        } else {
        if (pass != kNone) {
            if (pass != kNarrow) {
                if (stage == 0) tally<B, false, true>(piece, sh, row, bins, cl, turn, z, c, a.id_bits);
                else tally<B, true, true>(piece, sh, row, bins, cl, turn, z, c, a.id_bits);
            } else {
                if (stage == 0) tally<B, false, false>(piece, sh, row, bins, cl, turn, z, c, a.id_bits);
                else tally<B, true, false>(piece, sh, row, bins, cl, turn, z, c, a.id_bits);
            }
            turn ^= 1;  // a CTA that is ahead writes the other half
            if (pass == kOctaves) {
                if (tid < B) sh.cum[tid] = sh.total[tid];
                __syncthreads();
                whole = kept = rows.inside = sh.cum[B - 1];
                seek = stage == 0 ? (unsigned)top_k < whole.n : has_p;
                goal = stage == 0 ? (u64)top_k : max(1ull, times(top_p, whole.w, true));
                z = rows;
            } else if (pass == kMinP) {
                kept = sh.total[B - 1];
                stage = 2;
            }
            from_octaves = pass != kNarrow;
        }
        if (stage == 2 && pass != kNarrow) {
            seek = from_octaves = true;
            goal = times(u, kept.w, false) + 1ull;
            z = rows;
        }
        if (seek) {  // into the part in which the border is
            const Total *total = from_octaves ? sh.cum : sh.total;
            near = -1.f;
            if (from_octaves) c = octaves;
            Total t = lane < B ? total[lane] : Total{~0ull >> 1, ~0u >> 1, 0u}, before;
            const unsigned there = __ballot_sync(0xffffffffu, (stage == 0 ? (u64)(z.above.n + t.n) : z.above.w + t.w) >= goal);
            const int b = there ? min(__ffs(there) - 1, B - 1) : B - 1;
            before = b ? total[b - 1] : Total{0ull, 0u, 0u};
            t = total[b];
            const bool inner = from_octaves && b > 0 && b < B - 2;
            if (!from_octaves && (!c.by_value || t.n - before.n == z.inside.n)) near = -2.f;
            if (inner && warp == 2) {
                // About where in the octave the border is, if what octaves hold grows by the same factor g^2 from the one above to the
                // one below: 1 + share (g - 1) = g^near.
                auto held = [&](int i) {
                    const Total x = sh.cum[i], y = i ? sh.cum[i - 1] : Total{0ull, 0u, 0u};
                    return stage == 0 ? (float)(x.n - y.n) : (float)(x.w - y.w);
                };
                const float lg = 0.5f * __logf(__fdividef(held(b + 1), held(b - 1))), g = __expf(lg);
                const float share = __fdividef((float)(goal - (stage == 0 ? (u64)before.n : before.w)), held(b));
                near = fabsf(g - 1.f) < 1e-3f ? share : __fdividef(__logf(1.f + share * (g - 1.f)), lg);
                if (lane == 0) sh.near = near >= 0.f && near <= 1.f ? near : -1.f;
            }
            z.inside = Total{t.w - before.w, t.n - before.n, t.low - before.low};
            z.above = Total{z.above.w + before.w, z.above.n + before.n, z.above.low + before.low};
            if (c.by_value) {
                const unsigned low = (unsigned)(z.lo >> a.id_bits), high = (unsigned)((z.end - 1ull) >> a.id_bits);
                if (warp < 2 && (warp ? b < B - 1 : b > 0)) {
                    const unsigned e = edge_of(c, b - 1 + warp, low, high);
                    if (lane == 0) sh.edge[warp] = e;
                }
                __syncthreads();
                if (b > 0) z.end = min(z.end, (u64)sh.edge[0] << a.id_bits);
                if (b < B - 1) z.lo = max(z.lo, (u64)sh.edge[1] << a.id_bits);
                if (inner) near = sh.near;
            } else {
                z.lo += (u64)(B - 1 - b) << c.shift;
                z.end = min(z.end, z.lo + (1ull << c.shift));
            }
            __syncthreads();  // sh.edge and sh.total are read
        }

        // 3. the tokens down to the border, if they are few; 4. else the part about it
        const unsigned down = z.above.n + z.inside.n;
        const bool cut_more = seek && (stage < 2 && z.above.n < 3u * kList / 4 ? down > (unsigned)kShort && z.inside.n > (unsigned)kNear
                                                                              : z.inside.n > (unsigned)kPart);
        all = !cut_more && stage < 2 && down <= (unsigned)kList;
        if (cut_more) {
            // In parts of equal spans of logits while they have places enough between them, then of keys; of keys at once where such
            // a part had all of the tokens.  (Equal logits stop the spans at some 1e-6 of their value, but zeros at 1e-30 only: 8
            // rows of 151,936 of which half are 0 took 614 us.)
            const unsigned low = (unsigned)(z.lo >> a.id_bits), high = (unsigned)((z.end - 1ull) >> a.id_bits);
            const float xl = ord_value(low), xh = ord_value(high), width = xh * (1.f / B) - xl * (1.f / B);
            c.by_value = near > -2.f && high - low > 64u && width > fmaxf(fmaxf(fabsf(xl), fabsf(xh)) * 1e-6f, 1e-30f);
            c.top = xh;
            c.inv = 1.f / width;
            if (near >= 0.f && c.by_value) {  // narrow parts about the place where the border should be
                const float part = width * 0.25f;
                if (part > fmaxf(fabsf(xl), fabsf(xh)) * 1e-6f) c.top = xh - near * B * width + B / 2 * part, c.inv = 1.f / part;
            }
            c.shift = 0;
            if (z.end - z.lo > (u64)B) c.shift = 64 - __clzll((long long)((z.end - z.lo - 1ull) / B));
            pass = kNarrow;
            continue;
        }
        if (!all && !seek) {  // nothing is left out
            stage = stage + 1;
            pass = stage == 1 ? kOctaves : kNone;
            z = rows, c = octaves;
            continue;
        }

        // A list: the tokens of the zone (all: and the ones above it) to the first CTA, or to every one.
        if (!all) list = reinterpret_cast<Parts *>(bins)->list[side], room = kPart;
        side ^= 1;
        if (tid == 0) sh.listed = z.inside.low + (all ? z.above.low : 0u);
        __syncthreads();
        {
            const float xl = ord_value((unsigned)(z.lo >> a.id_bits)),
                        xh = all ? row.top : ord_value((unsigned)((z.end - 1ull) >> a.id_bits));
            const int quads = piece.quads();
            for (int g = tid; g < quads; g += kThreads) {
                const float4 v = piece.at(g);
                const float x[4] = {v.x, v.y, v.z, v.w};
                if (!(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= xl)) continue;
                for (int k = 0; k < 4; ++k) {
                    if (!(x[k] >= xl && x[k] <= xh)) continue;
                    const u64 key = key_of(x[k], piece.begin + 4 * g + k, a.id_bits);
                    if (key < z.lo || (!all && key >= z.end)) continue;
                    const unsigned at = atomicAdd(&sh.listed, 1u);
                    if (at >= room) continue;
                    for (unsigned to = 0; to < (all ? 1u : ctas); ++to) cl.map_shared_rank(list, to)[at] = key;
                }
            }
        }
        if (ctas > 1) cl.sync();
        else __syncthreads();
        n = (int)min(room, z.inside.n + (all ? z.above.n : 0u));
        }
        if (all && me != 0) return;
        auto entry = [&](unsigned i) {  // of the list, which the short way leaves in parts
            if (listed == 0) return list[i];
            unsigned part = 0;
            while (i >= sh.count[part]) i -= sh.count[part++];
            return list[part * seg + i];
        };
        // sorted, with the running sums of their weights; the first CTA is done with its piece of the row
        u64 *runs = all ? reinterpret_cast<u64 *>(sx) : reinterpret_cast<Parts *>(bins)->buf[0];
        u64 *keys = all ? runs + kList : reinterpret_cast<Parts *>(bins)->buf[1];
        if (tid < 3) sh.first[tid] = kList;
        auto order = [&](auto per) {
            constexpr int K = decltype(per)::value;
            u64 key[K], run[K];
#pragma unroll
            for (int k = 0; k < K; ++k) key[k] = K * tid + k < n ? entry(K * tid + k) : 0ull;
            if (K == 1 && n <= kThreads / 4) {  // a key's place is the number of greater ones: four threads count them (a bitonic sort takes 1.2 us more)
                runs[tid] = key[0];
                __syncthreads();
                const int i = tid >> 2;
                const u64 mine = runs[i];
                int place = 0;
                for (int j = tid & 3; j < n; j += 4) place += runs[j] > mine ? 1 : 0;
                place += __shfl_xor_sync(0xffffffffu, place, 1);
                place += __shfl_xor_sync(0xffffffffu, place, 2);
                if (i < n && (tid & 3) == 0) keys[place] = mine;
                __syncthreads();
                key[0] = tid < n ? keys[tid] : 0ull;
            } else {
                sort_keys(key, runs, keys, n);
            }
            u64 sum = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (K * tid + k < n) sum += weigh(row, sh.table, ord_value((uint32_t)(key[k] >> a.id_bits)));
                run[k] = sum;
            }
            u64 upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            if (lane == 31) sh.scan[warp] = upto;
            __syncthreads();
            upto += (all ? 0ull : z.above.w) - sum;
            for (int k = 0; k < warp; ++k) upto += sh.scan[k];
#pragma unroll
            for (int k = 0; k < K; ++k) keys[K * tid + k] = key[k], runs[K * tid + k] = run[k] + upto;
        };
        if (n <= kThreads) order(std::integral_constant<int, 1>());
        else order(std::integral_constant<int, kKeys>());
        __syncthreads();
        // first place for which something holds that holds from there on, n if none
        auto first_of = [&](int slot, auto holds) {
            int at = n;
            for (int i = tid; i < n; i += kThreads)
                if (holds(i)) {
                    at = i;
                    break;
                }
            at = __reduce_min_sync(0xffffffffu, at);
            if (lane == 0 && at < n) atomicMin(&sh.first[slot], at);
            __syncthreads();
            return min(n, sh.first[slot]);
        };
        if (all) {
            u64 Z = whole.w;
            const bool has_k = stage == 0 && seek;
            if (has_k || (unsigned)n == whole.n) {
                if (has_k) n = min(n, top_k);
                Z = runs[n - 1];
            }
            if (has_p) {
                const u64 at_p = times(top_p, Z, true);
                n = min(n, 1 + first_of(0, [&](int i) { return runs[i] >= at_p; }));
                if (min_p > 0.f) n = first_of(1, [&](int i) { return ord_value((uint32_t)(keys[i] >> a.id_bits)) < cut; });
            }
            const u64 S = runs[n - 1], at_u = times(u, S, false) + 1ull;
            const int j = min(n - 1, first_of(2, [&](int i) { return runs[i] >= at_u; }));
            if (tid == 0) answer((int)(id_mask - (keys[j] & id_mask)), ratio(j ? runs[j] - runs[j - 1] : runs[0], S), n);
            return;
        }
        int j = stage == 0 ? (int)(goal - z.above.n) - 1 : first_of(0, [&](int i) { return runs[i] >= goal; });
        j = max(0, min(j, n - 1));
        const u64 at = keys[j], weight = j ? runs[j] - runs[j - 1] : runs[0] - z.above.w;
        const Total to_it{runs[j], z.above.n + (unsigned)j + 1u, 0u};
        __syncthreads();
        if (stage == 2) {
            if (me == 0 && tid == 0) answer((int)(id_mask - (at & id_mask)), ratio(weight, kept.w), (int)kept.n);
            return;
        }
        if (stage == 0) {  // the tokens below top_k count for nothing from here on
            stage = 1;
            rows.lo = at;
            pass = kOctaves;
        } else if (min_p > 0.f) {
            pass = kMinP;
        } else {
            stage = 2;
            kept = to_it;
            pass = kNone;
        }
        z = rows, c = octaves;
        if (pass == kMinP) z.lo = max(at, (u64)ord_bits(cut) << a.id_bits);
    }
}

template <typename T, bool RES, int B>
cudaError_t launch_rows(const SampleArgs &a, const Table &t, int rows, int ctas, size_t smem, cudaStream_t st) {
    cudaError_t e = allow_smem<sample_rows_kernel<T, RES, B>>(227 * 1024);
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
    return cudaLaunchKernelEx(&cfg, sample_rows_kernel<T, RES, B>, a, t);
}

const Table &table() {
    static const Table t = [] {
        Table x;
        for (int i = 0; i < kSteps; ++i) {
            const double v = std::exp2((double)i / kSteps);
            x.fix[i] = (unsigned)std::llround(std::ldexp(v, 31));
            x.f[i] = (float)std::ldexp(v, kMantBits);
        }
        return x;
    }();
    return t;
}

int bits_for(int64_t n) {  // least b with n <= 2^b
    int b = 0;
    while ((1ll << b) < n) ++b;
    return b;
}

template <typename T>
cudaError_t launch_typed(const qw_sample_rows_args &q, cudaStream_t st) {
    auto fixed = [](int bins) {
        return bins == kFewBins ? (sizeof(Shared<kFewBins>) + 15) / 16 * 16 + kBinBytes<kFewBins>
                                : (sizeof(Shared<kManyBins>) + 15) / 16 * 16 + kBinBytes<kManyBins>;
    };
    const size_t most = 227 * 1024, room = most - fixed(kFewBins);
    // As many CTAs for a row as there are SMs to take them, or as hold it with another CTA on the SM.  (Clusters of 16 for up to
    // nine rows took 1.3 us more at 8 x 151,936: what grows with the cluster outweighs the shorter pieces.)
    auto per = [&](int n) { return (int)(((int64_t)q.vocab + n - 1) / n + 7) / 8 * 8; };
    auto ctas_for = [&](int64_t rows) {
        int n = 1;
        while (n < kMaxCluster && per(n) > 4096 && (rows * n * 2 <= 152 || (size_t)per(n) * 4 > room / 2)) n *= 2;
        return n;
    };
    const int ctas = ctas_for(q.n_rows);
    SampleArgs a{};
    a.logits = q.logits;
    a.stride = q.row_stride;
    a.V = q.vocab;
    a.per = per(ctas);
    a.id_bits = bits_for(q.vocab);
    // A thread's tokens fit its bins, whatever the number of rows: the weights' unit, and with it what a row draws, goes by the
    // vocabulary alone.
    a.wb = std::min(62 - a.id_bits, kCountBit - 1 - bits_for((per(ctas_for(INT32_MAX)) + 4 * kThreads - 1) / (4 * kThreads) * 4));
    a.rows = q.n_rows;
    // Worth it for one to eight waves of rows of four or more CTAs (us, mixed settings, with it and without: 48 rows of 151,936 70
    // and 78, 128 139 and 150; 150 of 65,000 92 and 95); more of them, or smaller ones, run better side by side with short ones (512 of
    // 151,936 481 and 462; 1,200 of 32,000 296 and 277).
    const int64_t all = (int64_t)q.n_rows * ctas;
    a.sorted = ctas >= 4 && all > 2 * 152 && all <= 16 * 152;
    a.u = q.u, a.temperature = q.temperature, a.top_p = q.top_p, a.min_p = q.min_p, a.top_k = q.top_k;
    a.tokens = q.tokens, a.kept = q.kept, a.probs = q.probs;
    const bool res = (size_t)a.per * 4 <= room;
    const size_t row = std::max<size_t>(res ? (size_t)a.per * 4 : 0, (size_t)kList * 16);  // lists are sorted where the row was
    if (!res) return launch_rows<T, false, kFewBins>(a, table(), q.n_rows, ctas, fixed(kFewBins) + row, st);
    if (all <= 2 * 152 && fixed(kManyBins) + row <= most)
        return launch_rows<T, true, kManyBins>(a, table(), q.n_rows, ctas, fixed(kManyBins) + row, st);
    return launch_rows<T, true, kFewBins>(a, table(), q.n_rows, ctas, fixed(kFewBins) + row, st);
}

}  // namespace

cudaError_t launch_sample_rows(const qw_sample_rows_args &q, cudaStream_t st) {
    return q.dtype == QW_DT_F32   ? launch_typed<float>(q, st)
           : q.dtype == QW_DT_F16 ? launch_typed<__half>(q, st)
                                  : launch_typed<__nv_bfloat16>(q, st);
}

}  // namespace qw
