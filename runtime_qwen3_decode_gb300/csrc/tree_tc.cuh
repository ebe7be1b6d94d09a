// tree_tc.cuh - attention of drafted-token trees on the tensor cores (16-bit queries), for tree_tc.cu and prefix_tc.cu.
//
// The query rows of a KV head (row r = node r / G, head r % G of its group) fill the 128 MMA
// rows, so the heads of a group and the nodes of a tree share every K and V row.  Per tile of
// 128 positions S = Q K^T (both in shared memory), the masks and the online softmax in the
// log2 domain, O += P V (P in TMEM over its scores, V in shared memory as it is cached: the
// MMA takes it MN-major, so nothing is transposed).  The bound is the cache's bytes: 128 x
// 128 x 128 MMAs, even where most of the 128 rows are empty, take 1024 cycles of a tile whose
// bytes take 3000 (bf16) or 1600 (8 bits) cycles of an SM's share of HBM.
//
// Work: the tiles of all (sequence, KV head, row tile) items in a row, cut into equal shares,
// one per CTA, whatever the lengths (each CTA finds its share from len and count).  An item
// inside one share is finished there; of one that is cut, each CTA writes a partial (O, max,
// sum), and the merge kernel adds them in order.
//
// Warps: 0-7 softmax and epilogue, one query row per lane and two groups of four: the groups
// take the tiles in turn, each with its own scores, maximum, sum and accumulator, so that one
// group's tile overlaps the other's (a single group needed 2800 cycles a tile, 1000 of them
// exponentials); the two are joined at the end of an item.  10 loads (TMA), 11 issues the
// MMAs; for caches that are not bf16 beside bf16 queries, 8, 9 and 12-17 convert, four of
// them K and four V.  bf16 beside bf16: TMA writes K and V tiles straight into swizzled operand
// tiles, three stages each.  Otherwise TMA fills two slots of 16 KB with raw rows for each
// plane, and the converters write the 16-bit operand tiles, double-buffered (one stage of
// two-term tiles of 128 positions; PREFIX has two of 64, see tile_log2 in prefix_tc.cu).  8-bit rows
// become fp16 (code * scale rounded once, 2^-11; bf16 would lose three more bits and cost twice the
// instructions), bf16 queries beside them fp16 after
// division by a power of two per row, so that only elements 2^-14 below the row's largest
// lose bits.  f32 rows become two fp16 terms beside fp16 queries and two bf16 terms beside bf16 ones,
// whose range they keep (one fp16 term took 77 us instead of 96, and made V infinite above 65504).
//
// Measured (device time with the merge; HBM floor): 64 nodes over 32768 bf16 positions 37 us
// (20): HBM while it streams, 5 us until the first tiles arrive, 8 us of last tile and merge.
// 16 sequences of up to 33 nodes over 8-bit caches of up to 4096 58 us (14): the chain softmax,
// product, next scores of each group, 2700 cycles a tile.  64 fp16 nodes over 32768 8-bit
// positions 51 us (11); over f32 ones 98 us (40), bf16 nodes 96 us.
//
// What a row does not see has weight 0, but 0 x NaN is NaN in the product with V: the V
// rows behind the sequence are zeroed, and elements of drafted rows that are not finite are
// replaced by 0 in the operand and added to the rows that do see them at the end.
//
// PREFIX (prefix_tc.cu): a batch whose sequences all see a prefix.  The MMA rows are rows of all sequences, one after the other
// (row = (sequence, node, head of the group)), so an item is a (tile of 128 rows, KV head), and its keys are the prefix's tiles and
// then the own tiles of each sequence that has rows among the 128 (Walk).  The prefix is so read once for 128 rows; a sequence's
// own tile costs the tensor cores what any tile does, though only its rows see it (the others' weights are 0, and warps
// without any of its rows do no softmax), but its bytes are read once and the stream of tiles never stops: with the own parts as
// items of their own, every one of them began with a wait for its queries and ended with an epilogue.  What is not finite in
// an own tile's V must not reach the other sequences' rows as 0 x NaN.  Looking every own tile through for it took twice as
// long as the tile otherwise needs (6,600 cycles instead of 3,100 over long bf16 ones), so a CTA does its share without looking, and where a row's
// accumulator comes out not finite does it all again, with such elements taken out as above (bf16 tiles by warps 8 and 9, which
// zero the rows behind an end in the first pass).
//
// Every wait is bounded (1 s); a CTA whose wait expired says so in its status word and the
// merge kernel then fills every output row with NaN.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "tc.cuh"
#include "tree_attn.h"

namespace qw {
namespace {

using namespace tc;

// cache rows and, behind it, the operands' type where they are converted
enum { SRC_BF16 = 0, SRC_Q8_F16 = 1, SRC_BF16_F16 = 2, SRC_F32_F16 = 3, SRC_F32_BF16 = 4 };

// The loading and the MMA warp sit on the SM sub-partitions of the last row quarters, whose softmax
// warps have nothing to do for small trees.
constexpr int kSoftWarps = 8, kLoadWarp = 10, kMmaWarp = 11, kPlainWarps = 12;
constexpr int kConvWarps = 8;              // warps 8, 9 and 12-17; four convert K and four V
constexpr int kPlaneWarps = kConvWarps / 2, kPlaneThreads = 32 * kPlaneWarps;
// TMEM columns of softmax group g: scores (and P over them) at 128 g, accumulator at 256 + 128 g
constexpr uint32_t kColO = 256;

// TERMS: 16-bit numbers per K or V element, 2 = a number of the operands' type and the one of what it leaves.
// TILE: positions of a tile.
template <int SRC, int D, int TERMS, int TILE>
struct Cfg {
    static constexpr bool kDirect = SRC == SRC_BF16;
    static constexpr bool kBf16 = SRC == SRC_BF16 || SRC == SRC_F32_BF16;  // the operands' type, else fp16
    // A tile's weights are 2^(score - reference + kLift).  The reference follows the maximum only when that has
    // risen by more than kLag (rescaling an accumulator costs a pass over it), so weights end below
    // 2^(kLag + kLift).  fp16 drops what is below 2^-25: lifted by 9, that is 2^-34 of the reference, and a
    // long tail of small weights is not lost (unlifted, 2^17 of them that were together 0.34% of the
    // whole counted for half of that).  A lag of 4 and a lift of 11 took 58.3 us for the 16-sequence case below
    // instead of 57.4, 8 and 7 56.7.  bf16 has f32's range.
    static constexpr float kLag = kBf16 ? 8.f : 6.f, kLift = kBf16 ? 0.f : 9.f;
    // PREFIX: sums of softmax weights are of the rounded ones, so that the result is a mean and what a large weight is off by does
    // not move it (16 rows over 200 keys: up to 1.43 times as far off as one rounding of the result leaves them, else
    // 1.77).  bf16 results beside fp16 weights (8-bit rows) do not show it.
    static constexpr bool kSumRounded = !(SRC == SRC_Q8_F16 && TERMS == 1);
    static constexpr int kElem = SRC == SRC_Q8_F16 ? 1 : SRC == SRC_F32_F16 || SRC == SRC_F32_BF16 ? 4 : 2;
    static constexpr int kThreads = 32 * (kDirect ? kPlainWarps : kPlainWarps + kConvWarps - 2);
    static constexpr int kTile = TILE;
    static constexpr int kQRegion = kTcRows * 128;         // 128 rows x 64 16-bit dims
    static constexpr int kRegion = kTile * 128;            // the same of a K or V operand tile
    static constexpr int kTerm = kRegion * (D / 64);       // one term of it
    static constexpr int kOperand = kTerm * TERMS;
    static constexpr int kStages = kDirect ? 3 : kTile * TERMS > 128 ? 1 : 2;
    static constexpr int kChunkRows = 16384 / (D * kElem) < kTile ? 16384 / (D * kElem) : kTile;
    static constexpr int kChunk = kChunkRows * D * kElem;  // raw bytes per ring slot
    static constexpr int kChunks = kTile / kChunkRows;       // per tile and plane
    static constexpr int kRing = kDirect ? 0 : 4;          // slots of raw rows: two for K, two for V
    static constexpr int kQ = 0, kK = kQ + kQRegion * (D / 64), kV = kK + kStages * kOperand, kRaw = kV + kStages * kOperand;
    static constexpr int kBar = kRaw + kRing * kChunk;
    static constexpr int kBytes = kBar + 512 + kTcRows * 4 + 256;  // barriers, one score factor per row, PREFIX: own tiles
    static constexpr size_t kSmem = 1024 + kBytes;
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
    static_assert(!kDirect || TERMS == 1, "tiles that TMA writes have one term");
};

template <bool PREFIX>
struct TcParams {
    AttnArgs<PREFIX> a;
    int n_seq, rows_max;  // rows_max: query rows per partial slot (a multiple of 4)
    int *status;
    float *part;          // [2 CTAs][D + 2][rows_max]
    long long *starts;    // PREFIX: [row tiles + 2] tiles of a KV head before each tile of rows, and 0; or its first CTA, and 1
    int tile_log2;        // PREFIX: of the positions of a tile
    unsigned long long inv_g;  // 2^32 / G + 1: row / G for the at most 4096 rows of a KV head
    __device__ __forceinline__ int node_of(int row) const { return (int)((unsigned)row * inv_g >> 32); }
    // The sequence, node and head of its group of row r: of KV head's rows of sequence b, or (PREFIX) of all sequences.
    __device__ __forceinline__ void place(int r, int &b, int &node, int &g) const {
        if constexpr (PREFIX) {
            b = (int)((unsigned)r * a.inv_rows >> 32);
            r -= b * a.n_max * a.G;
        }
        node = node_of(r);
        g = r - node * a.G;
    }
};
using Tree = TcParams<false>;
using Prefix = TcParams<true>;

__device__ __forceinline__ int seq_tiles(int total) { return (total + kTcTile - 1) / kTcTile; }
__device__ __forceinline__ int seq_tiles(const Prefix &p, int total) { return (total + (1 << p.tile_log2) - 1) >> p.tile_log2; }

// Tiles of sequence b over all its items; 0 for one without nodes or that does not fit.
__device__ __forceinline__ long long seq_work(const Tree &p, int b) {
    int len, n;
    if (!lengths(p.a, b, len, n) || n == 0) return 0;
    const int nrt = (n * p.a.G + kTcRows - 1) / kTcRows;
    return (long long)seq_tiles(len + n) * p.a.Hkv * nrt;
}

// A CTA's share is tiles [T c / C, T (c + 1) / C).
__device__ __forceinline__ long long share_start(long long T, int c, int C) {
    return T < (1 << 24) ? (long long)((unsigned)T * (unsigned)c / (unsigned)C) : T * c / C;  // C <= 152
}

struct Cursor {
    int b, h, rt, tile;
    long long left;
    int first_rt, own_tile;  // PREFIX: of the table of tiles; where in sequence b's own tiles the first segment begins
    int plen;                // PREFIX: the prefix's length
};

struct Seg {
    int b, h, r0, rows;      // rows: of the whole (sequence, KV head); this tile starts at r0
    int t0, t1, tiles;
    int len, n, total;       // PREFIX: len = the prefix's
    int b1, own_tile;        // PREFIX: b .. b1 have rows in the tile; where in b's own tiles it begins, -1: at the first ones
};

__device__ __forceinline__ bool next_seg(const Tree &p, Cursor &c, Seg &s) {
    while (c.left > 0 && c.b < p.n_seq) {
        int len, n;
        if (!lengths(p.a, c.b, len, n) || n == 0) {
            ++c.b;
            continue;
        }
        const int nrt = (n * p.a.G + kTcRows - 1) / kTcRows;
        s.b = c.b, s.h = c.h, s.r0 = c.rt * kTcRows, s.rows = n * p.a.G;
        s.len = len, s.n = n, s.total = len + n;
        s.tiles = seq_tiles(s.total);
        s.t0 = c.tile;
        s.t1 = (int)min((long long)s.tiles, c.tile + c.left);
        c.left -= s.t1 - s.t0;
        c.tile = 0;
        if (++c.rt == nrt) {
            c.rt = 0;
            if (++c.h == p.a.Hkv) {
                c.h = 0;
                ++c.b;
            }
        }
        return true;
    }
    return false;
}

// One whole warp: sum of seq_work over [0, n), and where the running sum passes `at`.
__device__ long long total_work(const Tree &p, int n) {
    const int lane = threadIdx.x & 31;
    long long w = 0;
    for (int b = lane; b < n; b += 32) w += seq_work(p, b);
#pragma unroll
    for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    return w;
}

__device__ Cursor find_start(const Tree &p, long long at, long long left) {
    const int lane = threadIdx.x & 31;
    Cursor c{p.n_seq, 0, 0, 0, left, 0, 0, 0};
    long long before = 0;
    for (int b0 = 0; b0 < p.n_seq; b0 += 32) {
        const long long own = b0 + lane < p.n_seq ? seq_work(p, b0 + lane) : 0;
        long long upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + upto > at);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const long long rest = at - before - (__shfl_sync(0xffffffffu, upto, l) - __shfl_sync(0xffffffffu, own, l));
            c.b = b0 + l;
            int len, n;
            lengths(p.a, c.b, len, n);
            const int tiles = seq_tiles(len + n), nrt = (n * p.a.G + kTcRows - 1) / kTcRows;
            // rest is below one sequence's tiles: 2^31 / 128 positions x 1024 heads x 32 row tiles
            const unsigned long long item = rest < (1ll << 32) ? (unsigned)rest / (unsigned)tiles : rest / tiles;
            c.tile = (int)(rest - (long long)item * tiles);
            c.h = (int)(item / (unsigned)nrt);
            c.rt = (int)(item - (unsigned long long)c.h * nrt);
            return c;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    c.left = 0;
    return c;
}

// ---- PREFIX: tiles of 128 rows of all sequences

constexpr int kOwnTable = 64;  // row tiles whose own tiles a CTA keeps at hand; more than a share has, but for rows without keys

__device__ __forceinline__ int own_tiles(const Prefix &p, int b) {
    int len, n;
    return lengths(p.a, b, len, n) && n > 0 ? seq_tiles(p, len + n) : 0;
}
__device__ __forceinline__ int row_count(const Prefix &p) { return p.n_seq * p.a.n_max * p.a.G; }
__device__ __forceinline__ int row_tiles(const Prefix &p) { return (row_count(p) + kTcRows - 1) / kTcRows; }
// Sequences with rows in row tile rt.
__device__ __forceinline__ void sequences(const Prefix &p, int rt, int &b0, int &b1) {
    b0 = (int)((unsigned)(rt * kTcRows) * p.a.inv_rows >> 32);
    b1 = (int)((unsigned)(min((rt + 1) * kTcRows, row_count(p)) - 1) * p.a.inv_rows >> 32);
}

__device__ __forceinline__ bool next_seg(const Prefix &p, Cursor &c, Seg &s, const unsigned *own) {
    const int nrt = row_tiles(p);
    while (c.left > 0 && c.rt < nrt) {
        s.len = c.plen;
        sequences(p, c.rt, s.b, s.b1);
        unsigned mine = 0;
        if (c.rt - c.first_rt < kOwnTable) mine = own[c.rt - c.first_rt];
        else
            for (int b = s.b; b <= s.b1; ++b) mine += own_tiles(p, b);
        s.tiles = seq_tiles(p, s.len) + (int)mine;
        if (s.tiles == 0) {
            ++c.rt;
            continue;
        }
        s.h = c.h, s.r0 = c.rt * kTcRows, s.rows = row_count(p), s.n = 64;
        s.t0 = c.tile;
        s.t1 = (int)min((long long)s.tiles, c.tile + c.left);
        s.own_tile = c.own_tile;
        if (s.own_tile >= 0) s.b = c.b;
        c.left -= s.t1 - s.t0;
        c.tile = 0;
        c.own_tile = -1;
        if (++c.h == p.a.Hkv) {
            c.h = 0;
            ++c.rt;
        }
        return true;
    }
    return false;
}
__device__ __forceinline__ bool next_seg(const Tree &p, Cursor &c, Seg &s, const unsigned *) { return next_seg(p, c, s); }

// Tables in shared memory that nothing else uses yet: tiles of every row tile's sequences [2^20 / 128], and of the sequences
// themselves while they are few.
constexpr int kRowTilesMax = (1 << 20) / kTcRows, kSeqTable = 4096;
struct Tables {
    unsigned rows[kRowTilesMax];
    int seq[kSeqTable];
};

__device__ __forceinline__ int tiles_of(const Prefix &p, const Tables &t, int b) {
    return p.n_seq <= kSeqTable ? t.seq[b] : own_tiles(p, b);
}

// All warps.
__device__ __forceinline__ void own_tables(const Prefix &p, Tables &t) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (p.n_seq <= kSeqTable) {
        for (int b = threadIdx.x; b < p.n_seq; b += blockDim.x) t.seq[b] = own_tiles(p, b);
        __syncthreads();
    }
    for (int rt = warp; rt < row_tiles(p); rt += warps) {
        int b0, b1;
        sequences(p, rt, b0, b1);
        unsigned w = 0;
        for (int b = b0 + lane; b <= b1; b += 32) w += tiles_of(p, t, b);
        w = __reduce_add_sync(0xffffffffu, w);
        if (lane == 0) t.rows[rt] = w;
    }
}

__device__ __forceinline__ long long scan64(long long v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// The part of the table that this CTA needs, and where in whose own tiles its first segment begins.
__device__ __forceinline__ void find_own(const Prefix &p, const Tables &t, unsigned *own, Cursor &c, int ptiles, int lane) {
    const int nrt = row_tiles(p);
    for (int i = lane; i < kOwnTable; i += 32) own[i] = c.rt + i < nrt ? t.rows[c.rt + i] : 0u;
    if (c.rt < nrt && c.tile > ptiles) {  // inside the sequences' own tiles: whose
        int b0, b1, at_tile = c.tile - ptiles;
        sequences(p, c.rt, b0, b1);
        for (; b0 <= b1; b0 += 32) {
            const int mine = b0 + lane <= b1 ? tiles_of(p, t, b0 + lane) : 0;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, upto > at_tile);
            if (hit) {
                const int l = __ffs(hit) - 1;
                c.b = b0 + l;
                c.own_tile = at_tile - (__shfl_sync(0xffffffffu, upto, l) - __shfl_sync(0xffffffffu, mine, l));
                break;
            }
            at_tile -= __shfl_sync(0xffffffffu, upto, 31);
        }
    }
}

// One whole warp: where this CTA's share begins, and the part of the table that it needs.  CTA 0 leaves the row tiles' starts
// for the merge.  plen: the prefix's length, negative if it does not fit.
__device__ __forceinline__ Cursor find_start(const Prefix &p, const Tables &t, unsigned *own, int plen) {
    const int lane = threadIdx.x & 31, nrt = row_tiles(p);
    Cursor c{0, 0, nrt, 0, 0, 0, -1, plen};
    if (plen < 0) {
        if (blockIdx.x == 0)
            for (int i = lane; i <= nrt + 1; i += 32) p.starts[i] = 0;
        return c;
    }
    const int ptiles = seq_tiles(p, plen);
    long long T = 0;
    for (int r0 = 0; r0 < nrt; r0 += 32) {
        const long long mine = r0 + lane < nrt ? (long long)ptiles + t.rows[r0 + lane] : 0, upto = scan64(mine, lane);
        if (blockIdx.x == 0 && r0 + lane < nrt) p.starts[r0 + lane] = T + upto - mine;
        T += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (blockIdx.x == 0 && lane == 0) p.starts[nrt] = T, p.starts[nrt + 1] = 0;
    T *= p.a.Hkv;
    const int C = (int)gridDim.x;
    if (nrt * p.a.Hkv * 2 <= C && T > 0 && T < (1ll << 24)) {  // 32-bit products
        // Few items: each to CTAs of its own if that makes no share longer than two tiles more.  A CTA whose share spans two items ends
        // one with an epilogue and waits for the next one's queries, which is some 5 us.
        const unsigned fair = (unsigned)((T + C - 1) / C), size = fair + (unsigned)lane;
        unsigned need = 0;
        for (int rt = 0; rt < nrt; ++rt) need += (unsigned)p.a.Hkv * ((ptiles + t.rows[rt] + size - 1u) / size);
        const unsigned fit = __ballot_sync(0xffffffffu, need <= (unsigned)C);
        if (fit & 7u) {
            const unsigned longest = fair + (unsigned)__ffs(fit) - 1u;
            int base = 0;
            for (int rt = 0; rt < nrt; ++rt) {
                const unsigned tiles = ptiles + t.rows[rt];
                const int k = (int)((tiles + longest - 1u) / longest), at = (int)blockIdx.x - base;
                if (blockIdx.x == 0 && lane == 0) p.starts[rt] = base;
                if (at >= 0 && at < p.a.Hkv * k) {
                    const int j = at % k;
                    c.rt = c.first_rt = rt;
                    c.h = at / k;
                    c.tile = (int)(tiles * (unsigned)j / (unsigned)k);
                    c.left = (int)(tiles * (unsigned)(j + 1) / (unsigned)k) - c.tile;
                }
                base += p.a.Hkv * k;
            }
            if (blockIdx.x == 0 && lane == 0) p.starts[nrt] = base, p.starts[nrt + 1] = 1;
            find_own(p, t, own, c, ptiles, lane);
            return c;
        }
    }
    const long long at = share_start(T, blockIdx.x, gridDim.x);
    c.left = share_start(T, blockIdx.x + 1, gridDim.x) - at;
    long long before = 0;
    for (int r0 = 0; r0 < nrt && c.left > 0; r0 += 32) {
        const long long mine = r0 + lane < nrt ? ((long long)ptiles + t.rows[r0 + lane]) * p.a.Hkv : 0, upto = scan64(mine, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, before + upto > at);
        if (hit) {
            const int l = __ffs(hit) - 1;
            c.rt = c.first_rt = r0 + l;
            const long long tiles = (long long)ptiles + t.rows[c.rt];
            const long long rest = at - before - (__shfl_sync(0xffffffffu, upto, l) - __shfl_sync(0xffffffffu, mine, l));
            c.h = (int)(T < (1ll << 32) ? (unsigned)rest / (unsigned)tiles : rest / tiles);  // a 64-bit division takes 0.2 us
            c.tile = (int)(rest - c.h * tiles);
            break;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    find_own(p, t, own, c, ptiles, lane);
    return c;
}

// The tiles of a segment, one after the other: positions pos .. pos + 127 of a plane, of which [len, end) are drafted rows.
template <bool PREFIX>
struct Walk;

template <>
struct Walk<false> {
    int b, pos, len, end;
    static constexpr bool pre = false;
    __device__ __forceinline__ void start(const Tree &, const Seg &s) { b = s.b, pos = s.t0 * kTcTile, len = s.len, end = s.total; }
    __device__ __forceinline__ void next(const Tree &) { pos += kTcTile; }
};

// The prefix's tiles (pre), then those of each sequence.  The next sequence's lengths are on their way while the tiles of one
// are worked on.
template <>
struct Walk<true> {
    int b, pos, len, end, b1, next_len, next_n;
    bool pre;
    __device__ __forceinline__ void look(const Prefix &p) {  // at the sequence behind b: loads whose values nothing needs yet
        const int i = min(b + 1, b1);
        next_len = p.a.len[i];
        next_n = p.a.count ? p.a.count[i] : p.a.n_max;
    }
    __device__ __forceinline__ void step(const Prefix &p) {  // to the next sequence with rows
        int n;
        bool is;
        do {
            ++b;
            len = next_len, n = next_n;
            look(p);
            is = n > 0 && n <= p.a.n_max && len >= 0 && len <= p.a.max_ctx - n;
        } while (!is && b < b1);
        pre = false, pos = 0, end = len + n;
    }
    __device__ __forceinline__ void start(const Prefix &p, const Seg &s) {
        b1 = s.b1;
        pre = s.t0 < seq_tiles(p, s.len);
        b = s.b - 1;
        look(p);
        if (pre) {
            pos = s.t0 << p.tile_log2, len = end = s.len;
            return;
        }
        step(p);
        if (s.own_tile > 0) pos = s.own_tile << p.tile_log2;
    }
    __device__ __forceinline__ void next(const Prefix &p) {
        const int tile = 1 << p.tile_log2;
        if (pos + tile < end) pos += tile;
        else step(p);
    }
};

__device__ __forceinline__ uint8_t *smem_base() {
    extern __shared__ __align__(1024) uint8_t smem_tree[];
    const uint32_t off = (1024u - (su32(smem_tree) & 1023u)) & 1023u;
    return smem_tree + off;
}

// The whole warp waits, bounded, with one verdict: every lane tests the barrier (one instruction for the
// warp; a lane that waits for the others and a shuffle took 300 cycles of a tile's 3000 each time).
__device__ __forceinline__ bool warp_wait(uint64_t *b, unsigned parity, volatile int *abort) {
    if (__all_sync(0xffffffffu, mbar_test(b, parity))) return true;
    return __all_sync(0xffffffffu, mbar_sleep(b, parity, abort, true, kWaitLimitNs));
}

// 2^x on the special-function unit (ex2.approx: about 2 ulp; 2^-inf = +0).
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The columns of a 32-column block that a row sees, one bit each: drafted index `off` of its first
// column; earlier positions are cached ones, which every row sees.
__device__ __forceinline__ uint32_t visible(unsigned long long mask, int off) {
    return off <= -32 ? 0xffffffffu
           : off >= 64 ? 0u
           : off >= 0 ? (uint32_t)(mask >> off)
                      : (uint32_t)(mask << -off) | ((1u << -off) - 1u);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Two packed weights added to a pair of f32 sums (by unpacking them, fp16 ones take 8% of a call; the mixed addition takes 1%,
// but of bf16 ones, which are f32's upper halves, a percent more than that).
template <bool BF16>
__device__ __forceinline__ void add2(float2 &l, uint32_t p) {
    if constexpr (BF16)
        l = __fadd2_rn(l, make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u)));
    else
        asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tadd.rn.f32.f16 %0, a, %0;\n\tadd.rn.f32.f16 %1, b, %1;}" : "+f"(l.x), "+f"(l.y) : "r"(p));
}

// Two packed weights times a power of two.
template <bool BF16>
__device__ __forceinline__ uint32_t scale2(uint32_t p, float f) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&p), __float2bfloat162_rn(f));
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&p), __float2half2_rn(f));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Zeroes the elements of eight packed 16-bit values that are not finite; true if there were any.
template <bool BF16>
__device__ __forceinline__ bool only_finite(uint4 &u) {
    constexpr uint32_t E = BF16 ? 0x7f80u : 0x7c00u;
    uint32_t *w = reinterpret_cast<uint32_t *>(&u);
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & E) == E) w[i] &= 0xffff0000u, any = true;
        if ((w[i] & (E << 16)) == (E << 16)) w[i] &= 0x0000ffffu, any = true;
    }
    return any;
}

// Eight int8 codes times an fp16 scale, each rounded once to fp16, and what that leaves (it has
// eight bits: exact where it is not subnormal).  Byte u = code + 128 beside 0x64 is the fp16
// number 1024 + u.
template <int TERMS>
__device__ __forceinline__ void widen_q8(uint32_t c0, uint32_t c1, __half2 s2, uint4 &o, uint4 &rest) {
    const __half2 off = __float2half2_rn(1152.f);
    uint32_t *ow = reinterpret_cast<uint32_t *>(&o), *rw = reinterpret_cast<uint32_t *>(&rest);
    const uint32_t in[2] = {c0 ^ 0x80808080u, c1 ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = __byte_perm(in[i >> 1], 0x64646464u, (i & 1) ? 0x4342u : 0x4140u);
        const __half2 c = __hsub2(*reinterpret_cast<const __half2 *>(&b), off), h = __hmul2(c, s2);
        ow[i] = *reinterpret_cast<const uint32_t *>(&h);
        if constexpr (TERMS == 2) {
            const __half2 r = __hfma2(c, s2, __hneg2(h));
            rw[i] = *reinterpret_cast<const uint32_t *>(&r);
        }
    }
}

// Two f32 as fp16 pairs, and what the rounding left.
__device__ __forceinline__ uint32_t rest2(float a, float b, uint32_t hi) {
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return pack2<false>(a - h.x, b - h.y);
}

// Two f32 as two bf16 terms each: the first cut, so that what is finite stays finite, the second the rest
// rounded; together they are off by 2^-16 at most.  Beside an infinity the rest, inf - inf, is made finite.
__device__ __forceinline__ uint32_t cut2(float a, float b) {
    uint32_t d;
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}
__device__ __forceinline__ uint32_t cut_rest2(float a, float b, uint32_t hi) {
    const float ha = __uint_as_float(hi << 16), hb = __uint_as_float(hi & 0xffff0000u);
    return pack2<true>(fmaxf(a - ha, -1e38f), fmaxf(b - hb, -1e38f));
}

// Whether one of eight fp16 numbers is infinite (or both of a pair's are NaN).
__device__ __forceinline__ bool any_infinite(const uint4 &o) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&o);
    const __half2 top = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
    return !__hbne2(top, __half2half2(__ushort_as_half(0x7c00)));
}

// Second terms beside infinite first ones become 0, so that the two together are that infinity and not NaN.
__device__ __forceinline__ void drop_rest(const uint8_t *first, uint8_t *rest) {
    const __half *h = reinterpret_cast<const __half *>(first);
#pragma unroll 1
    for (int i = 0; i < 8; ++i)
        if (__hisinf(h[i])) reinterpret_cast<uint16_t *>(rest)[i] = 0;
}

// Raw cache elements e .. e + 7 of a row as the operand holds them, for the fix-up of values that
// are not finite.
template <int SRC>
__device__ __forceinline__ float operand_value(const TreeArgs &a, const uint8_t *plane, const __half *scales, int64_t row,
                                               int64_t srow, int d) {
    if constexpr (SRC == SRC_Q8_F16)
        return __half2float(__float2half_rn((float)reinterpret_cast<const int8_t *>(plane)[row + d] *
                                            __half2float(scales[srow + d / kQGroup])));
    else if constexpr (SRC == SRC_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(plane)[row + d]);
    else if constexpr (SRC == SRC_BF16_F16)
        return __half2float(__float2half_rn(__bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(plane)[row + d])));
    else if constexpr (SRC == SRC_F32_BF16) return reinterpret_cast<const float *>(plane)[row + d];
    else return __half2float(__float2half_rn(reinterpret_cast<const float *>(plane)[row + d]));
}

// Tensor maps of K and V; PREFIX: then of the prefix's.
template <bool PREFIX>
struct Maps {
    CUtensorMap m[PREFIX ? 4 : 2];
};

template <int SRC, int D, int TERMS, bool PREFIX, int TILE>
__global__ void __launch_bounds__(Cfg<SRC, D, TERMS, TILE>::kThreads, 1)
    tree_tc_kernel(const __grid_constant__ Maps<PREFIX> maps, const TcParams<PREFIX> p) {
    using C = Cfg<SRC, D, TERMS, TILE>;
    constexpr int ST = C::kStages;
    uint8_t *base = smem_base();
    uint8_t *sQ = base + C::kQ, *sK = base + C::kK, *sV = base + C::kV, *raw = base + C::kRaw;
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + C::kBar);
    uint64_t *q_full = bars, *k_full = bars + 1, *k_empty = bars + 4, *v_full = bars + 7, *v_empty = bars + 10,
             *s_full = bars + 13, *p_full = bars + 15, *pv_done = bars + 17, *joined = bars + 19, *drain = bars + 20,
             *r_full = bars + 21, *r_empty = bars + 25;
    Cursor *start = reinterpret_cast<Cursor *>(bars + 32);
    int *bad_seg = reinterpret_cast<int *>(bars + 40);  // [4]: 1 + the segment that last set it
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + 42);
    volatile int *abort = reinterpret_cast<volatile int *>(tslot + 1);
    volatile int *redo = abort + 1;  // PREFIX: a row of the first pass is not finite
    float *row_scale = reinterpret_cast<float *>(base + C::kBar + 512);
    unsigned *own = reinterpret_cast<unsigned *>(base + C::kBar + 512 + kTcRows * 4);  // PREFIX: [kOwnTable]
    uint64_t *v_ready = bars + 21;  // PREFIX, bf16 tiles from TMA (which have no ring): looked through
    const AttnArgs<PREFIX> &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(q_full, kSoftWarps);
        for (int i = 0; i < ST; ++i) {
            mbar_init(&k_full[i], C::kDirect ? 1 : kPlaneWarps);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], C::kDirect ? 1 : kPlaneWarps);
            mbar_init(&v_empty[i], PREFIX && C::kDirect ? 3 : 1);  // the MMAs, and warps 8 and 9 where they look V through
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(joined, kSoftWarps);
        mbar_init(drain, 1);
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(&r_full[i], 1);
            mbar_init(&r_empty[i], kPlaneWarps);
        }
        if (PREFIX && C::kDirect)
            for (int i = 0; i < ST; ++i) mbar_init(&v_ready[i], 2);
        for (int i = 0; i < 4; ++i) bad_seg[i] = 0;
        *abort = 0;
        *redo = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) tmem_alloc(tslot, 512);
    if (warp == kLoadWarp && lane == 0) {
        for (int i = 0; i < (PREFIX ? 4 : 2); ++i) prefetch_map(&maps.m[i]);
    }
    chain_wait();
    if constexpr (PREFIX) {
        Tables &tables = *reinterpret_cast<Tables *>(base);  // in the place of operand tiles
        static_assert(sizeof(Tables) <= C::kBar, "fits over them");
        const int plen = *a.plen;  // on its way while the tables are made
        own_tables(p, tables);
        __syncthreads();
        if (warp == 0) {
            const Cursor c = find_start(p, tables, own, plen >= 0 && plen <= a.p_max ? plen : -1);
            if (lane == 0) *start = c;
        }
        fence_async_shared();  // before copies write there
    } else if (warp == 0) {
        const long long T = total_work(p, p.n_seq);
        const long long at = share_start(T, blockIdx.x, gridDim.x), end = share_start(T, blockIdx.x + 1, gridDim.x);
        const Cursor c = find_start(p, at, end - at);
        if (lane == 0) *start = c;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    chain_release();
    const uint32_t tmem = *tslot;
    Seg s;
    Walk<PREFIX> w;
    bool ok = true;
    // What a role has done so far: tiles (they give the phases of the barriers), segments; PREFIX, bf16: phase of each stage's v_ready
    int it = 0, seg = 0;
    unsigned looked = 0;

#pragma unroll 1
    for (int pass = 0; pass < (PREFIX ? 2 : 1); ++pass) {
    Cursor cur = *start;
    const bool careful_pass = PREFIX && pass > 0;
    const bool look = !PREFIX || careful_pass;  // drafted (PREFIX: and own) rows for what is not finite

    if (warp == kLoadWarp) {
        if (lane == 0) {
            // ---- loads
            if constexpr (C::kDirect) {
                int kp[ST], vp[ST];
                for (int i = 0; i < ST; ++i) kp[i] = vp[i] = -1;
                while (ok && next_seg(p, cur, s, own)) {
                    w.start(p, s);
                    for (int t = s.t0; ok && t < s.t1; ++t, ++it) {
                        if (t > s.t0) w.next(p);
                        const CUtensorMap *m = maps.m + (w.pre ? 2 : 0);
                        const int b = w.pre ? 0 : w.b;
                        const int st = it % ST;
                        const unsigned ph = (unsigned)(it / ST) & 1u;
                        if (!mbar_sleep(&k_empty[st], ph ^ 1u, abort, true, kWaitLimitNs)) {
                            ok = false;
                            break;
                        }
                        mbar_expect_tx(&k_full[st], C::kOperand);
                        for (int r = 0; r < D / 64; ++r)
                            tma_load_4d(sK + st * C::kOperand + r * C::kRegion, m, 64 * r, w.pos, s.h, b, &k_full[st]);
                        kp[st] = (int)ph;
                        if (!mbar_sleep(&v_empty[st], ph ^ 1u, abort, true, kWaitLimitNs)) {
                            ok = false;
                            break;
                        }
                        mbar_expect_tx(&v_full[st], C::kOperand);
                        for (int r = 0; r < D / 64; ++r)
                            tma_load_4d(sV + st * C::kOperand + r * C::kRegion, m + 1, 64 * r, w.pos, s.h, b, &v_full[st]);
                        vp[st] = (int)ph;
                    }
                }
                if (!ok) *abort = 1;
                // no copy may land in shared memory after this CTA has exited, whoever gave up
                for (int i = 0; i < ST; ++i) {
                    if (kp[i] >= 0) mbar_sleep(&k_full[i], (unsigned)kp[i], abort, false, kWaitLimitNs);
                    if (vp[i] >= 0) mbar_sleep(&v_full[i], (unsigned)vp[i], abort, false, kWaitLimitNs);
                }
            } else {
                int rp[4] = {-1, -1, -1, -1};
                int i0 = it;  // chunks per plane of the tiles before; chunk i of a plane goes to the plane's slot i & 1
                while (ok && next_seg(p, cur, s, own)) {
                    w.start(p, s);
                    for (int t = s.t0; ok && t < s.t1; ++t, i0 += C::kChunks) {
                        if (t > s.t0) w.next(p);
                        const CUtensorMap *m = maps.m + (w.pre ? 2 : 0);
                        const int b = w.pre ? 0 : w.b;
                        // All of K first: the scores of this tile are issued before the product of the last one,
                        // which V's operand tile waits for, so a K chunk must not wait behind a V chunk.
                        for (int ch = 0; ch < 2 * C::kChunks; ++ch) {
                            const int plane = ch / C::kChunks, c = ch % C::kChunks, i = i0 + c;
                            const int slot = 2 * plane + (i & 1);
                            const unsigned ph = (unsigned)(i >> 1) & 1u;
                            if (!mbar_sleep(&r_empty[slot], ph ^ 1u, abort, true, kWaitLimitNs)) {
                                ok = false;
                                break;
                            }
                            mbar_expect_tx(&r_full[slot], C::kChunk);
                            tma_load_4d(raw + slot * C::kChunk, m + plane, 0, w.pos + c * C::kChunkRows, s.h, b, &r_full[slot]);
                            rp[slot] = (int)ph;
                        }
                    }
                }
                it = i0;
                if (!ok) *abort = 1;
                for (int i = 0; i < C::kRing; ++i)
                    if (rp[i] >= 0) mbar_sleep(&r_full[i], (unsigned)rp[i], abort, false, kWaitLimitNs);
            }
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            // ---- MMAs.  Tile jj's scores and product belong to softmax group jj & 1.  A group's next scores
            // follow its product at once (they overwrite the weights that the product reads), and
            // what they need is waited for before the weights are: that wait is the one that both groups'
            // time hangs on.  With one stage K of two tiles on cannot be there yet (its chunks come
            // behind V chunks that wait for this product): there S runs one tile ahead.
            constexpr uint32_t idS = idesc_16_f32(128, C::kTile, C::kBf16, false), idO = idesc_16_f32(128, D, C::kBf16, true);
            constexpr int kAhead = ST >= 2 ? 2 : 1;
            // Descriptors of the first tiles; the others differ in the address field (in units of 16 bytes), which
            // the offsets below do not carry out of: building each anew held the issue back.
            const uint64_t dQ = desc_sw128(su32(sQ)), dK = desc_sw128(su32(sK)), dV = desc_sw128_mn(su32(sV), C::kRegion);
            auto wait_k = [&](int jn) {
                return mbar_sleep(&k_full[jn % ST], (unsigned)(jn / ST) & 1u, abort, true, kWaitLimitNs);
            };
            auto scores = [&](int jn) {
                const int st = jn % ST;
                tc_fence_after();
                const uint64_t kd = dK + (unsigned)(st * (C::kOperand >> 4));
#pragma unroll
                for (int k = 0; k < TERMS * (D / 16); ++k) {
                    const int term = k / (D / 16), kk = k % (D / 16);
                    const unsigned step = 2u * (kk & 3);
                    mma_f16(tmem + 128u * (jn & 1), dQ + ((kk >> 2) * (C::kQRegion >> 4) + step),
                            kd + ((kk >> 2) * (C::kRegion >> 4) + step + term * (C::kTerm >> 4)), idS, k != 0);
                }
                mma_commit(&s_full[jn & 1]);
                mma_commit(&k_empty[st]);
            };
            while (ok && next_seg(p, cur, s, own)) {
                const int nt = s.t1 - s.t0;
                ok = mbar_sleep(q_full, (unsigned)seg & 1u, abort, true, kWaitLimitNs);
                for (int j = 0; ok && j < min(nt, kAhead); ++j) {
                    ok = wait_k(it + j);
                    if (ok) scores(it + j);
                }
                for (int j = 0; ok && j < nt; ++j) {
                    const int jj = it + j, st = jj % ST;
                    const bool more = j + kAhead < nt;
                    if (kAhead == 1 && more) {
                        ok = wait_k(jj + 1);
                        if (ok) scores(jj + 1);
                    }
                    if (!ok || (kAhead == 2 && more && !wait_k(jj + 2)) ||
                        !mbar_sleep(&v_full[st], (unsigned)(jj / ST) & 1u, abort, true, kWaitLimitNs) ||
                        !mbar_sleep(&p_full[jj & 1], (unsigned)(jj >> 1) & 1u, abort, true, kWaitLimitNs)) {
                        ok = false;
                        break;
                    }
                    if constexpr (PREFIX && C::kDirect) {
                        if (s.t0 + j >= s.len / kTcTile) {  // not a whole tile of the prefix
                            if (!mbar_sleep(&v_ready[st], looked >> st & 1u, abort, true, kWaitLimitNs)) {
                                ok = false;
                                break;
                            }
                            looked ^= 1u << st;
                        }
                    }
                    tc_fence_after();
                    const uint64_t vd = dV + (unsigned)(st * (C::kOperand >> 4));
                    const uint32_t tp = tmem + 128u * (jj & 1);
#pragma unroll
                    for (int k = 0; k < TERMS * (C::kTile / 16); ++k) {
                        const int term = k / (C::kTile / 16), kk = k % (C::kTile / 16);
                        mma_f16_ts(tp + kColO, tp + 8u * kk, vd + (unsigned)(term * (C::kTerm >> 4) + 128 * kk), idO,
                                   j > 1 || k > 0);
                    }
                    mma_commit(&pv_done[jj & 1]);
                    mma_commit(&v_empty[st]);
                    if (kAhead == 2 && more) scores(jj + 2);
                }
                it += nt;
                ++seg;
            }
            if (!ok) *abort = 1;
            mma_commit(drain);  // every MMA completes before TMEM is released
            mbar_sleep(drain, (unsigned)pass & 1u, abort, false, kWaitLimitNs);
        }
    } else if (warp < kSoftWarps) {
        // ---- softmax and epilogue: group grp, TMEM lane quarter q, one query row per lane
        const int grp = warp >> 2, q = warp & 3, r = 32 * q + lane;
        const uint32_t lb = (uint32_t)(32 * q) << 16;
        const uint32_t tS = tmem + lb + 128u * grp, tO = tmem + kColO + lb + 128u * grp;
        while (ok && next_seg(p, cur, s, own)) {
            const int row = s.r0 + r, nt = s.t1 - s.t0, nr = min(kTcRows, s.rows - s.r0);
            bool live = r < nr;
            const bool warp_live = 32 * q < nr;
            int mb_ = s.b, node = 0, head = 0, nodes = s.n;  // this row's sequence, node, query head; its sequence's nodes
            unsigned long long mask = 0ull;
            if (live) {
                p.place(row, mb_, node, head);
                if constexpr (PREFIX) {
                    int len;
                    live = lengths(a, mb_, len, nodes) && node < nodes;
                }
                if (!live) nodes = 64;
                if (live) mask = PREFIX ? node_mask(a, mb_, node) : a.mask[(int64_t)mb_ * a.n_max + node];
            }
            head += s.h * a.G;
            int own_lo = 0, own_hi = 0;  // PREFIX: positions of this row's own sequence in the segment
            // Q into its swizzled tile: D / 8 lanes per row, the eight warps take the live rows in turn, all
            // copies in flight at once.  Then, in place: bf16 queries to fp16 (the row divided by 2^e, 2^e <=
            // amax < 2^(e + 1)), a negative scale flips the signs, a scale of 0 makes them 0.
            {
                constexpr int LPR = D / 8, RPP = 8 * 32 / LPR;  // lanes per row; rows per pass of all warps
                const int c = lane % LPR, first = warp * (32 / LPR) + lane / LPR;
                const bool scaled = !C::kBf16 && a.dtype == QW_DT_BF16;
                const uint16_t *qb = reinterpret_cast<const uint16_t *>(a.q) + (int64_t)s.h * a.G * a.qhead + 8 * c;
                uint8_t *tile = sQ + (c >> 3) * C::kQRegion;
                for (int x = first; x < nr; x += RPP) {
                    int b = s.b, nd, g;
                    p.place(s.r0 + x, b, nd, g);
                    copy16(tile + swz128(x, c & 7), qb + b * a.qseq + nd * a.qnode + g * a.qhead);
                }
                wait_copies();
                if (scaled || a.scale_log2 <= 0.f) {
                    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
                    for (int x0 = first - lane / LPR; x0 < nr; x0 += RPP) {  // whole warps: x0 is the warp's first row
                        const int x = x0 + lane / LPR;
                        uint4 *at = reinterpret_cast<uint4 *>(tile + swz128(x, c & 7));
                        uint4 u = x < nr ? *at : make_uint4(0u, 0u, 0u, 0u);
                        uint32_t *w = reinterpret_cast<uint32_t *>(&u);
                        if (scaled) {
                            float f[8], amax = 0.f, up = 1.f, down = 1.f;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[k]));
                                f[2 * k] = v.x;
                                f[2 * k + 1] = v.y;
                                amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
                            }
#pragma unroll
                            for (int o = LPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                            if (amax > 0.f && amax < INFINITY) {
                                const int e = min(max((int)((__float_as_uint(amax) >> 23) & 255u) - 127, -126), 126);
                                up = __uint_as_float((uint32_t)(127 - e) << 23);
                                down = __uint_as_float((uint32_t)(127 + e) << 23);
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k) w[k] = pack2<false>(f[2 * k] * up, f[2 * k + 1] * up);
                            if (c == 0 && x < nr) row_scale[x] = down;
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k] = a.scale_log2 == 0.f ? 0u : w[k] ^ flip;
                        if (x < nr) *at = u;
                    }
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
                if (!warp_wait(q_full, (unsigned)seg & 1u, abort)) {
                    ok = false;
                    break;
                }
            }
            if (nodes < 64) mask &= (1ull << nodes) - 1ull;
            const bool scaled_row = !C::kBf16 && a.dtype == QW_DT_BF16 && live;
            // not below the least normal number: times 0 a hidden score (-inf) would be NaN, and the seen ones of such a row are 0
            // beside it all the same
            const float sc = a.scale_log2 == 0.f ? 1.f : fmaxf(fabsf(a.scale_log2) * (scaled_row ? row_scale[r] : 1.f), FLT_MIN);
            float m_used = -INFINITY, l = 0.f;
            int mine = 0;  // tiles of this segment that this group has done
            w.start(p, s);
            int walked = 0;
            for (int j = (it & 1) == grp ? 0 : 1; ok && j < nt; j += 2, ++mine) {
                if constexpr (PREFIX) {
                    for (; walked <= j; ++walked) {
                        if (walked > 0) w.next(p);
                        if (!w.pre && w.b == mb_) {
                            if (own_hi == 0) own_lo = w.pos;
                            own_hi = min(w.pos + C::kTile, w.end);
                        }
                    }
                } else {
                    w.pos = (s.t0 + j) * kTcTile;
                }
                const int jj = it + j;
                const unsigned par = (unsigned)(jj >> 1) & 1u;
                if (!warp_wait(&s_full[grp], par, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();  // the group's last product was issued before these scores: it is done too
                const int first = w.pos;
                // rows of other sequences see nothing of a sequence's own tile
                const bool sees = !PREFIX || w.pre || w.b == mb_;
                const bool tail = first + C::kTile > w.len;
                const unsigned long long seen = PREFIX && w.pre ? 0ull : mask;
                // blocks of 32 columns up to the end (a sequence's last tile may hold few)
                const int blocks = PREFIX ? min(C::kTile / 32, (w.end - first + 31) >> 5) : 4;
                bool busy = warp_live;
                if constexpr (PREFIX) busy = __any_sync(0xffffffffu, live && sees);
                if (PREFIX && warp_live && !busy) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) pk[i] = 0u;
#pragma unroll 1
                    for (int c = 0; c < C::kTile / 32; ++c) tmem_st16u(tS + 16u * c, pk);
                }
                if constexpr (PREFIX) {
                    if (busy) {
                        // One pass, 32 columns at a time, each with the reference that the ones before it left: the reference follows the
                        // maximum only when that has risen by more than kLag, which it seldom does behind a row's first tiles,
                        // and then the accumulator and the tile's weights so far are scaled by a power of two.  (With a pass for the
                        // maximum first, as below, 64 sequences of 64 rows over 4096 bf16 positions took 189 us instead of 182.)
#pragma unroll 1
                        for (int c = 0; c < blocks; ++c) {
                            const uint32_t vis = tail ? visible(seen, first + 32 * c - w.len) : 0xffffffffu;
                            float v[32];
                            tmem_ld32(tS + 32u * c, v);
                            float top = -INFINITY;
                            if (vis != 0xffffffffu) {
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] = (vis >> i) & 1u ? v[i] : -INFINITY;
                            }
#pragma unroll
                            for (int i = 0; i < 32; ++i) top = fmaxf(top, v[i]);
                            top = sees ? top * sc : -INFINITY;
                            const bool resc = top > m_used + C::kLag;
                            if (__any_sync(0xffffffffu, resc)) {
                                const float m_new = resc ? ceilf(top) : m_used, factor = resc ? fast_exp2(m_used - m_new) : 1.f;
                                if (mine > 0) {
#pragma unroll 1
                                    for (int k = 0; k < D / 16; ++k) {
                                        uint32_t o[16];
                                        tmem_ld16u(tO + 16u * k, o);
#pragma unroll
                                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
                                        tmem_st16u(tO + 16u * k, o);
                                    }
                                }
#pragma unroll 1
                                for (int k = 0; k < c; ++k) {
                                    uint32_t pk[16];
                                    tmem_ld16u(tS + 16u * k, pk);
#pragma unroll
                                    for (int i = 0; i < 16; ++i) pk[i] = scale2<C::kBf16>(pk[i], factor);
                                    tmem_st16u(tS + 16u * k, pk);
                                }
                                l *= factor;
                                m_used = m_new;
                            }
                            const float mm = m_used == -INFINITY ? 0.f : m_used - C::kLift;  // nothing seen yet: every weight 2^-inf
                            uint32_t pk[16];
                            float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 z = __ffma2_rn(make_float2(v[2 * i], v[2 * i + 1]), make_float2(sc, sc), make_float2(-mm, -mm));
                                const float2 e = make_float2(sees ? fast_exp2(z.x) : 0.f, sees ? fast_exp2(z.y) : 0.f);
                                pk[i] = pack2<C::kBf16>(e.x, e.y);
                                if constexpr (C::kSumRounded) add2<C::kBf16>(l2, pk[i]);
                                else l2 = __fadd2_rn(l2, e);
                            }
                            l += l2.x + l2.y;
                            tmem_st16u(tS + 16u * c, pk);
                        }
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) pk[i] = 0u;
#pragma unroll 1
                        for (int c = blocks; c < C::kTile / 32; ++c) tmem_st16u(tS + 16u * c, pk);
                    }
                } else if (busy) {
                    // halves of 64 columns, rolled: unrolled over the tile the code outgrows the
                    // instruction cache that all roles share
                    float mb = -INFINITY;
                    if (tail) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t vis = visible(seen, first + 32 * c - w.len);
                            float v[32];
                            tmem_ld32(tS + 32u * c, v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) mb = fmaxf(mb, (vis >> i) & 1u ? v[i] : -INFINITY);
                        }
                    } else if constexpr (!C::kDirect) {  // 18 warps: 96 registers
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            float v[32];
                            tmem_ld32(tS + 32u * c, v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) mb = fmaxf(mb, v[i]);
                        }
                    } else {
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            float v[2][32];
                            tmem_ld64(tS + 64u * c, v);
                            float m1 = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                mb = fmaxf(mb, v[0][i]);
                                m1 = fmaxf(m1, v[1][i]);
                            }
                            mb = fmaxf(mb, m1);
                        }
                    }
                    mb *= sc;
                    const bool resc = mb > m_used + C::kLag;
                    const float m_new = resc ? mb : m_used;
                    const float factor = resc ? fast_exp2(m_used - m_new) : 1.f;
                    if (mine > 0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            float o[32];
                            tmem_ld32(tO + 32u * c, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= factor;
                            tmem_st32(tO + 32u * c, o);
                        }
                    }
                    l *= factor;
                    m_used = m_new;
                    const float mm = m_used == -INFINITY ? 0.f : m_used - C::kLift;  // nothing seen yet: every weight 2^-inf
                    // P over the scores: block c's 16 columns end before block c + 1's scores begin
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t vis = tail ? visible(seen, first + 32 * c - w.len) : 0xffffffffu;
                        float v[32];
                        tmem_ld32(tS + 32u * c, v);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 z = __ffma2_rn(make_float2(v[i], v[i + 1]), make_float2(sc, sc), make_float2(-mm, -mm));
                            v[i] = fast_exp2(z.x);
                            v[i + 1] = fast_exp2(z.y);
                        }
                        if (vis != 0xffffffffu) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = (vis >> i) & 1u ? v[i] : 0.f;
                        }
                        uint32_t pk[16];
                        float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            l2 = __fadd2_rn(l2, make_float2(v[2 * i], v[2 * i + 1]));
                            pk[i] = pack2<C::kBf16>(v[2 * i], v[2 * i + 1]);
                        }
                        l += l2.x + l2.y;
                        tmem_st16u(tS + 16u * c, pk);
                    }
                }
                if constexpr (C::kDirect && !PREFIX) {
                    // the tile's V rows behind the sequence, and what is not finite in the drafted rows: one
                    // position per lane of the four warps
                    if (tail) {
                        const int st = jj % ST;
                        if (!warp_wait(&v_full[st], (unsigned)(jj / ST) & 1u, abort)) {
                            ok = false;
                            break;
                        }
                        const int pos = first + r;
                        bool any = false;
                        if (pos >= s.len) {
                            for (int c = 0; c < D / 8; ++c) {
                                uint4 *w = reinterpret_cast<uint4 *>(sV + st * C::kOperand + (c >> 3) * C::kRegion + swz128(r, c & 7));
                                uint4 u = pos < s.total ? *w : make_uint4(0u, 0u, 0u, 0u);
                                const bool hit = only_finite<true>(u);
                                if (hit || pos >= s.total) *w = u;
                                any |= hit;
                            }
                        }
                        if (any) bad_seg[seg & 3] = seg + 1;
                        fence_async_shared();
                    }
                }
                // A warp without live rows may run ahead, but reaches the group's next scores only
                // after the product that all four warps released.
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[grp]);
            }
            if constexpr (PREFIX) {
                for (; walked < nt; ++walked) {  // the other group's last tile
                    if (walked > 0) w.next(p);
                    if (!w.pre && w.b == mb_) {
                        if (own_hi == 0) own_lo = w.pos;
                        own_hi = min(w.pos + C::kTile, w.end);
                    }
                }
            }
            // the group's last product; the ones before it were done when its scores came
            const int last = it + nt - 1 - ((it + nt - 1) & 1 ^ grp);
            if (ok && mine > 0 && !warp_wait(&pv_done[grp], (unsigned)(last >> 1) & 1u, abort)) ok = false;
            if (ok) {
                // join the groups: (m, l) through the free scores, then each group finishes half of the dims
                tc_fence_after();
                if (warp_live) tmem_st2(tS, m_used, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(joined);
                if (!warp_wait(joined, (unsigned)seg & 1u, abort)) ok = false;
            }
            if (ok && warp_live) {
                tc_fence_after();
                float m_other, l_other;
                tmem_ld2(tmem + lb + 128u * (grp ^ 1), m_other, l_other);
                const float m = fmaxf(m_used, m_other), mm = m == -INFINITY ? 0.f : m;
                const bool other = nt > 1;                   // a group without a tile has no accumulator to read
                const float w_own = mine > 0 ? fast_exp2(m_used - mm) : 0.f;
                const float w_other = mine > 0 ? (other ? fast_exp2(m_other - mm) : 0.f) : fast_exp2(m_other - mm);
                const float lt = l * w_own + l_other * w_other;
                const bool whole = s.t0 == 0 && s.t1 == s.tiles;
                const bool bad = *reinterpret_cast<volatile int *>(&bad_seg[seg & 3]) == seg + 1;
                const float inv = whole ? (lt == 0.f ? 0.f : 1.0f / lt) : 1.f;
                float *part = p.part + (size_t)(2 * blockIdx.x + (s.t0 > 0 ? 0 : 1)) * (D + 2) * p.rows_max + r;
                const int64_t at = mb_ * a.oseq + node * a.onode + head * a.ohead;
#pragma unroll 1
                for (int c = grp * (D / 64); c < (grp + 1) * (D / 64); ++c) {
                    float o[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                    if (mine > 0) {
                        tmem_ld32(tO + 32u * c, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= w_own;
                    }
                    if (mine == 0 || other) {
                        float x[32];
                        tmem_ld32(tmem + kColO + lb + 128u * (grp ^ 1) + 32u * c, x);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = fmaf(x[i], w_other, o[i]);
                    }
                    if (bad && live) {
                        // drafted rows; PREFIX: and cached ones, which all of the sequence's rows see
                        const int len = PREFIX ? a.len[mb_] : s.len;
                        const int j0 = PREFIX ? own_lo : max(s.t0 * kTcTile, len), j1 = PREFIX ? own_hi : min(s.t1 * kTcTile, s.total);
                        for (int jx = j0; jx < j1; ++jx) {
                            if (jx >= len && !((mask >> (jx - len)) & 1ull)) continue;
                            const int64_t vr = mb_ * a.seq + s.h * a.head + (int64_t)jx * a.pos;
                            const int64_t sr = mb_ * a.sseq + s.h * a.shead + (int64_t)jx * a.spos;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float v = operand_value<SRC>(a, a.v, a.vs, vr, sr, 32 * c + i);
                                if (!isfinite(v)) o[i] += v;
                            }
                        }
                    }
                    if (!live) continue;
                    if constexpr (PREFIX) {
                        if (pass == 0 && m != -INFINITY) {  // NaN if one of them is not finite
                            float2 probe = make_float2(0.f, 0.f);
#pragma unroll
                            for (int i = 0; i < 32; i += 2) probe = __ffma2_rn(make_float2(o[i], o[i + 1]), make_float2(0.f, 0.f), probe);
                            if (!(probe.x + probe.y == 0.f)) *redo = 1;
                        }
                    }
                    if (!whole) {
                        if (PREFIX && m == -INFINITY) continue;  // nothing seen: the merge does not look at it
#pragma unroll
                        for (int i = 0; i < 32; ++i) part[(size_t)(32 * c + i) * p.rows_max] = o[i];
                        continue;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = lt == 0.f ? 0.f : o[8 * i + e] * inv;
                        if (a.dtype == QW_DT_F16) store8(reinterpret_cast<__half *>(a.out) + at + 32 * c + 8 * i, w);
                        else store8(reinterpret_cast<__nv_bfloat16 *>(a.out) + at + 32 * c + 8 * i, w);
                    }
                }
                if (!whole && live && grp == 0) {
                    part[(size_t)D * p.rows_max] = m;
                    part[(size_t)(D + 1) * p.rows_max] = lt;
                }
                tc_fence_before();
            }
            it += nt;
            ++seg;
        }
        if (!ok && lane == 0) *abort = 1;
    } else if constexpr (!C::kDirect) {
        // ---- converters: four warps for K, four for V, each with two slots of the ring (a slot that both
        // used would have them wait for every other phase of its barrier, which a parity cannot tell apart)
        const int cw = warp - (warp < kLoadWarp ? kSoftWarps : kSoftWarps + 2);
        const int plane = cw / kPlaneWarps, ct = (cw % kPlaneWarps) * 32 + lane;
        uint64_t *full = plane ? v_full : k_full, *empty = plane ? v_empty : k_empty;
        uint8_t *operand = plane ? sV : sK;
        // Eight elements of position `pos` (o: fp16, rest: second term) into their 16-byte chunk.
        auto put = [&](uint8_t *at, uint4 o, uint4 rest, auto checked, int pos) {
            bool any = false;
            if constexpr (decltype(checked)::value) {  // V rows of the sequence's end
                if (pos >= w.end) {
                    o = rest = make_uint4(0u, 0u, 0u, 0u);
                } else if (look && pos >= (PREFIX ? w.pre ? w.end : 0 : w.len) && only_finite<C::kBf16>(o)) {
                    any = true;
                    only_finite<C::kBf16>(rest);  // not finite where o was not
                }
            }
            *reinterpret_cast<uint4 *>(at) = o;
            if constexpr (TERMS == 2) *reinterpret_cast<uint4 *>(at + C::kTerm) = rest;
            return any;
        };
        // After a chunk: its slot is free, and (done) the plane's operand tile complete.
        auto finish = [&](bool any, int slot, uint64_t *done) {
            if (any) bad_seg[seg & 3] = seg + 1;
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&r_empty[slot]);
                if (done) mbar_arrive(done);
            }
        };
        if constexpr (SRC == SRC_Q8_F16) {
            // A thread takes whole 32-element groups, one scale each: row ct / GPR + RSTEP u, group ct % GPR.
            // Scales are loaded two tiles ahead.  The group's 32 bytes go as two halves; threads of
            // groups 2 and 3 take the second half first, which spreads a warp's 16-byte stores
            // over all banks.
            constexpr int GPR = D / kQGroup, RSTEP = kPlaneThreads / GPR, U = C::kTile / RSTEP;
            static_assert(C::kChunks == 1, "an 8-bit tile is one chunk per plane");
            const int g = ct % GPR, row0 = ct / GPR, flip = g >> 1;
            const __half *scales = plane ? a.vs : a.ks;
            __half sc[2][U];  // this tile's and the next one's
            while (ok && next_seg(p, cur, s, own)) {
                const __half *own_scales = scales + s.b * a.sseq + s.h * a.shead + g;
                auto plane_scales = [&](const Walk<PREFIX> &x, int64_t &stride) {
                    stride = a.spos;
                    if constexpr (PREFIX) {
                        if (x.pre) {
                            stride = a.pspos;
                            return (plane ? a.pvs : a.pks) + s.h * a.pshead + g;
                        }
                        return scales + x.b * a.sseq + s.h * a.shead + g;
                    }
                    return own_scales;
                };
                auto fetch = [&](__half(&x)[U], const Walk<PREFIX> &at) {
                    int64_t stride;
                    const __half *from = plane_scales(at, stride);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int pos = at.pos + row0 + RSTEP * u;
                        x[u] = pos < at.end ? from[(int64_t)pos * stride] : __half(0);
                    }
                };
                w.start(p, s);
                Walk<PREFIX> ahead = w;
                fetch(sc[0], ahead);
                if (s.t0 + 1 < s.t1) {
                    ahead.next(p);
                    fetch(sc[1], ahead);
                }
                for (int t = s.t0; ok && t < s.t1; ++t, ++it) {
                    if (t > s.t0) w.next(p);
                    const int st = it % ST, slot = 2 * plane + (it & 1);
                    const bool check = plane && (w.pos + C::kTile > (PREFIX ? w.end : w.len) || (careful_pass && !w.pre));
                    __half2 s2[U];
                    bool over = false;  // codes times a scale above 65504 / 127 may be infinite
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        s2[u] = __half2half2(sc[0][u]);
                        if constexpr (TERMS == 2) over |= !(__habs(sc[0][u]) <= __float2half_rn(515.f));
                        sc[0][u] = sc[1][u];
                    }
                    if (t + 2 < s.t1) {
                        ahead.next(p);
                        fetch(sc[1], ahead);
                    }
                    if (!warp_wait(&empty[st], ((unsigned)(it / ST) & 1u) ^ 1u, abort) ||
                        !warp_wait(&r_full[slot], (unsigned)(it >> 1) & 1u, abort)) {
                        ok = false;
                        break;
                    }
                    const uint8_t *src = raw + slot * C::kChunk + row0 * D + 32 * g;
                    uint8_t *dst = operand + st * C::kOperand + (g >> 1) * C::kRegion;
                    // every read before the first write: nothing tells the compiler that they do not overlap
                    uint4 x[U][2];
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj)
                            x[u][jj] = *reinterpret_cast<const uint4 *>(src + RSTEP * u * D + 16 * (jj ^ flip));
                    bool any = false;
                    auto all = [&](auto checked) {
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int row = row0 + RSTEP * u;
#pragma unroll
                            for (int jj = 0; jj < 2; ++jj) {
                                const int c = 4 * (g & 1) + 2 * (jj ^ flip);
                                uint4 o, rest = make_uint4(0u, 0u, 0u, 0u);
                                widen_q8<TERMS>(x[u][jj].x, x[u][jj].y, s2[u], o, rest);
                                any |= put(dst + swz128(row, c), o, rest, checked, w.pos + row);
                                widen_q8<TERMS>(x[u][jj].z, x[u][jj].w, s2[u], o, rest);
                                any |= put(dst + swz128(row, c + 1), o, rest, checked, w.pos + row);
                            }
                        }
                    };
                    // A tile with such scales, element chunk by chunk.  It stands apart from the others' code: any check
                    // between their conversion and finish() costs a call of one tile 0.5 of 15 us.
                    auto careful = [&] {
#pragma unroll 1
                        for (int i = 0; i < 2 * U; ++i) {
                            const int row = row0 + RSTEP * (i >> 1), pos = w.pos + row, c = 4 * (g & 1) + 2 * (i & 1);
                            const uint4 y = *reinterpret_cast<const uint4 *>(src + RSTEP * (i >> 1) * D + 16 * (i & 1));
                            int64_t stride;
                            const __half *from = plane_scales(w, stride);
                            const __half2 sv = __half2half2(pos < w.end ? from[(int64_t)pos * stride] : __half(0));
#pragma unroll 1
                            for (int k = 0; k < 2; ++k) {
                                uint4 o, rest = make_uint4(0u, 0u, 0u, 0u);
                                widen_q8<TERMS>(k ? y.z : y.x, k ? y.w : y.y, sv, o, rest);
                                uint8_t *at = dst + swz128(row, c + k);
                                if (check) any |= put(at, o, rest, std::true_type(), pos);
                                else put(at, o, rest, std::false_type(), pos);
                                drop_rest(at, at + C::kTerm);
                            }
                        }
                    };
                    if (TERMS == 2 && over) careful();
                    else if (check) all(std::true_type());
                    else all(std::false_type());
                    finish(any, slot, &full[st]);
                }
                ++seg;
            }
        } else {
            // unit = eight elements of a row; a chunk's units over the plane's threads
            constexpr int UPR = D / 8, U = C::kChunkRows * UPR / kPlaneThreads, RSTEP = kPlaneThreads / UPR;
            static_assert(U * kPlaneThreads == C::kChunkRows * UPR, "whole units per thread");
            const int c = ct % UPR, row0 = ct / UPR;
            while (ok && next_seg(p, cur, s, own)) {
                w.start(p, s);
                for (int t = s.t0; ok && t < s.t1; ++t, ++it) {
                    if (t > s.t0) w.next(p);
                    const int st = it % ST;
                    const bool check = plane && (w.pos + C::kTile > (PREFIX ? w.end : w.len) || (careful_pass && !w.pre));
                    for (int ch = 0; ch < C::kChunks; ++ch) {
                        const int i = it * C::kChunks + ch, slot = 2 * plane + (i & 1), crow = ch * C::kChunkRows;
                        if ((ch == 0 && !warp_wait(&empty[st], ((unsigned)(it / ST) & 1u) ^ 1u, abort)) ||
                            !warp_wait(&r_full[slot], (unsigned)(i >> 1) & 1u, abort)) {
                            ok = false;
                            break;
                        }
                        const uint8_t *src = raw + slot * C::kChunk;
                        uint8_t *dst = operand + st * C::kOperand + (c >> 3) * C::kRegion;
                        using Raw = typename std::conditional<C::kElem == 2, __nv_bfloat16, float>::type;
                        float v[U][8];
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            load8(reinterpret_cast<const Raw *>(src) + (row0 + RSTEP * u) * D + 8 * c, v[u]);
                        bool any = false, over = false;
                        auto all = [&](auto checked) {
#pragma unroll
                            for (int u = 0; u < U; ++u) {
                                const int row = crow + row0 + RSTEP * u;
                                const float *f = v[u];
                                auto first = [](float x, float y) { return C::kBf16 ? cut2(x, y) : pack2<false>(x, y); };
                                const uint4 o = make_uint4(first(f[0], f[1]), first(f[2], f[3]), first(f[4], f[5]),
                                                           first(f[6], f[7]));
                                uint4 rest = make_uint4(0u, 0u, 0u, 0u);
                                if constexpr (C::kBf16) {
                                    rest = make_uint4(cut_rest2(f[0], f[1], o.x), cut_rest2(f[2], f[3], o.y),
                                                      cut_rest2(f[4], f[5], o.z), cut_rest2(f[6], f[7], o.w));
                                } else if constexpr (TERMS == 2) {
                                    rest = make_uint4(rest2(f[0], f[1], o.x), rest2(f[2], f[3], o.y), rest2(f[4], f[5], o.z),
                                                      rest2(f[6], f[7], o.w));
                                    over |= any_infinite(o);
                                }
                                any |= put(dst + swz128(row, c & 7), o, rest, checked, w.pos + row);
                            }
                        };
                        if (check) all(std::true_type());
                        else all(std::false_type());
                        if constexpr (TERMS == 2) {
                            if (over) {
#pragma unroll 1
                                for (int u = 0; u < U; ++u) {
                                    uint8_t *at = dst + swz128(crow + row0 + RSTEP * u, c & 7);
                                    drop_rest(at, at + C::kTerm);
                                }
                            }
                        }
                        finish(any, slot, ch == C::kChunks - 1 ? &full[st] : nullptr);
                    }
                }
                ++seg;
            }
        }
        if (!ok && lane == 0) *abort = 1;
    } else if constexpr (PREFIX) {
        // ---- bf16 tiles that TMA wrote: V rows behind the end are zeroed, and in the second pass what is not finite in a sequence's
        // own rows.  Warps 8 and 9, half of the rows each.
        while (ok && next_seg(p, cur, s, own)) {
            w.start(p, s);
            for (int t = s.t0; ok && t < s.t1; ++t, ++it) {
                if (t > s.t0) w.next(p);
                const int st = it % ST;
                // Every tile is waited for and given back: a parity does not tell this phase of a stage from the one before the last,
                // so the stage must not be filled again while a warp has yet to see that it was.
                if (!warp_wait(&v_full[st], (unsigned)(it / ST) & 1u, abort)) {
                    ok = false;
                    break;
                }
                if (t < s.len / kTcTile) {  // a whole tile of the prefix: every row sees it
                    if (lane == 0) mbar_arrive(&v_empty[st]);
                    continue;
                }
                bool any = false;
                constexpr int CH = D / 8;  // chunks of a row
                // rows alternate between the two warps; TMA has zeroed the ones behind the cache
                const int r1 = min(kTcTile, (w.pre ? a.p_max : a.max_ctx) - w.pos), r0 = careful_pass && !w.pre ? 0 : w.end - w.pos;
                const int sub = lane / CH, c = lane % CH;
                uint8_t *column = sV + st * C::kOperand + (c >> 3) * C::kRegion;
#pragma unroll 4
                for (int row = r0 + (32 / CH) * (warp - kSoftWarps) + sub; row < r1; row += 2 * (32 / CH)) {
                    uint4 *at = reinterpret_cast<uint4 *>(column + swz128(row, c & 7));
                    if (w.pos + row >= w.end) {
                        *at = make_uint4(0u, 0u, 0u, 0u);
                    } else {
                        uint4 u = *at;
                        if (only_finite<true>(u)) *at = u, any = true;
                    }
                }
                if (any) bad_seg[seg & 3] = seg + 1;
                fence_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&v_ready[st]);
                    mbar_arrive(&v_empty[st]);
                }
            }
            ++seg;
        }
        if (!ok && lane == 0) *abort = 1;
    }
    if constexpr (PREFIX) {
        __syncthreads();  // every row of the pass is finished
        if (!*redo || *abort) break;
    }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0) p.status[blockIdx.x] = *abort;
}

constexpr int kMergeThreads = 128;
constexpr int kMergeBatch = 10;

// The partials of one row and four dims (4 dq ..) of an item that CTAs c0 .. c1 had parts of, added in order: num / den.  `total`:
// tiles of all CTAs.  The loads of kMergeBatch partials are in flight at once: the merge is nothing but their latency.
// first, step: which of them (mx is the greatest maximum of those).
template <int D, bool PREFIX>
__device__ __forceinline__ void add_partials(const TcParams<PREFIX> &p, int ctas, long long total, int c0, int c1, int rl, int dq,
                                             float (&num)[4], float &den, float &mx, int first = 0, int step = 1) {
    // c0 holds the item's first tile: its second slot; the later CTAs begin inside the item: their
    // first.  Where there are more CTAs than tiles some shares are empty.
    const size_t slot = (size_t)(D + 2) * p.rows_max;
    const bool gaps = total < ctas;
    auto partial = [&](int c) { return p.part + (size_t)(2 * c + (c == c0 ? 1 : 0)) * slot + rl; };
    auto holds = [&](int c) { return c <= c1 && !(gaps && share_start(total, c, ctas) == share_start(total, c + 1, ctas)); };
    mx = -INFINITY;
    for (int c = c0 + first; c0 < c1 && c <= c1; c += kMergeBatch * step) {
        float m[kMergeBatch], l[kMergeBatch], v[kMergeBatch][4], top = mx;
#pragma unroll
        for (int i = 0; i < kMergeBatch; ++i) {
            const bool is = holds(c + i * step);
            const float *src = partial(c + i * step);
            m[i] = is ? src[(size_t)D * p.rows_max] : -INFINITY;
            l[i] = is ? src[(size_t)(D + 1) * p.rows_max] : 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = is ? src[(size_t)(4 * dq + k) * p.rows_max] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kMergeBatch; ++i) top = fmaxf(top, m[i]);
        const float old = mx == -INFINITY ? 0.f : exp2f(mx - top);
        mx = top;
        den *= old;
#pragma unroll
        for (int k = 0; k < 4; ++k) num[k] *= old;
#pragma unroll
        for (int i = 0; i < kMergeBatch; ++i) {
            if (m[i] == -INFINITY && l[i] == 0.f) continue;  // the share showed the row nothing
            const float w = exp2f(m[i] - mx);
            den += l[i] * w;
#pragma unroll
            for (int k = 0; k < 4; ++k) num[k] += v[i][k] * w;
        }
    }
}

// ---------------------------------------------------------------- host side

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
    static EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return (EncodeFn)f;
    }();
    return fn;
}

// Map of one plane of the cache, [seq][head][pos][dim] with its strides, read in boxes of
// box_rows positions and box_dims elements.
bool plane_map(CUtensorMap *m, const void *ptr, const qw_kv_view &kv, CUtensorMapDataType type, int elem, int box_dims,
               int box_rows, bool swizzle) {
    const EncodeFn enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)kv.head_dim, (cuuint64_t)kv.max_ctx, (cuuint64_t)kv.n_kv_heads, (cuuint64_t)kv.n_seq};
    // the stride of a dimension of one is never used, but has to be valid
    const cuuint64_t row = (cuuint64_t)kv.head_dim * elem;
    const cuuint64_t strides[3] = {kv.max_ctx > 1 ? (cuuint64_t)kv.pos_stride * elem : row,
                                   kv.n_kv_heads > 1 ? (cuuint64_t)kv.head_stride * elem : row,
                                   kv.n_seq > 1 ? (cuuint64_t)kv.seq_stride * elem : row};
    const cuuint32_t box[4] = {(cuuint32_t)box_dims, (cuuint32_t)box_rows, 1, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, type, 4, const_cast<void *>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Few rows lie close together, so that the merge's loads of neighbouring dims share lines (with rows of
// 32 a single node over 4096 8-bit positions took 35 us instead of 21).
int slot_rows(int rows) { return std::min(kTcRows, (rows + 3) / 4 * 4); }

// prefix: PREFIX only.  The merge is the caller's.
template <int SRC, int D, int TERMS, bool PREFIX, int TILE>
cudaError_t launch_src(const TcParams<PREFIX> &p, const qw_kv_view &kv, const qw_kv_view *prefix, int ctas, cudaStream_t st, bool chained) {
    using C = Cfg<SRC, D, TERMS, TILE>;
    Maps<PREFIX> maps;
    const CUtensorMapDataType type = C::kElem == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : C::kElem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const int dims = C::kDirect ? 64 : D, rows = C::kDirect ? kTcTile : C::kChunkRows;
    for (int i = 0; i < (PREFIX ? 4 : 2); ++i) {
        const qw_kv_view &view = i < 2 ? kv : *prefix;
        if (!plane_map(&maps.m[i], i & 1 ? view.v : view.k, view, type, C::kElem, dims, rows, C::kDirect)) return cudaErrorInvalidValue;
    }
    cudaError_t e = allow_smem<tree_tc_kernel<SRC, D, TERMS, PREFIX, TILE>>((int)C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_k(chained, tree_tc_kernel<SRC, D, TERMS, PREFIX, TILE>, dim3(ctas), dim3(C::kThreads), C::kSmem, st, maps, p);
}

// 16-bit results next to fp16 operands: beside bf16 queries one rounding of 8-bit K and V (2^-11) drowns in
// the result's own (2^-8); beside fp16 queries it would be most of the error (rounded scores alone
// left a relative error of 5.5e-4 where the result's rounding leaves 2.1e-4), so K and V
// that fp16 does not hold exactly come as two terms.  bf16 queries over f32 rows: fp16 would lose the range that
// both the rows and the result have, and one bf16 term most of the rows' bits, so two bf16 terms.
template <int D, bool PREFIX>
cudaError_t launch_dim(const TcParams<PREFIX> &p, const qw_kv_view &kv, const qw_kv_view *pre, int ctas, cudaStream_t st, bool ch) {
    const bool f16 = p.a.dtype == QW_DT_F16;
    auto go = [&](auto src, auto terms, auto tile) {
        return launch_src<decltype(src)::value, D, decltype(terms)::value, PREFIX, decltype(tile)::value>(p, kv, pre, ctas, st, ch);
    };
    constexpr std::integral_constant<int, 1> one{};
    constexpr std::integral_constant<int, 2> two{};
    constexpr std::integral_constant<int, kTcTile> whole{};
    constexpr std::integral_constant<int, PREFIX ? 64 : kTcTile> half{};
    if (kv.format == QW_KV_INT8_G32) {
        constexpr std::integral_constant<int, SRC_Q8_F16> src{};
        if constexpr (PREFIX) {
            if (f16 && p.tile_log2 == 6) return go(src, two, half);
        }
        return f16 ? go(src, two, whole) : go(src, one, whole);
    }
    if (kv.format == QW_KV_BF16)
        return f16 ? go(std::integral_constant<int, SRC_BF16_F16>(), one, whole) : go(std::integral_constant<int, SRC_BF16>(), one, whole);
    return f16 ? go(std::integral_constant<int, SRC_F32_F16>(), two, half) : go(std::integral_constant<int, SRC_F32_BF16>(), two, half);
}

}  // namespace
}  // namespace qw
