// ops_api.cu - argument checks of the operators on caller-owned buffers (qw_kv_append,
// qw_kv_read, qw_tree_attention, qw_prefix_attention, qw_process_logits, qw_sample_rows).  Everything is checked before a launch;
// nothing here touches the device.
#include <algorithm>
#include <cmath>

#include "qw.h"
#include "qw_ops.h"

namespace {

int status_of(cudaError_t e) {
    if (e == cudaSuccess) return QW_OK;
    cudaGetLastError();
    return QW_CUDA_ERROR;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

int elem_bytes(int32_t dtype) {
    return dtype == QW_DT_F32 ? 4 : dtype == QW_DT_F16 || dtype == QW_DT_BF16 ? 2 : 0;
}

constexpr int32_t kMostEntries = 1 << 28;  // of a list: a token's count in two of them stays below 2^30, where the flags are

bool stride_ok(int64_t s, int64_t unit) { return s >= 0 && s % unit == 0; }

// Whether two arrays of n 32-bit elements share any (NULL: there is none).
bool arrays_meet(const void *a, const void *b, int64_t n) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && (x < y ? y - x : x - y) < (uintptr_t)n * 4;
}

// Whether rows of `len` elements along three dimensions have addresses of their own: taken from the smallest
// stride up, each one is no shorter than all that the dimensions before it span.
struct Dim {
    int64_t size, stride;
};
bool rows_apart(int64_t len, Dim a, Dim b, Dim c) {
    Dim d[3] = {a, b, c};
    std::sort(d, d + 3, [](const Dim &x, const Dim &y) { return x.stride < y.stride; });
    __int128 span = len;
    for (const Dim &x : d) {
        if (x.size <= 1) continue;
        if (x.stride < span) return false;
        span += (__int128)(x.size - 1) * x.stride;
    }
    return true;
}

// The cache as something that is written: no two of its rows may share an address, nor may its planes.
bool writable(const qw_kv_view *kv) {
    if (kv->k == kv->v || !rows_apart(kv->head_dim, {kv->n_seq, kv->seq_stride}, {kv->n_kv_heads, kv->head_stride},
                                      {kv->max_ctx, kv->pos_stride}))
        return false;
    return kv->format != QW_KV_INT8_G32 ||
           (kv->k_scale != kv->v_scale &&
            rows_apart(kv->head_dim / qw::kQGroup, {kv->n_seq, kv->scale_seq_stride}, {kv->n_kv_heads, kv->scale_head_stride},
                       {kv->max_ctx, kv->scale_pos_stride}));
}

int check_view(const qw_kv_view *kv) {
    if (!kv || !kv->k || !kv->v) return QW_INVALID_ARGUMENT;
    if (kv->format != QW_KV_F32 && kv->format != QW_KV_BF16 && kv->format != QW_KV_INT8_G32) return QW_INVALID_ARGUMENT;
    if (kv->n_seq < 1 || kv->n_kv_heads < 1 || kv->max_ctx < 1) return QW_INVALID_ARGUMENT;
    if (kv->head_dim != 64 && kv->head_dim != 128) return QW_UNSUPPORTED_SHAPE;
    if (kv->n_seq > 65535 || kv->n_kv_heads > 1024) return QW_UNSUPPORTED_SHAPE;
    const int64_t unit = kv->format == QW_KV_F32 ? 4 : kv->format == QW_KV_BF16 ? 8 : 16;  // elements of 16 bytes
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !stride_ok(kv->seq_stride, unit) ||
        !stride_ok(kv->head_stride, unit) || !stride_ok(kv->pos_stride, unit))
        return QW_ALIGNMENT;
    // rows of one dimension do not overlap (those of a cache that is written share no address at all: writable())
    if ((kv->max_ctx > 1 && kv->pos_stride < kv->head_dim) || (kv->n_kv_heads > 1 && kv->head_stride < kv->head_dim) ||
        (kv->n_seq > 1 && kv->seq_stride < kv->head_dim))
        return QW_INVALID_ARGUMENT;
    if (kv->format == QW_KV_INT8_G32) {
        const int64_t g = kv->head_dim / qw::kQGroup;
        if (!kv->k_scale || !kv->v_scale) return QW_INVALID_ARGUMENT;
        if (!aligned(kv->k_scale, 2 * g) || !aligned(kv->v_scale, 2 * g) || !stride_ok(kv->scale_seq_stride, g) ||
            !stride_ok(kv->scale_head_stride, g) || !stride_ok(kv->scale_pos_stride, g))
            return QW_ALIGNMENT;
        if ((kv->max_ctx > 1 && kv->scale_pos_stride < g) || (kv->n_kv_heads > 1 && kv->scale_head_stride < g) ||
            (kv->n_seq > 1 && kv->scale_seq_stride < g))
            return QW_INVALID_ARGUMENT;
    }
    return QW_OK;
}

// written: the rows are the call's output, of which no two may share an address.
int check_rows(const qw_kv_view *kv, const qw_kv_rows *r, const int32_t *start, const int32_t *count, bool written) {
    if (!r || !start || r->n_max < 0) return QW_INVALID_ARGUMENT;
    if (!aligned(start, 4) || !aligned(count, 4)) return QW_ALIGNMENT;
    const int e = elem_bytes(r->dtype);
    if (!e) return QW_INVALID_ARGUMENT;
    if (r->n_max == 0) return QW_OK;
    if ((int64_t)r->n_max * kv->n_kv_heads > (int64_t)1 << 30) return QW_UNSUPPORTED_SHAPE;
    if (!r->k || !r->v) return QW_INVALID_ARGUMENT;
    const int64_t unit = 16 / e;
    if (!aligned(r->k, 16) || !aligned(r->v, 16) || !stride_ok(r->seq_stride, unit) ||
        !stride_ok(r->head_stride, unit) || !stride_ok(r->row_stride, unit))
        return QW_ALIGNMENT;
    if (r->row_stride < kv->head_dim && r->n_max > 1) return QW_INVALID_ARGUMENT;
    if (written && (r->k == r->v || !rows_apart(kv->head_dim, {kv->n_seq, r->seq_stride}, {kv->n_kv_heads, r->head_stride},
                                                {r->n_max, r->row_stride})))
        return QW_INVALID_ARGUMENT;
    return QW_OK;
}

int check_tree_sizes(const qw_kv_view *kv, int32_t n_max, int32_t n_heads, int32_t max_len) {
    if (n_max < 0 || n_heads < 1 || max_len < 0 || max_len > kv->max_ctx) return QW_INVALID_ARGUMENT;
    // 16384 heads: (KV head, row tile) pairs are one dimension of a grid
    if (n_max > QW_TREE_NODES_MAX || n_heads > 16384 || n_heads % kv->n_kv_heads || n_heads / kv->n_kv_heads > 64)
        return QW_UNSUPPORTED_SHAPE;
    return QW_OK;
}

// What the two attentions check of their arguments beside the sizes; masks: they must be given.
int check_attention(const qw_kv_view *kv, const qw_tree_attention_args *a, const void *scratch, bool masks) {
    const int e = elem_bytes(a->dtype);
    if (!a->q || !a->out || (masks && !a->mask) || !scratch) return QW_INVALID_ARGUMENT;
    const int64_t unit = 16 / e;
    if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(scratch, 256) || !stride_ok(a->q_seq_stride, unit) ||
        !stride_ok(a->q_node_stride, unit) || !stride_ok(a->q_head_stride, unit) ||
        !stride_ok(a->out_seq_stride, unit) || !stride_ok(a->out_node_stride, unit) ||
        !stride_ok(a->out_head_stride, unit) || !aligned(a->mask, 8) || !aligned(a->len, 4) || !aligned(a->count, 4))
        return QW_ALIGNMENT;
    // no two rows of the result may share an address
    if (!rows_apart(kv->head_dim, {kv->n_seq, a->out_seq_stride}, {a->n_max, a->out_node_stride},
                    {a->n_heads, a->out_head_stride}))
        return QW_INVALID_ARGUMENT;
    return QW_OK;
}

int check_prefix(const qw_kv_view *prefix, const qw_kv_view *kv, int32_t n_max, int32_t n_heads, int32_t max_len,
                 int32_t max_prefix) {
    int rc = check_view(prefix);
    if (!rc) rc = check_view(kv);
    if (rc) return rc;
    if (prefix->n_seq != 1 || prefix->format != kv->format || prefix->n_kv_heads != kv->n_kv_heads ||
        prefix->head_dim != kv->head_dim || max_prefix < 0 || max_prefix > prefix->max_ctx)
        return QW_INVALID_ARGUMENT;
    rc = check_tree_sizes(kv, n_max, n_heads, max_len);
    if (rc) return rc;
    // the rows that share the prefix are numbered in a word, and divided by what a sequence has of them in another
    if ((int64_t)kv->n_seq * n_max * (n_heads / kv->n_kv_heads) > 1 << 20) return QW_UNSUPPORTED_SHAPE;
    return QW_OK;
}

}  // namespace

extern "C" {

int qw_kv_append(const qw_kv_view *kv, const qw_kv_rows *rows, const int32_t *start_dev, const int32_t *count_dev,
                 void *cuda_stream) {
    int rc = check_view(kv);
    if (!rc) rc = check_rows(kv, rows, start_dev, count_dev, false);
    if (!rc && !writable(kv)) rc = QW_INVALID_ARGUMENT;
    if (rc) return rc;
    return status_of(qw::launch_kv_append(*kv, *rows, start_dev, count_dev, (cudaStream_t)cuda_stream));
}

int qw_kv_read(const qw_kv_view *kv, const qw_kv_rows *rows, const int32_t *start_dev, const int32_t *count_dev,
               void *cuda_stream) {
    int rc = check_view(kv);
    if (!rc) rc = check_rows(kv, rows, start_dev, count_dev, true);
    if (rc) return rc;
    return status_of(qw::launch_kv_read(*kv, *rows, start_dev, count_dev, (cudaStream_t)cuda_stream));
}

size_t qw_tree_attention_scratch_bytes(const qw_kv_view *kv, int32_t n_max, int32_t n_heads, int32_t max_len) {
    if (check_view(kv) || check_tree_sizes(kv, n_max, n_heads, max_len)) return 0;
    return qw::tree_attn_scratch_bytes(kv->n_seq, kv->n_kv_heads, n_max, n_heads, kv->head_dim, max_len);
}

int qw_tree_attention(const qw_kv_view *kv, const qw_tree_attention_args *a, void *scratch_dev, size_t scratch_bytes,
                      void *cuda_stream) {
    int rc = check_view(kv);
    if (rc) return rc;
    if (!a) return QW_INVALID_ARGUMENT;
    rc = check_tree_sizes(kv, a->n_max, a->n_heads, a->max_len);
    if (rc) return rc;
    const int e = elem_bytes(a->dtype);
    if (!e || !a->len || !std::isfinite(a->scale)) return QW_INVALID_ARGUMENT;
    if (a->n_max == 0) return QW_OK;
    rc = check_attention(kv, a, scratch_dev, true);
    if (rc) return rc;
    if (scratch_bytes < qw_tree_attention_scratch_bytes(kv, a->n_max, a->n_heads, a->max_len)) return QW_OUT_OF_MEMORY;
    return status_of(qw::launch_tree_attn(*kv, *a, scratch_dev, (cudaStream_t)cuda_stream));
}

size_t qw_prefix_attention_scratch_bytes(const qw_kv_view *prefix, const qw_kv_view *kv, int32_t n_max, int32_t n_heads,
                                         int32_t max_len, int32_t max_prefix) {
    if (check_prefix(prefix, kv, n_max, n_heads, max_len, max_prefix) || n_max == 0) return 0;
    return qw::prefix_attn_scratch_bytes(*kv, n_max, n_heads, max_len, max_prefix);
}

int qw_prefix_attention(const qw_kv_view *prefix, const qw_kv_view *kv, const qw_tree_attention_args *a,
                        const int32_t *prefix_len_dev, int32_t max_prefix, void *scratch_dev, size_t scratch_bytes,
                        void *cuda_stream) {
    if (!prefix || !kv || !a) return QW_INVALID_ARGUMENT;
    int rc = check_prefix(prefix, kv, a->n_max, a->n_heads, a->max_len, max_prefix);
    if (rc) return rc;
    if (!elem_bytes(a->dtype) || !a->len || !prefix_len_dev || !std::isfinite(a->scale)) return QW_INVALID_ARGUMENT;
    if (!aligned(prefix_len_dev, 4)) return QW_ALIGNMENT;
    if (a->n_max == 0) return QW_OK;
    rc = check_attention(kv, a, scratch_dev, false);
    if (rc) return rc;
    const size_t need = qw::prefix_attn_scratch_bytes(*kv, a->n_max, a->n_heads, a->max_len, max_prefix);
    if (need == 0) return QW_UNSUPPORTED_SHAPE;
    if (scratch_bytes < need) return QW_OUT_OF_MEMORY;
    if (a->q == a->out) return QW_INVALID_ARGUMENT;  // rows are read again where a result was not finite
    return status_of(qw::launch_prefix_attn(*prefix, *kv, *a, prefix_len_dev, max_prefix, scratch_dev, (cudaStream_t)cuda_stream));
}

int qw_process_logits(const qw_process_logits_args *a, void *cuda_stream) {
    if (!a || !elem_bytes(a->dtype) || a->n_rows < 0 || a->vocab < 1 || a->vocab > (1 << 24)) return QW_INVALID_ARGUMENT;
    if (a->n_rows == 0) return QW_OK;
    if (!a->logits || !a->out || a->row_stride < 0 || a->out_row_stride < (a->n_rows > 1 ? a->vocab : 0))
        return QW_INVALID_ARGUMENT;
    if (a->n_rows > 65535) return QW_UNSUPPORTED_SHAPE;
    const int e = elem_bytes(a->dtype);
    if (!aligned(a->logits, e) || !aligned(a->out, e)) return QW_ALIGNMENT;
    for (const void *p : {(const void *)a->penalties, (const void *)a->history, (const void *)a->history_range,
                          (const void *)a->path, (const void *)a->bias_ids, (const void *)a->bias,
                          (const void *)a->bias_range, (const void *)a->mask, (const void *)a->mask_index})
        if (!aligned(p, 4)) return QW_ALIGNMENT;
    if (a->out == a->logits && a->row_stride != a->out_row_stride && a->n_rows > 1) return QW_INVALID_ARGUMENT;
    if (a->n_history < 0 || a->path_len < 0 || a->n_bias < 0 || a->n_masks < 0) return QW_INVALID_ARGUMENT;
    if (a->n_history > kMostEntries || a->path_len > kMostEntries || a->n_bias > kMostEntries) return QW_UNSUPPORTED_SHAPE;
    if (a->history && !a->history_range) return QW_INVALID_ARGUMENT;
    if ((a->bias || a->bias_ids) && !(a->bias && a->bias_ids && a->bias_range)) return QW_INVALID_ARGUMENT;
    return status_of(qw::launch_process_logits(*a, (cudaStream_t)cuda_stream));
}

int qw_sample_rows(const qw_sample_rows_args *a, void *cuda_stream) {
    if (!a || !elem_bytes(a->dtype) || a->n_rows < 0 || a->vocab < 1 || a->vocab > (1 << 24)) return QW_INVALID_ARGUMENT;
    if (a->n_rows == 0) return QW_OK;
    if (!a->logits || !a->u || !a->tokens || a->row_stride < 0) return QW_INVALID_ARGUMENT;
    if (a->n_rows > 65535) return QW_UNSUPPORTED_SHAPE;
    if (!aligned(a->logits, elem_bytes(a->dtype))) return QW_ALIGNMENT;
    for (const void *p : {(const void *)a->u, (const void *)a->temperature, (const void *)a->top_k, (const void *)a->top_p,
                          (const void *)a->min_p, (const void *)a->tokens, (const void *)a->probs, (const void *)a->kept})
        if (!aligned(p, 4)) return QW_ALIGNMENT;
    // a row is answered while others have yet to read every row's settings: which of them take long
    const void *const in[] = {a->temperature, a->top_k, a->top_p, a->min_p}, *const out[] = {a->tokens, a->probs, a->kept};
    for (int i = 0; i < 3; ++i) {
        for (const void *p : in)
            if (arrays_meet(out[i], p, a->n_rows)) return QW_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (arrays_meet(out[i], out[j], a->n_rows)) return QW_INVALID_ARGUMENT;
    }
    return status_of(qw::launch_sample_rows(*a, (cudaStream_t)cuda_stream));
}

}  // extern "C"
