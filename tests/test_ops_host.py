"""Refusals of the operators on caller-owned buffers (qw_kv_append, qw_kv_read, qw_tree_attention,
qw_process_logits): checked before the device is touched, so these run without a GPU."""
import ctypes

import numpy as np
import pytest

P = 0x7F0000000000  # an aligned address that is never read


@pytest.fixture(scope="module")
def qw():
    from runtime_qwen3_decode_gb300 import build, qw as binding
    build.build()
    return binding


def view(qw, **kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, format=qw.KV_INT8_G32, n_seq=2, n_kv_heads=8, head_dim=128, max_ctx=64,
             seq_stride=8 * 64 * 128, head_stride=64 * 128, pos_stride=128, scale_seq_stride=8 * 64 * 4,
             scale_head_stride=64 * 4, scale_pos_stride=4)
    d.update(kw)
    return qw.KvViewStruct(**d)


def rows(qw, **kw):
    d = dict(k=P, v=P, dtype=qw.DT_F32, n_max=4, seq_stride=8 * 4 * 128, head_stride=4 * 128, row_stride=128)
    d.update(kw)
    return qw.KvRowsStruct(**d)


BAD_VIEWS = [
    (dict(k=None), "INVALID_ARGUMENT"), (dict(v=None), "INVALID_ARGUMENT"), (dict(k_scale=None), "INVALID_ARGUMENT"),
    (dict(v_scale=None), "INVALID_ARGUMENT"), (dict(format=3), "INVALID_ARGUMENT"), (dict(format=-1), "INVALID_ARGUMENT"),
    (dict(n_seq=0), "INVALID_ARGUMENT"), (dict(n_kv_heads=0), "INVALID_ARGUMENT"), (dict(max_ctx=0), "INVALID_ARGUMENT"),
    (dict(head_dim=96), "UNSUPPORTED_SHAPE"), (dict(head_dim=256), "UNSUPPORTED_SHAPE"),
    (dict(n_seq=65536), "UNSUPPORTED_SHAPE"), (dict(k=P + 8), "ALIGNMENT"), (dict(v=P + 1), "ALIGNMENT"),
    (dict(pos_stride=136), "ALIGNMENT"), (dict(head_stride=8), "ALIGNMENT"), (dict(seq_stride=-16), "ALIGNMENT"),
    (dict(pos_stride=64), "INVALID_ARGUMENT"), (dict(head_stride=0), "INVALID_ARGUMENT"), (dict(seq_stride=64), "INVALID_ARGUMENT"),
    (dict(scale_head_stride=0), "INVALID_ARGUMENT"), (dict(k_scale=P + 4), "ALIGNMENT"), (dict(scale_pos_stride=6), "ALIGNMENT"),
    (dict(scale_pos_stride=0), "INVALID_ARGUMENT"),
]


@pytest.mark.parametrize("bad,code", BAD_VIEWS)
def test_view_refusals(qw, bad, code):
    v, r = view(qw, **bad), rows(qw)
    for call in (qw.lib().qw_kv_append, qw.lib().qw_kv_read):
        assert call(ctypes.byref(v), ctypes.byref(r), P, None, None) == getattr(qw, code)
    assert qw.lib().qw_tree_attention_scratch_bytes(ctypes.byref(v), 4, 16, 60) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(k=None), "INVALID_ARGUMENT"), (dict(dtype=3), "INVALID_ARGUMENT"),
    (dict(n_max=-1), "INVALID_ARGUMENT"), (dict(v=P + 4), "ALIGNMENT"), (dict(row_stride=130), "ALIGNMENT"),
    (dict(row_stride=64), "INVALID_ARGUMENT"), (dict(head_stride=2), "ALIGNMENT")])
def test_rows_refusals(qw, bad, code):
    v, r = view(qw), rows(qw, **bad)
    for call in (qw.lib().qw_kv_append, qw.lib().qw_kv_read):
        assert call(ctypes.byref(v), ctypes.byref(r), P, None, None) == getattr(qw, code)
        assert call(ctypes.byref(v), ctypes.byref(rows(qw)), None, None, None) == qw.INVALID_ARGUMENT
        assert call(None, ctypes.byref(rows(qw)), P, None, None) == qw.INVALID_ARGUMENT
        assert call(ctypes.byref(v), None, P, None, None) == qw.INVALID_ARGUMENT


def tree_args(qw, **kw):
    d = dict(q=P, out=P, dtype=qw.DT_BF16, n_max=4, n_heads=16, max_len=60, scale=0.1, q_seq_stride=4 * 16 * 128,
             q_node_stride=16 * 128, q_head_stride=128, out_seq_stride=4 * 16 * 128, out_node_stride=16 * 128,
             out_head_stride=128, mask=P, len=P, count=None)
    d.update(kw)
    return qw.TreeAttentionArgs(**d)


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), "INVALID_ARGUMENT"), (dict(out=None), "INVALID_ARGUMENT"), (dict(mask=None), "INVALID_ARGUMENT"),
    (dict(len=None), "INVALID_ARGUMENT"), (dict(dtype=4), "INVALID_ARGUMENT"), (dict(dtype=3), "INVALID_ARGUMENT"),
    (dict(n_max=-1), "INVALID_ARGUMENT"), (dict(n_max=65), "UNSUPPORTED_SHAPE"), (dict(n_heads=12), "UNSUPPORTED_SHAPE"),
    (dict(n_heads=0), "INVALID_ARGUMENT"), (dict(n_heads=8 * 65), "UNSUPPORTED_SHAPE"), (dict(n_heads=16392), "UNSUPPORTED_SHAPE"), (dict(max_len=-1), "INVALID_ARGUMENT"),
    (dict(max_len=65), "INVALID_ARGUMENT"), (dict(scale=float("nan")), "INVALID_ARGUMENT"), (dict(q=P + 8), "ALIGNMENT"),
    (dict(out=P + 2), "ALIGNMENT"), (dict(q_head_stride=130), "ALIGNMENT"), (dict(out_node_stride=4), "ALIGNMENT")])
def test_tree_refusals(qw, bad, code):
    v, a = view(qw), tree_args(qw, **bad)
    assert qw.lib().qw_tree_attention(ctypes.byref(v), ctypes.byref(a), P, 1 << 40, None) == getattr(qw, code)


def test_tree_scratch_refusals(qw):
    v, a = view(qw), tree_args(qw)
    n = qw.lib().qw_tree_attention_scratch_bytes(ctypes.byref(v), 4, 16, 60)
    assert n > 0
    call = qw.lib().qw_tree_attention
    assert call(ctypes.byref(v), ctypes.byref(a), P, n - 1, None) == qw.OUT_OF_MEMORY
    assert call(ctypes.byref(v), ctypes.byref(a), P + 16, n, None) == qw.ALIGNMENT
    assert call(ctypes.byref(v), ctypes.byref(a), None, n, None) == qw.INVALID_ARGUMENT
    assert call(ctypes.byref(v), None, P, n, None) == qw.INVALID_ARGUMENT
    assert call(None, ctypes.byref(a), P, n, None) == qw.INVALID_ARGUMENT


def test_tree_scratch_of_a_bound_covers_shorter_lengths(qw):
    # a workspace made for the longest cache serves every shorter max_len
    for ctx in (1, 63, 64, 65, 1000, 40000):
        v = view(qw, max_ctx=ctx, head_stride=ctx * 128, seq_stride=8 * ctx * 128)
        sizes = [qw.lib().qw_tree_attention_scratch_bytes(ctypes.byref(v), 9, 16, m) for m in range(0, ctx + 1, max(1, ctx // 50))]
        assert sizes == sorted(sizes)


def logits_args(qw, **kw):
    d = dict(logits=P, out=P, dtype=qw.DT_F32, n_rows=3, vocab=1001, row_stride=1001, out_row_stride=1001, penalties=P,
             history=P, history_range=P, n_history=5, path=P, path_len=2, bias_ids=P, bias=P, bias_range=P, n_bias=4,
             mask=P, mask_index=P, n_masks=1)
    d.update(kw)
    return qw.ProcessLogitsArgs(**d)


@pytest.mark.parametrize("bad,code", [
    (dict(logits=None), "INVALID_ARGUMENT"), (dict(out=None), "INVALID_ARGUMENT"), (dict(dtype=3), "INVALID_ARGUMENT"),
    (dict(n_rows=-1), "INVALID_ARGUMENT"), (dict(vocab=0), "INVALID_ARGUMENT"), (dict(vocab=(1 << 24) + 1), "INVALID_ARGUMENT"),
    (dict(n_rows=65536), "UNSUPPORTED_SHAPE"), (dict(logits=P + 2), "ALIGNMENT"), (dict(out=P + 1), "ALIGNMENT"),
    (dict(out_row_stride=1000), "INVALID_ARGUMENT"), (dict(row_stride=-1), "INVALID_ARGUMENT"),
    (dict(row_stride=1024), "INVALID_ARGUMENT"), (dict(history_range=None), "INVALID_ARGUMENT"),
    (dict(bias=None), "INVALID_ARGUMENT"), (dict(bias_ids=None), "INVALID_ARGUMENT"), (dict(bias_range=None), "INVALID_ARGUMENT"),
    (dict(n_history=-1), "INVALID_ARGUMENT"), (dict(path_len=-1), "INVALID_ARGUMENT"), (dict(n_bias=-1), "INVALID_ARGUMENT"),
    (dict(n_masks=-1), "INVALID_ARGUMENT"), (dict(n_history=2**30 + 1), "UNSUPPORTED_SHAPE"),
    (dict(n_bias=2**30 + 1), "UNSUPPORTED_SHAPE")])
def test_logits_refusals(qw, bad, code):
    a = logits_args(qw, **bad)
    assert qw.lib().qw_process_logits(ctypes.byref(a), None) == getattr(qw, code)
    assert qw.lib().qw_process_logits(None, None) == qw.INVALID_ARGUMENT


def test_tree_mask(qw):
    #        0 -> 1 -> 3 ; 0 -> 2 ; 4 a second root with child 5
    m = qw.tree_mask([-1, 0, 0, 1, -1, 4])
    assert m.dtype == np.uint64
    assert [int(x) for x in m] == [0b1, 0b11, 0b101, 0b1011, 0b10000, 0b110000]
    chain = qw.tree_mask(range(-1, 63))
    assert int(chain[63]) == (1 << 64) - 1
    assert qw.tree_mask([]).size == 0
    for bad in ([0], [-1, 1], [-2], [-1, 0, 5], [-1] * 65):
        with pytest.raises(ValueError):
            qw.tree_mask(bad)


def test_packed_arguments_have_the_c_layout(qw):
    # the binding packs its arguments; field by field they land where the ctypes classes have them
    for packer, cls in ((qw._KV_ROWS, qw.KvRowsStruct), (qw._TREE_ARGS, qw.TreeAttentionArgs),
                        (qw._LOGITS_ARGS, qw.ProcessLogitsArgs)):
        assert packer.size == ctypes.sizeof(cls)
        values = [i + 1 for i in range(len(cls._fields_))]
        got = cls.from_buffer_copy(packer.pack(*values))
        assert [getattr(got, name) for name, _ in cls._fields_] == values


def test_arrays_off_their_types_boundary_are_refused(qw):
    v, r, L = view(qw), rows(qw), qw.lib()
    for call in (L.qw_kv_append, L.qw_kv_read):
        assert call(ctypes.byref(v), ctypes.byref(r), P + 2, None, None) == qw.ALIGNMENT
        assert call(ctypes.byref(v), ctypes.byref(r), P, P + 1, None) == qw.ALIGNMENT
    for bad in (dict(mask=P + 4), dict(len=P + 2), dict(count=P + 2)):
        a = tree_args(qw, **bad)
        assert L.qw_tree_attention(ctypes.byref(v), ctypes.byref(a), P, 1 << 40, None) == qw.ALIGNMENT
    for name in ("penalties", "history", "history_range", "path", "bias_ids", "bias", "bias_range", "mask", "mask_index"):
        a = logits_args(qw, **{name: P + 2})
        assert L.qw_process_logits(ctypes.byref(a), None) == qw.ALIGNMENT, name


def test_results_that_share_an_address_are_refused(qw):
    v, L = view(qw), qw.lib()
    for bad in (dict(head_stride=0), dict(seq_stride=64)):
        assert L.qw_kv_read(ctypes.byref(v), ctypes.byref(rows(qw, **bad)), P, None, None) == qw.INVALID_ARGUMENT
    for bad in (dict(out_seq_stride=0), dict(out_node_stride=64), dict(out_head_stride=0)):
        a = tree_args(qw, **bad)
        assert L.qw_tree_attention(ctypes.byref(v), ctypes.byref(a), P, 1 << 40, None) == qw.INVALID_ARGUMENT


def test_lists_longer_than_the_counters_are_refused(qw):
    for bad in (dict(n_history=2**28 + 1), dict(path_len=2**28 + 1), dict(n_bias=2**28 + 1)):
        a = logits_args(qw, **bad)
        assert qw.lib().qw_process_logits(ctypes.byref(a), None) == qw.UNSUPPORTED_SHAPE
