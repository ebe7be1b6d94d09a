"""Layouts that the operators on caller-owned buffers refuse: results and written caches whose rows share
addresses.  Checked before the device is touched, so these run without a GPU."""
import ctypes

import pytest

from test_ops_host import P, rows, tree_args, view

Q = P + (1 << 30)


@pytest.fixture(scope="module")
def qw():
    from runtime_qwen3_decode_gb300 import build, qw as binding
    build.build()
    return binding


def planes(**kw):
    return dict(dict(v=Q, v_scale=Q), **kw)


def append(qw, v):
    """No rows: checked, and nothing to launch."""
    return qw.lib().qw_kv_append(ctypes.byref(v), ctypes.byref(rows(qw, n_max=0)), P, None, None)


# 2 sequences, 8 heads, 64 positions of 128
@pytest.mark.parametrize("good", [
    dict(), dict(seq_stride=64 * 8 * 128, head_stride=128, pos_stride=8 * 128),                     # token-major
    dict(seq_stride=128, head_stride=256, pos_stride=2048),                                         # sequences innermost
    dict(n_seq=1, seq_stride=0), dict(n_kv_heads=1, head_stride=0), dict(max_ctx=1, pos_stride=0),  # a dimension of one
    dict(pos_stride=144, head_stride=64 * 144, seq_stride=8 * 64 * 144 + 16),                       # padded rows
    dict(n_seq=65535, max_ctx=2**31 - 1, pos_stride=128, head_stride=2**31 * 128, seq_stride=2**34 * 128,
         scale_pos_stride=4, scale_head_stride=2**33, scale_seq_stride=2**36),
    dict(format=0), dict(format=1, v_scale=P)])
def test_a_cache_whose_rows_are_apart_can_be_written(qw, good):
    assert append(qw, view(qw, **planes(**good))) == qw.OK


@pytest.mark.parametrize("bad", [
    dict(head_stride=128), dict(head_stride=63 * 128), dict(seq_stride=128), dict(seq_stride=8 * 64 * 128 - 16),
    dict(seq_stride=64 * 8 * 128, head_stride=128, pos_stride=7 * 128), dict(seq_stride=128, head_stride=128, pos_stride=2048),
    dict(scale_head_stride=4), dict(scale_head_stride=63 * 4), dict(scale_seq_stride=4), dict(scale_seq_stride=8 * 64 * 4 - 4),
    dict(n_seq=65535, seq_stride=2**62, head_stride=2**62, pos_stride=2**62),
    dict(v=P), dict(v_scale=P)])
def test_a_cache_whose_rows_share_addresses_is_not_written(qw, bad):
    v = view(qw, **planes(**bad))
    assert append(qw, v) == qw.INVALID_ARGUMENT
    assert qw.lib().qw_tree_attention_scratch_bytes(ctypes.byref(v), 4, 16, 60) > 0  # reading it is fine


@pytest.mark.parametrize("bad", [dict(v=P), dict(head_stride=128), dict(row_stride=8 * 128, head_stride=128, seq_stride=128),
                                 dict(seq_stride=7 * 4 * 128), dict(head_stride=3 * 128 + 64)])
def test_rows_that_share_addresses_are_not_read_into(qw, bad):
    v, r = view(qw), rows(qw, **dict(dict(v=Q), **bad))
    assert qw.lib().qw_kv_read(ctypes.byref(v), ctypes.byref(r), P, None, None) == qw.INVALID_ARGUMENT


# 2 sequences, 4 nodes, 16 heads of 128
@pytest.mark.parametrize("out,code", [
    (dict(), "OUT_OF_MEMORY"), (dict(out_node_stride=128, out_head_stride=4 * 128), "OUT_OF_MEMORY"),
    (dict(out_seq_stride=128, out_node_stride=256, out_head_stride=1024), "OUT_OF_MEMORY"),
    (dict(out_head_stride=136, out_node_stride=16 * 136, out_seq_stride=4 * 16 * 136), "OUT_OF_MEMORY"),
    (dict(out_node_stride=128), "INVALID_ARGUMENT"), (dict(out_node_stride=15 * 128), "INVALID_ARGUMENT"),
    (dict(out_seq_stride=3 * 16 * 128), "INVALID_ARGUMENT"), (dict(out_head_stride=136), "INVALID_ARGUMENT"),
    (dict(out_seq_stride=2**62, out_node_stride=2**62, out_head_stride=2**62), "INVALID_ARGUMENT")])
def test_attention_results_that_share_addresses_are_refused(qw, out, code):
    # without scratch: nothing that passes the other checks is launched
    v, a = view(qw), tree_args(qw, **out)
    assert qw.lib().qw_tree_attention(ctypes.byref(v), ctypes.byref(a), P, 0, None) == getattr(qw, code)
