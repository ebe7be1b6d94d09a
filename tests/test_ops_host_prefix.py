"""Refusals of qw_prefix_attention and qw_sample_rows: checked before the device is touched, so these run without a GPU."""
import ctypes

import pytest

from test_ops_host import P, qw, view  # noqa: F401


def attention(lib, **kw):
    d = dict(q=P, out=P, dtype=lib.DT_BF16, n_max=4, n_heads=16, max_len=60, scale=0.1, q_seq_stride=4 * 16 * 128,
             q_node_stride=16 * 128, q_head_stride=128, out_seq_stride=4 * 16 * 128, out_node_stride=16 * 128,
             out_head_stride=128, mask=None, len=P, count=None)
    d.update(kw)
    return lib.TreeAttentionArgs(**d)


def call(qw, pre=None, own=None, args=None, plen=P, max_prefix=60, scratch=P, room=1 << 40):  # noqa: F811
    p, o = view(qw, **{"n_seq": 1, **(pre or {})}), view(qw, **(own or {}))
    a = attention(qw, **(args or {}))
    return qw.lib().qw_prefix_attention(ctypes.byref(p), ctypes.byref(o), ctypes.byref(a), plen, max_prefix, scratch, room, None)


@pytest.mark.parametrize("kw,code", [
    (dict(pre=dict(n_seq=2)), "INVALID_ARGUMENT"), (dict(pre=dict(format=1)), "INVALID_ARGUMENT"),
    (dict(pre=dict(n_kv_heads=4)), "INVALID_ARGUMENT"), (dict(pre=dict(k=None)), "INVALID_ARGUMENT"),
    (dict(pre=dict(k=P + 8)), "ALIGNMENT"), (dict(own=dict(v=P + 1)), "ALIGNMENT"), (dict(own=dict(pos_stride=64)), "INVALID_ARGUMENT"),
    (dict(max_prefix=-1), "INVALID_ARGUMENT"), (dict(max_prefix=65), "INVALID_ARGUMENT"), (dict(plen=None), "INVALID_ARGUMENT"),
    (dict(plen=P + 2), "ALIGNMENT"), (dict(scratch=None), "INVALID_ARGUMENT"), (dict(scratch=P + 16), "ALIGNMENT"),
    (dict(room=0), "OUT_OF_MEMORY"), (dict(args=dict(q=None)), "INVALID_ARGUMENT"), (dict(args=dict(out=P + 2)), "ALIGNMENT"),
    (dict(args=dict(len=None)), "INVALID_ARGUMENT"), (dict(args=dict(dtype=3)), "INVALID_ARGUMENT"),
    (dict(args=dict(scale=float("nan"))), "INVALID_ARGUMENT"), (dict(args=dict(n_max=65)), "UNSUPPORTED_SHAPE"),
    (dict(args=dict(n_max=-1)), "INVALID_ARGUMENT"), (dict(args=dict(n_heads=12)), "UNSUPPORTED_SHAPE"),
    (dict(args=dict(max_len=65)), "INVALID_ARGUMENT"), (dict(args=dict(out_node_stride=0)), "INVALID_ARGUMENT"),
    (dict(args=dict(q_head_stride=4)), "ALIGNMENT"), (dict(args=dict(mask=P + 4)), "ALIGNMENT"),
    (dict(own=dict(n_seq=9000), args=dict(n_max=64)), "UNSUPPORTED_SHAPE"),
    (dict(args=dict(n_max=0, q=None, out=None)), "OK")])
def test_prefix_refusals(qw, kw, code):  # noqa: F811
    assert call(qw, **kw) == getattr(qw, code)


def test_null_arguments(qw):  # noqa: F811
    o, a = view(qw), attention(qw)
    L = qw.lib()
    for x, y, z in ((None, ctypes.byref(o), ctypes.byref(a)), (ctypes.byref(o), None, ctypes.byref(a)), (ctypes.byref(o), ctypes.byref(o), None)):
        assert L.qw_prefix_attention(x, y, z, P, 4, P, 1 << 40, None) == qw.INVALID_ARGUMENT
    assert L.qw_prefix_attention_scratch_bytes(None, ctypes.byref(o), 1, 16, 4, 4) == 0
    assert L.qw_sample_rows(None, None) == qw.INVALID_ARGUMENT


def test_scratch_of_a_bound_covers_shorter_lengths(qw):  # noqa: F811
    big = dict(max_ctx=40000, seq_stride=8 * 40000 * 128, head_stride=40000 * 128, scale_seq_stride=8 * 40000 * 4,
               scale_head_stride=40000 * 4)
    for n_seq in (1, 3, 8, 64, 300):
        for n_max in (1, 5, 64):
            p, o = view(qw, n_seq=1, **big), view(qw, n_seq=n_seq, **big)
            need = lambda m, pre: qw.lib().qw_prefix_attention_scratch_bytes(ctypes.byref(p), ctypes.byref(o), n_max, 16, m, pre)  # noqa: E731
            last = [0, 0]
            for x in (0, 1, 64, 100, 700, 3000, 9999, 40000):
                now = [need(x, 40000), need(500, x)]
                assert now[0] >= last[0] > -1 and now[1] >= last[1] and min(now) > 0
                last = now


@pytest.mark.parametrize("Hkv,G", [(8, 2), (2, 7), (1, 64), (3, 3)])
def test_scratch_covers_fewer_sequences_and_rows(qw, Hkv, G):  # noqa: F811
    def need(n_seq, n_max, ctx):
        big = dict(max_ctx=ctx, n_kv_heads=Hkv, seq_stride=Hkv * ctx * 128, head_stride=ctx * 128, scale_seq_stride=Hkv * ctx * 4,
                   scale_head_stride=ctx * 4)
        p, o = view(qw, n_seq=1, **big), view(qw, n_seq=n_seq, **big)
        return qw.lib().qw_prefix_attention_scratch_bytes(ctypes.byref(p), ctypes.byref(o), n_max, Hkv * G, ctx, ctx)
    for ctx in (64, 700, 4096, 32768):
        for other in (1, 3, 8):
            by_seq = [need(n, other, ctx) for n in range(1, 70)]
            by_row = [need(other, n, ctx) for n in range(1, 65)]
            assert by_seq == sorted(by_seq) and by_row == sorted(by_row) and min(by_seq + by_row) > 0


def sample(lib, **kw):
    d = dict(logits=P, dtype=lib.DT_F32, n_rows=2, vocab=100, row_stride=100, u=P, temperature=P, top_k=P, top_p=P, min_p=P, tokens=P,
             probs=P, kept=P)
    d.update(kw)
    return lib.SampleRowsArgs(**d)


@pytest.mark.parametrize("bad,code", [
    (dict(logits=None), "INVALID_ARGUMENT"), (dict(u=None), "INVALID_ARGUMENT"), (dict(tokens=None), "INVALID_ARGUMENT"),
    (dict(dtype=3), "INVALID_ARGUMENT"), (dict(dtype=-1), "INVALID_ARGUMENT"), (dict(n_rows=-1), "INVALID_ARGUMENT"),
    (dict(n_rows=65536), "UNSUPPORTED_SHAPE"), (dict(vocab=0), "INVALID_ARGUMENT"), (dict(vocab=(1 << 24) + 1), "INVALID_ARGUMENT"),
    (dict(row_stride=-1), "INVALID_ARGUMENT"), (dict(logits=P + 2), "ALIGNMENT"), (dict(u=P + 1), "ALIGNMENT"),
    (dict(temperature=P + 2), "ALIGNMENT"), (dict(top_k=P + 2), "ALIGNMENT"), (dict(top_p=P + 2), "ALIGNMENT"),
    (dict(min_p=P + 2), "ALIGNMENT"), (dict(tokens=P + 2), "ALIGNMENT"), (dict(probs=P + 2), "ALIGNMENT"),
    (dict(kept=P + 2), "ALIGNMENT"), (dict(n_rows=0, logits=None), "OK")])
def test_sample_refusals(qw, bad, code):  # noqa: F811
    a = sample(qw, **bad)
    assert qw.lib().qw_sample_rows(ctypes.byref(a), None) == getattr(qw, code)


def test_packed_arguments_have_the_c_layout(qw):  # noqa: F811
    a = sample(qw, logits=P, u=P + 4, temperature=P + 8, top_k=P + 12, top_p=P + 16, min_p=P + 20, tokens=P + 24, probs=P + 28,
               kept=P + 32, row_stride=1 << 33)
    packed = qw._SAMPLE_ARGS.pack(P, qw.DT_F32, 2, 100, 1 << 33, *[P + 4 * i for i in range(1, 9)])
    assert bytes(a) == packed
