"""Prompt rows that the oracle takes in blocks leave the bits that a step for each leaves, for every weight format."""
import numpy as np
import pytest

import oracle
import qw_inputs as qi

FORMATS = {"bf16": {}, "int8": dict(weight_format="int8_g32"), "q8q8": dict(weight_format="int8_g32", act_format="q8")}


def models(fmt, **kw):
    wl = qi.Workload("small", seed=3, n_layers=2, hidden=192, n_heads=6, n_kv_heads=3, intermediate=352, vocab=512, **FORMATS[fmt])
    w = qi.make_weights(wl)
    return wl, [oracle.OracleModel(wl, w, **kw) for _ in range(2)]


def same_cache(wl, a, b):
    assert a.length == b.length
    for l in range(wl.n_layers):
        for h in range(wl.n_kv_heads):
            for p in range(a.length):
                for x, y in zip(a.kv_row(l, h, p), b.kv_row(l, h, p)):
                    np.testing.assert_array_equal(x.view(np.uint32), y.view(np.uint32))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 64, 65, 130])
def test_blocks_are_steps(fmt, n):
    wl, (a, b) = models(fmt, max_ctx=300, nthreads=3)
    g = np.random.default_rng(n)
    for model in (a, b):
        model.step(5)
    for _ in range(2):                                  # behind positions that are there already
        t = g.integers(0, wl.vocab, n)
        a.prompt(t)
        for x in t:
            b.step(int(x), want_logits=False)
    same_cache(wl, a, b)
    for x, y in zip(a.step(9, want_hidden=True), b.step(9, want_hidden=True)):
        np.testing.assert_array_equal(x.view(np.uint32), y.view(np.uint32))


def test_rows_rounded_as_they_are_stored():
    wl, (a, b) = models("bf16", max_ctx=80)
    for m in (a, b):
        m.set_kv_round_bf16(True)
    t = np.arange(70) * 7 % wl.vocab
    a.prompt(t)
    for x in t:
        b.step(int(x))
    same_cache(wl, a, b)


def test_many_positions_with_heads_on_threads():
    """Attention starts its threads from 256 positions on."""
    wl, (a, b) = models("bf16", max_ctx=400, nthreads=1)
    c = oracle.OracleModel(wl, a._w, max_ctx=400, nthreads=8)
    t = np.random.default_rng(1).integers(0, wl.vocab, 300)
    a.prompt(t)
    c.prompt(t)
    for x in t:
        b.step(int(x), want_logits=False)
    same_cache(wl, a, b)
    same_cache(wl, a, c)
    for x in (3, 4):
        want = a.step(x, want_hidden=True)
        for m in (b, c):
            for p, q in zip(m.step(x, want_hidden=True), want):
                np.testing.assert_array_equal(p.view(np.uint32), q.view(np.uint32))


def test_run_sequence_takes_long_prompts_in_blocks():
    wl, (a, b) = models("bf16", max_ctx=100)
    t = np.random.default_rng(2).integers(0, wl.vocab, 80)
    got = oracle.run_sequence(a, t, 3, want_hidden=True)
    for x in t[:-1]:
        b.step(int(x), want_logits=False)
    logits, hidden = b.step(int(t[-1]), want_hidden=True)
    np.testing.assert_array_equal(got["logits"][0], logits)
    np.testing.assert_array_equal(got["hidden"][0], hidden)
    for x, lg in zip(got["inputs"], got["logits"][1:]):
        np.testing.assert_array_equal(lg, b.step(x)[0])


def test_refusals():
    wl, (a, _) = models("bf16", max_ctx=20)
    for bad, code in (([1, wl.vocab], oracle.INVALID_ARGUMENT), ([-1], oracle.INVALID_ARGUMENT), ([1] * 21, oracle.CONTEXT_EXCEEDED)):
        with pytest.raises(oracle.OracleError) as e:
            a.prompt(bad)
        assert e.value.code == code and a.length == 0
    a.prompt([])
    a.prompt([1] * 20)
    assert a.length == 20
    w = qi.make_weights(wl)
    w["layers"][0]["up"][3, 3] = 0x7F80                 # +inf in bf16
    m = oracle.OracleModel(wl, w, max_ctx=80)
    with pytest.raises(oracle.OracleError) as e:
        m.prompt([1] * 70)
    assert e.value.code == oracle.NUMERICAL_FAILURE and m.length == 0
