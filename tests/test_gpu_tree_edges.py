"""Drafted trees and 8-bit batches where tests/test_gpu_tree.py does not reach: caller memory that changes behind a call,
and contexts long enough that the steps attend on the tensor cores."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import qw_inputs as qi  # noqa: E402
from _helpers import HIDDEN_REL_L2, check_position, rel_l2  # noqa: E402
from test_gpu_tree import Q8_ROW, cache_tensors, path_of, setup, values  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from runtime_qwen3_decode_gb300 import build, qw as binding
    build.build()
    return binding


def test_a_tree_step_is_done_with_the_callers_memory_when_it_returns(qw):
    wl = qi.WORKLOADS["tiny"]
    host, m, b = setup(qw, wl, 4, 64, flags=False)
    b.prefill(1, [3, 1, 4, 1, 5])
    toks, parents = [9, 2, 6, 5], [-1, 0, 0, 1]
    b.tree_step(1, toks, parents)
    want = b.logits().clone()
    t = torch.tensor(toks, dtype=torch.int32).pin_memory()
    p = torch.tensor(parents, dtype=torch.int32).pin_memory()
    i32p = ctypes.POINTER(ctypes.c_int32)
    busy = torch.ones(1 << 26, device="cuda")
    torch.cuda.synchronize()
    for _ in range(100):  # some 10 ms before the step's turn comes
        busy.mul_(1.0)
    rc = qw.lib().qw_batch_tree_step(b._h, 1, 4, ctypes.cast(t.data_ptr(), i32p), ctypes.cast(p.data_ptr(), i32p), None)
    t.fill_(7)
    p.fill_(-1)
    assert rc == qw.OK
    b.last_n = 4
    assert torch.equal(b.logits(), want)
    b.close()
    m.close()


LONG = 1300  # with the tiny model's 8 KV heads: past the calls that attend on the CUDA cores


@pytest.mark.parametrize("kv", ["f32", "bf16"])
def test_every_node_of_a_long_sequence_is_its_path(qw, kv):
    """Against a batch that takes each node's path one decode step at a time (the attention of plain steps)."""
    wl = qi.WORKLOADS["tiny"].with_(kv_format=kv)
    host, m, b = setup(qw, wl, 8, LONG + 200)
    one = qw.Batch(m, 1, LONG + 200)
    g = np.random.default_rng(11)
    done = [int(t) for t in g.integers(0, wl.vocab, size=LONG)]
    b.prefill(3, done)
    parents = [-1, 0, 1, 1, 0, 4, 5, -1]
    for keep in ([0, 1, 3], [7]):
        toks = [int(t) for t in g.integers(0, wl.vocab, size=8)]
        picks = b.tree_step(3, toks, parents)
        lg, hid = b.logits().cpu().numpy(), b.debug_hidden().cpu().numpy()
        for i in (2, 3, 6, 7):
            path = [toks[j] for j in path_of(parents, i)]
            one.reset(0)
            one.prefill(0, done)
            for t in path:
                last = one.step(1, [t])
            check_position(lg[i], one.logits().cpu().numpy()[0], hid[:, i], one.debug_hidden().cpu().numpy()[:, 0],
                           picks[i], last[0], what=f"node {i}", hidden_tol=HIDDEN_REL_L2 * (1 if kv == "f32" else 2))
        b.tree_accept(3, keep)
        done += [toks[j] for j in keep]
        assert b.length(3) == len(done)
    for o in (b, one, m):
        o.close()


@pytest.mark.parametrize("tree", [False, True])
def test_a_long_8_bit_step_is_the_f32_step_over_the_values(qw, tree):
    wl = qi.WORKLOADS["tiny"]
    host, m, b8 = setup(qw, wl, 8, LONG + 200, 2)
    bf = qw.Batch(m, 8, LONG + 200)
    g = np.random.default_rng(12)
    lens = [LONG, 3, 700, 1100]
    for s, n in enumerate(lens):
        p = g.integers(0, wl.vocab, size=n)
        b8.prefill(s, p)
        bf.prefill(s, p)
    parents = [-1, 0, 0, 1, 3, 2, 5, -1]
    for step in range(2):
        k8, v8, ks, vs = cache_tensors(qw, b8)
        kf, vf = cache_tensors(qw, bf)
        kf.copy_(values(k8, ks))
        vf.copy_(values(v8, vs))
        n = 8 if tree else 4
        toks = g.integers(0, wl.vocab, size=n)
        for b in (b8, bf):
            if tree:
                b.tree_step(0, toks, parents)
            else:
                b.step(4, toks)
        h8, hf = b8.debug_hidden().cpu().numpy(), bf.debug_hidden().cpu().numpy()
        assert torch.isfinite(b8.logits()).all()
        for i in range(n):
            for l in range(wl.n_layers + 1):
                assert rel_l2(h8[l, i], hf[l, i]) <= HIDDEN_REL_L2 + Q8_ROW, (step, i, l)
        if tree:
            for b in (b8, bf):
                b.tree_accept(0, [0, 1, 3])
                assert b.length(0) == LONG + 3 * (step + 1)
    for o in (b8, bf, m):
        o.close()
