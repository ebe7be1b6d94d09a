"""Edges of continuations in a batch (qw_batch_fork, qw_batch_sample): logits that are no longer a sequence's last
position's, that the shared positions are read once, steps long enough for the tensor cores, draws from logits that a fork
took over."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import qw_inputs as qi  # noqa: E402
from _helpers import HIDDEN_REL_L2, LOGITS_MAX_ABS, rel_l2  # noqa: E402
from test_gpu_fork import prompt, qw, tiny  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def refused(qw, call):  # noqa: F811
    with pytest.raises(qw.QwError) as e:
        call()
    assert e.value.code == qw.INVALID_ARGUMENT


@pytest.mark.parametrize("seq", [1, 2])
def test_accepted_nodes_leave_no_logits_behind(qw, tiny, seq):  # noqa: F811
    """Row seq of the logits is behind all of the tree's nodes: it keeps what the position before them gave."""
    wl, _, m = tiny
    b, c = qw.Batch(m, 4, 64), qw.Batch(m, 4, 64)
    u = torch.full((4,), 0.5, device="cuda")
    for s in range(seq + 1):
        b.prefill(s, prompt(wl, 20, s))
        c.prefill(s, prompt(wl, 20, s))
    pick = b.tree_step(seq, [5], [-1])[0]
    b.tree_accept(seq, [0])
    refused(qw, lambda: b.sample(seq + 1, u[:seq + 1]))
    b.fork(seq, 3)                                   # takes no logits over
    for s in (0, 1, 2):
        if s != seq:
            b.prefill(s, prompt(wl, 1, 9))
            c.prefill(s, prompt(wl, 1, 9))
    refused(qw, lambda: b.sample(4, u))
    b.step(seq)                                      # the rows below are there again, row seq is not
    c.step(seq)
    refused(qw, lambda: b.sample(seq + 1, u[:seq + 1]))
    c.prefill(seq, [5], want_token=False)
    tokens = [7] * seq
    b.step(seq + 1, tokens + [-1])                   # and goes on with the last node's pick
    c.step(seq + 1, tokens + [pick])
    assert np.abs(b.logits().cpu().numpy() - c.logits().cpu().numpy()).max() <= 5e-2
    assert b.sample(seq + 1, u[:seq + 1]) == qw.sample_rows(b.logits(), u[:seq + 1]).tolist()
    b.close()
    c.close()


def test_a_tree_of_which_nothing_is_kept_leaves_the_logits(qw, tiny):  # noqa: F811
    wl, _, m = tiny
    b = qw.Batch(m, 2, 64)
    u = torch.tensor([0.3, 0.6], device="cuda")
    for s in range(2):
        b.prefill(s, prompt(wl, 20, s))
    b.step(2, [1, 2])
    want = qw.sample_rows(b.logits(), u).tolist()
    b.tree_step(1, [5], [-1])
    b.tree_accept(1, [])
    b.prefill(0, prompt(wl, 1, 3))                   # row 0 was the node's
    assert b.sample(2, u)[1] == want[1]
    b.close()


@pytest.fixture(scope="module")
def long(qw):  # noqa: F811
    wl = qi.WORKLOADS["tiny"]
    m = qw.Model(wl, qw.weights_to_device(qi.make_weights(wl), int8=False), max_ctx=4200)
    m.set_debug(qw.DEBUG_HIDDEN)
    yield wl, m
    m.close()


LAYERS, KV_HEADS, DIM = 2, 8, 128                    # of the small model


def key_rows(b, seq, kv, ctx):
    """The K codes or f32 rows of one sequence of a batch, [layer][KV head][position][dim] in its workspace."""
    t = b.workspace if kv == "int8" else b.workspace.view(torch.float32)
    n = LAYERS * KV_HEADS * ctx * DIM
    return t[seq * n:(seq + 1) * n].view(LAYERS, KV_HEADS, ctx, DIM)


@pytest.mark.parametrize("kv,n_seq,n", [("model", 2, 256), ("model", 3, 300), ("model", 8, 511), ("int8", 8, 256), ("int8", 6, 511)])
def test_shared_positions_are_read_once(qw, tiny, kv, n_seq, n):  # noqa: F811
    """A step's result does not depend on a later sequence's copies of what all share, and does on the first one's; where
    nothing is known to be shared it is the other way round."""
    wl, _, m = tiny
    assert (wl.n_layers, wl.n_kv_heads, wl.head_dim) == (LAYERS, KV_HEADS, DIM)
    fmt = qw.KV_INT8_G32 if kv == "int8" else None
    p = prompt(wl, n, n)

    def logits(shared, seq):
        b = qw.Batch(m, n_seq, 600, fmt)
        b.prefill(0, p)
        for s in range(1, n_seq):
            b.fork(0, s) if shared else b.prefill(s, p)
        if seq is not None:
            rows = key_rows(b, seq, kv, 600)
            before = rows[:, :, 100].clone()
            assert before.any()
            rows[:, :, 100] = before.flip(-1)
        b.step(n_seq, list(range(5, 5 + n_seq)))
        out = b.logits().clone()
        b.close()
        return out
    last = n_seq - 1
    want = logits(True, None)
    assert torch.equal(logits(True, last), want)
    moved = logits(True, 0)
    assert not torch.equal(moved[0], want[0]) and not torch.equal(moved[last], want[last])
    want = logits(False, None)
    moved = logits(False, last)
    assert torch.equal(moved[0], want[0]) and not torch.equal(moved[last], want[last])


@pytest.mark.parametrize("n_seq,n", [(2, 1023), (3, 767), (5, 767), (2, 1024), (3, 768), (5, 768)])
def test_few_sequences_over_8_bits_share_long_prefixes_only(qw, long, n_seq, n):  # noqa: F811
    """Below the bound a step is the one over copies, bit for bit; from it on it does not read a later sequence's copy."""
    wl, m = long
    p = prompt(wl, n, n)
    out = []
    for spoilt in (False, True):
        b = qw.Batch(m, n_seq, 1100, qw.KV_INT8_G32)
        b.prefill(0, p)
        for s in range(1, n_seq):
            b.fork(0, s)
        if spoilt:
            rows = key_rows(b, n_seq - 1, "int8", 1100)
            rows[:, :, 100] = rows[:, :, 100].flip(-1)
        b.step(n_seq, list(range(5, 5 + n_seq)))
        out.append(b.logits().clone())
        b.close()
    assert torch.equal(out[0][:-1], out[1][:-1])
    assert torch.equal(out[0][-1], out[1][-1]) == (n in (768, 1024))


def test_the_first_draw_is_from_the_logits_that_a_fork_took_over(qw, tiny):  # noqa: F811
    wl, _, m = tiny
    b = qw.Batch(m, 4, 400)
    b.prefill(0, prompt(wl, 260, 8))
    b.step(1)
    row = b.logits().clone()                         # of the position that the forks go on from
    for s in range(1, 4):
        b.fork(0, s)
    u = torch.tensor([0.05, 0.4, 0.7, 0.95], device="cuda")
    k = torch.tensor([0, 20, 5, 1], dtype=torch.int32, device="cuda")
    t = torch.tensor([2.0, 2.0, 0.7, 0.0], device="cuda")
    drawn = b.sample(4, u, temperature=t, top_k=k)
    assert drawn == qw.sample_rows(row.expand(4, -1), u, temperature=t, top_k=k).tolist()
    assert len(set(drawn)) > 1
    c = qw.Batch(m, 4, 400)
    c.prefill(0, prompt(wl, 260, 8))
    c.step(1)
    for s in range(1, 4):
        c.fork(0, s)
    b.step(4)                                        # goes on with them
    c.step(4, drawn)
    assert torch.equal(b.logits(), c.logits())
    b.close()
    c.close()


@pytest.mark.parametrize("kv", ["model", "int8"])
@pytest.mark.parametrize("n_seq,n", [(8, 1100), (8, 4000), (3, 4001)])
def test_steps_behind_a_long_prefix(qw, long, kv, n_seq, n):  # noqa: F811
    """Long enough for the tensor cores inside a captured step: tensor maps that begin behind the prefix, replayed for own
    parts of different lengths, against batches that hold the same rows as copies."""
    wl, m = long
    fmt = qw.KV_INT8_G32 if kv == "int8" else None
    p = prompt(wl, n, n)
    cut = [n - (7 * s if s % 2 else 0) for s in range(n_seq)]
    shared, apart = qw.Batch(m, n_seq, 4200, fmt), qw.Batch(m, n_seq, 4200, fmt)
    shared.prefill(0, p)
    for s in range(1, n_seq):
        shared.fork(0, s, cut[s])
    for s in range(n_seq):
        apart.prefill(s, p[:cut[s]])
        for b in (shared, apart):
            b.prefill(s, prompt(wl, 3 + s, s))
    assert [shared.length(s) for s in range(n_seq)] == [apart.length(s) for s in range(n_seq)]
    g = np.random.default_rng(n)
    same = True
    for _ in range(130 if n_seq == 3 else 12):       # past a tile of a sequence's own positions
        tokens = g.integers(0, wl.vocab, n_seq)
        shared.step(n_seq, tokens)
        apart.step(n_seq, tokens)
        a, c = shared.logits().cpu().numpy(), apart.logits().cpu().numpy()
        same = same and np.array_equal(a, c)
        assert np.abs(a - c).max() <= LOGITS_MAX_ABS
        ha, hc = shared.debug_hidden().cpu().numpy(), apart.debug_hidden().cpu().numpy()
        for s in range(n_seq):
            assert rel_l2(ha[:, s], hc[:, s]) <= HIDDEN_REL_L2
    assert not same
    shared.close()
    apart.close()
