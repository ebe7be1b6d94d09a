"""Edges of continuations in a batch (qw_batch_fork, qw_batch_sample): logits that are no longer a sequence's last
position's, that the shared positions are read once, steps long enough for the tensor cores, draws from logits that a fork
took over."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

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
