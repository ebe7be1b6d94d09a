"""Continuations of one prompt in a batch (qw_batch_fork, qw_batch_sample): forked sequences, whose steps read their
shared positions once, against one oracle run each, held to the parity bar; draws in the place of greedy picks;
and a run of the operators together as such a batch uses them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import qw_inputs as qi  # noqa: E402
from _helpers import HIDDEN_REL_L2, LOGITS_MAX_ABS, check_position, rel_l2  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from runtime_qwen3_decode_gb300 import build, qw as binding
    build.build()
    return binding


@pytest.fixture(scope="module")
def tiny(qw):
    wl = qi.WORKLOADS["tiny"]
    host = qi.make_weights(wl)
    m = qw.Model(wl, qw.weights_to_device(host, int8=False), max_ctx=640)
    m.set_debug(qw.DEBUG_HIDDEN)
    yield wl, host, m
    m.close()


def prompt(wl, n, seed):
    return np.random.default_rng(seed).integers(0, wl.vocab, size=n).astype(np.int32)


def test_forked_sequences_match_independent_ones(qw, tiny):
    wl, host, m = tiny
    p = prompt(wl, 300, 1)
    cut = [300, 300, 280, 300]
    b = qw.Batch(m, 4, 400)
    b.prefill(0, p)
    for s in (1, 2, 3):
        b.fork(0, s, cut[s])
    assert [b.length(s) for s in range(4)] == cut
    refs = [oracle.OracleModel(wl, host, max_ctx=400) for _ in range(4)]
    for s in range(4):
        oracle.run_sequence(refs[s], p[:cut[s]], 0)
    g = np.random.default_rng(2)
    for step in range(6):
        tokens = g.integers(0, wl.vocab, 4)
        outs = [refs[s].step(int(tokens[s]), want_hidden=True) for s in range(4)]
        picks = b.step(4, tokens)
        lg, hid = b.logits().cpu().numpy(), b.debug_hidden().cpu().numpy()
        for s in range(4):
            check_position(lg[s], outs[s][0], hid[:, s], outs[s][1], picks[s], oracle.argmax(outs[s][0]), what=f"sequence {s} step {step}")
    for r in refs:
        r.close()
    b.close()


@pytest.mark.parametrize("kv", ["model", "int8"])
@pytest.mark.parametrize("n_seq,n", [(2, 256), (3, 300), (8, 511)])
def test_a_shared_prefix_gives_what_copies_give(qw, tiny, kv, n_seq, n):
    """The same rows, once known to be shared and once not: results within the parity bar of one another."""
    wl, _, m = tiny
    fmt = qw.KV_INT8_G32 if kv == "int8" else None
    p = prompt(wl, n, n)
    shared, apart = qw.Batch(m, n_seq, 600, fmt), qw.Batch(m, n_seq, 600, fmt)
    shared.prefill(0, p)
    for s in range(1, n_seq):
        shared.fork(0, s)
    for s in range(n_seq):
        apart.prefill(s, p)
    g = np.random.default_rng(n)
    same = True
    for step in range(5):
        tokens = g.integers(0, wl.vocab, n_seq)
        a, c = shared.step(n_seq, tokens), apart.step(n_seq, tokens)
        la, lc = shared.logits().cpu().numpy(), apart.logits().cpu().numpy()
        same = same and np.array_equal(la, lc)
        assert np.abs(la - lc).max() <= LOGITS_MAX_ABS
        ha, hc = shared.debug_hidden().cpu().numpy(), apart.debug_hidden().cpu().numpy()
        for s in range(n_seq):
            assert rel_l2(ha[:, s], hc[:, s]) <= HIDDEN_REL_L2
        if step == 2 and n_seq > 2:  # the last sequence starts anew: nothing is shared any more by all
            for b in (shared, apart):
                b.reset(n_seq - 1)
                b.prefill(n_seq - 1, p[:50])
    assert not same or kv == "int8"  # the two ways add in other orders: the shared one did run
    shared.close()
    apart.close()


def test_forks_of_forks_share_what_all_have(qw, tiny):
    wl, host, m = tiny
    p = prompt(wl, 290, 5)
    b, c = qw.Batch(m, 3, 400), qw.Batch(m, 3, 400)
    for x in (b, c):
        x.prefill(0, p)
    b.fork(0, 1, 270)
    b.step(2, [3, 4])                 # sequence 1 goes its own way from 270 on
    b.fork(1, 2)                      # 271 positions, 270 of them the prompt's
    assert [b.length(s) for s in range(3)] == [291, 271, 271]
    c.prefill(1, p[:270])
    c.prefill(2, np.concatenate([p[:270], [4]]).astype(np.int32))
    c.step(2, [3, 4])
    for tokens in ([9, 8, 7], [1, 2, 3]):
        b.step(3, tokens)
        c.step(3, tokens)
        assert np.abs(b.logits().cpu().numpy() - c.logits().cpu().numpy()).max() <= LOGITS_MAX_ABS
    b.close()
    c.close()


def test_short_prefixes_and_single_sequences_step_as_ever(qw, tiny):
    wl, _, m = tiny
    p = prompt(wl, 100, 6)
    b, c = qw.Batch(m, 2, 200), qw.Batch(m, 2, 200)
    b.prefill(0, p)
    b.fork(0, 1)
    for s in range(2):
        c.prefill(s, p)
    b.step(2, [5, 6])
    c.step(2, [5, 6])
    assert torch.equal(b.logits(), c.logits())
    b.step(1, [7])
    c.step(1, [7])
    assert torch.equal(b.logits(), c.logits())
    b.close()
    c.close()


def test_a_fork_takes_over_the_last_pick_and_logits(qw, tiny):
    wl, _, m = tiny
    b, c = qw.Batch(m, 3, 200), qw.Batch(m, 3, 200)
    p = prompt(wl, 40, 7)
    pick = b.prefill(0, p)
    b.fork(0, 2)
    b.fork(0, 1, 39)
    with pytest.raises(qw.QwError) as e:
        b.step(2)                      # sequence 1 has no last pick
    assert e.value.code == qw.INVALID_ARGUMENT
    c.prefill(0, p)
    c.prefill(1, p[:39])
    c.prefill(2, p)
    b.step(3, [-1, 11, -1])
    c.step(3, [pick, 11, pick])
    assert torch.equal(b.logits(), c.logits())
    u = torch.tensor([0.1, 0.5, 0.9], device="cuda")
    t = torch.full((3,), 1.5, device="cuda")
    b.reset(1)
    b.fork(0, 1)
    drawn = b.sample(3, u, temperature=t)   # rows 0 and 2 of the step, row 1 what the fork took over
    lg = b.logits()
    lg = torch.stack([lg[0], lg[0], lg[2]])
    assert drawn == qw.sample_rows(lg, u, temperature=t).tolist()
    b.close()
    c.close()


def test_draws_go_on(qw, tiny):
    """Drawn tokens are what qw_sample_rows draws from the step's logits, and what the next step is fed."""
    wl, _, m = tiny
    b, c = qw.Batch(m, 4, 400), qw.Batch(m, 4, 400)
    p = prompt(wl, 260, 8)
    for x in (b, c):
        x.prefill(0, p)
        for s in range(1, 4):
            x.fork(0, s)
    f = lambda *v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    k = torch.tensor([0, 20, 5, 1], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for step in range(5):
        u = torch.rand((4,), generator=g, device="cuda")
        args = dict(temperature=f(1.0, 2.0, 0.7, 0.0), top_k=k, top_p=f(0.9, 1.0, 0.8, 1.0), min_p=f(0.0, 0.01, 0.0, 0.0))
        drawn = b.sample(4, u, **args)
        if step:
            assert drawn == qw.sample_rows(b.logits(), u, **args).tolist()
        b.step(4)                      # goes on with the drawn tokens
        c.step(4, drawn)
        assert torch.equal(b.logits(), c.logits())
    b.close()
    c.close()


def test_refusals(qw, tiny):
    wl, _, m = tiny
    b = qw.Batch(m, 3, 64)
    b.prefill(0, prompt(wl, 20, 9))
    for args in ((0, 0, 5), (0, 3, 5), (-1, 1, 5), (0, 1, 0), (0, 1, 21), (1, 0, 1)):
        with pytest.raises(qw.QwError) as e:
            b.fork(*args)
        assert e.value.code == qw.INVALID_ARGUMENT
    u = torch.full((3,), 0.5, device="cuda")
    with pytest.raises(qw.QwError) as e:
        b.sample(2, u[:2])             # sequence 1 has no logits
    assert e.value.code == qw.INVALID_ARGUMENT
    with pytest.raises(ValueError):
        b.sample(1, u)
    b.fork(0, 1)
    b.tree_step(0, [1, 2], [-1, 0])
    with pytest.raises(qw.QwError) as e:
        b.sample(1, u[:1])             # row 0 is a node's
    assert e.value.code == qw.INVALID_ARGUMENT
    b.fork(0, 1, 10)                   # the waiting tree is sequence 0's
    b.tree_accept(0, [0])
    b.step(2, [1, 2])
    with pytest.raises(qw.QwError) as e:
        b.sample(2, u[:2], temperature=torch.tensor([-1.0, 1.0], device="cuda"))
    assert e.value.code == qw.INVALID_ARGUMENT
    with pytest.raises(qw.QwError):
        b.step(2)                      # recorded until the reset
    b.reset()
    b.prefill(0, prompt(wl, 20, 9))
    b.sample(1, u[:1])
    b.close()


@pytest.mark.parametrize("kind,dt", [("bf16", torch.bfloat16), ("int8", torch.float16), ("f32", torch.float32)])
def test_a_run_of_the_operators_together(qw, kind, dt):
    """Eight continuations of one prompt, by hand: their rows appended, attention over the prefix and their own, logits
    of a head, processed and drawn from; each stage against its definition."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    B, H, G, D, P, C, V = 8, 4, 2, 128, 700, 40, 5003
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731

    def cache(n, c):
        if kind == "int8":
            z = [torch.zeros((n, H, c, D), dtype=torch.int8, device="cuda") for _ in range(2)]
            return qw.KvView(*z, *[torch.zeros((n, H, c, D // 32), dtype=torch.float16, device="cuda") for _ in range(2)])
        return qw.KvView(*[torch.zeros((n, H, c, D), device="cuda", dtype={"bf16": torch.bfloat16, "f32": torch.float32}[kind]) for _ in range(2)])
    pre, own = cache(1, P), cache(B, C)
    zero, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    qw.kv_append(pre, rnd(1, H, P, D).to(dt), rnd(1, H, P, D).to(dt), zero)
    plen = torch.full((1,), P, dtype=torch.int32, device="cuda")
    head = rnd(H * G * D, V) / 30
    history = torch.zeros((B, 16), dtype=torch.int32, device="cuda")
    back = lambda view, n, c: [torch.zeros((n, H, c, D), device="cuda") for _ in range(2)]  # noqa: E731
    pk, pv = back(pre, 1, P)
    qw.kv_read(pre, pk, pv, zero)
    for step in range(12):
        k, v, q = rnd(B, H, 1, D).to(dt), rnd(B, H, 1, D).to(dt), rnd(B, 1, H * G, D).to(dt)
        qw.kv_append(own, k, v, lens)
        out = qw.prefix_attention(pre, own, q, lens, plen, max_len=C - 1)
        ok, ov = back(own, B, step + 1)
        qw.kv_read(own, ok, ov, torch.zeros_like(lens))
        kk, vv = (torch.cat([a.expand(B, -1, -1, -1), o], 2).double().repeat_interleave(G, 1) for a, o in ((pk, ok), (pv, ov)))
        s = (q.double().transpose(1, 2) @ kk.transpose(2, 3)) * D ** -0.5
        want = (torch.softmax(s, -1) @ vv).transpose(1, 2)
        u = torch.finfo(dt).eps / 2
        # scores of a few units whose K and q are rounded to 16 bits, weights and V too, the result once more
        tol = (2 * 8 * u + 4 * u + 2.0 ** -13) * float(vv.abs().max())
        assert float((out.double() - want).abs().max()) <= tol
        logits = out.reshape(B, -1).float() @ head
        tok = torch.empty(B, dtype=torch.int32, device="cuda")
        ranges = torch.stack([torch.arange(B, device="cuda") * 16, torch.arange(B, device="cuda") * 16 + step], 1).int().contiguous()
        qw.process_logits(logits, history=history.flatten(), history_range=ranges,
                          penalties=torch.tensor([[1.3, 0.5, 0.1]], device="cuda").expand(B, 3).contiguous())
        uu = torch.rand((B,), generator=g, device="cuda")
        qw.sample_rows(logits, uu, top_k=torch.full((B,), 40, dtype=torch.int32, device="cuda"), tokens=tok)
        top = logits.double().topk(40, 1)
        p = torch.softmax(top.values, 1).cumsum(1)
        pick = torch.searchsorted(p, uu.double()[:, None], right=True).clamp(max=39)
        near = (p - uu.double()[:, None]).abs().min(1).values < 1e-8
        assert ((top.indices.gather(1, pick)[:, 0] == tok) | near).all()
        history[:, step] = tok
        lens += 1
