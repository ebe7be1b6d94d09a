"""Drafted tokens in a batch (qw_batch_tree_step, qw_batch_tree_accept) and batches over 8-bit caches
(qw_batch_create_kv).

Every node of a tree is held to the parity bar against an oracle that runs the prompt and the node's
path token by token.  The oracle has no 8-bit cache: there, the rows of layer 0 (which no
attention precedes) must be the quantised rows of the f32 cache, bit for bit, and a step must agree with a
step of an f32-cache batch whose cached rows were overwritten by the values that the 8-bit ones stand for.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import qw_inputs as qi  # noqa: E402
from _helpers import HIDDEN_REL_L2, check_position, rel_l2  # noqa: E402

pytestmark = pytest.mark.gpu

# One 8-bit row: an element is off by a uniform error of up to half of d = amax / 127, d / sqrt(12)
# root-mean-square, and the largest of 32 elements is at most about 4 times their rms.  A step's own
# new row is the one row that differs between the 8-bit batch and the overwritten f32 one.
Q8_ROW = 4 / (127 * 12 ** 0.5)


@pytest.fixture(scope="module")
def qw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from runtime_qwen3_decode_gb300 import build, qw as binding
    build.build()
    return binding


def setup(qw, wl, max_batch, ctx, kv_format=None, flags=True):
    host = qi.make_weights(wl)
    m = qw.Model(wl, qw.weights_to_device(host, int8=wl.weight_format == "int8_g32"), max_ctx=ctx)
    if flags:
        m.set_debug(qw.DEBUG_HIDDEN)
    return host, m, qw.Batch(m, max_batch, ctx, kv_format)


def path_of(parents, i):
    out = []
    while i >= 0:
        out.insert(0, i)
        i = parents[i]
    return out


def oracle_after(wl, host, tokens, ctx):
    """(logits, hidden) of the last of `tokens`."""
    ref = oracle.OracleModel(wl, host, max_ctx=ctx)
    for t in tokens[:-1]:
        ref.step(int(t))
    out = ref.step(int(tokens[-1]), want_hidden=True)
    ref.close()
    return out


TREES = [[-1], [-1, 0, 1, 2], [-1, 0, 0, 1, 2, 2, -1, 6], [-1, -1, -1]]


@pytest.mark.parametrize("parents", TREES)
@pytest.mark.parametrize("kv", ["f32", "bf16"])
def test_every_node_is_its_path(qw, parents, kv):
    wl = qi.WORKLOADS["tiny"].with_(kv_format=kv)
    n = len(parents)
    host, m, b = setup(qw, wl, 8, 64)
    g = np.random.default_rng(n)
    prompt = g.integers(0, wl.vocab, size=9)
    toks = g.integers(0, wl.vocab, size=n)
    b.prefill(2, prompt)
    picks = b.tree_step(2, toks, parents)
    assert b.length(2) == 9  # nothing is appended before the accept
    lg, hid = b.logits().cpu().numpy(), b.debug_hidden().cpu().numpy()
    tol = HIDDEN_REL_L2 if kv == "f32" else 2 * HIDDEN_REL_L2  # both sides round their own bf16 rows
    for i in range(n):
        seq = list(prompt) + [toks[j] for j in path_of(parents, i)]
        ologits, ohid = oracle_after(wl, host, seq, 64)
        check_position(lg[i], ologits, hid[:, i], ohid, picks[i], oracle.argmax(ologits), what=f"node {i}", hidden_tol=tol)
    b.close()
    m.close()


@pytest.mark.parametrize("kv_format", [None, 2])
def test_accept_then_go_on(qw, kv_format):
    """Draft, accept a path, decode on and draft again; against the oracle (f32 cache), or, over 8 bits, against a
    batch that took the same tokens one step at a time."""
    wl = qi.WORKLOADS["tiny"]
    host, m, b = setup(qw, wl, 8, 160, kv_format)
    g = np.random.default_rng(3)
    prompt = g.integers(0, wl.vocab, size=120)
    parents = [-1, 0, 0, 2, 2, 4]
    one = qw.Batch(m, 2, 160, kv_format) if kv_format else None
    done = [int(t) for t in prompt]
    b.prefill(1, prompt)
    if one:
        one.prefill(0, prompt)
    for rnd, keep in enumerate([[0, 2, 4], [0], [], [0, 2, 4, 5], [0, 1]]):
        toks = [int(t) for t in g.integers(0, wl.vocab, size=6)]
        picks = b.tree_step(1, toks, parents)
        b.tree_accept(1, keep)
        done += [toks[i] for i in keep]
        assert b.length(1) == len(done)
        if one:
            for i in keep:
                one.step(1, [toks[i]])
        nxt = picks[keep[-1]] if keep else int(g.integers(0, wl.vocab))
        # the batch's rows before the drafted sequence decode beside it
        if rnd == 0:
            b.prefill(0, prompt[:5])
        b.step(2, [7, -1 if keep else nxt])  # -1: the accepted path's last pick
        done.append(nxt)
        lg, hid = b.logits().cpu().numpy()[1], b.debug_hidden().cpu().numpy()[:, 1]
        if one:
            one.step(1, [nxt])
            ol, oh = one.logits().cpu().numpy()[0], one.debug_hidden().cpu().numpy()[:, 0]
            # the same codes up to those that sit on a rounding border (the attention's split differs): the bar of f32
            check_position(lg, ol, hid, oh, what=f"round {rnd}", hidden_tol=HIDDEN_REL_L2 + Q8_ROW)
        else:
            ol, oh = oracle_after(wl, host, done, 160)
            check_position(lg, ol, hid, oh, what=f"round {rnd}")
    b.close()
    m.close()


def test_last_pick_feeds_node_zero(qw):
    wl = qi.WORKLOADS["tiny"]
    host, m, b = setup(qw, wl, 4, 32)
    prompt = np.arange(5) * 11 + 3
    first = b.prefill(3, prompt)
    a = b.tree_step(3, [-1, 9, 10], [-1, 0, 0])
    la = b.logits().clone()
    c = b.tree_step(3, [first, 9, 10], [-1, 0, 0])
    assert a == c and torch.equal(la, b.logits())
    b.tree_accept(3, [0, 2])
    x = b.step(4, [1, 1, 1, -1])
    y_tok = c[2]
    b2 = qw.Batch(m, 1, 32)
    b2.prefill(0, list(prompt) + [first, 10])
    y = b2.step(1, [y_tok])
    lx, ly = b.logits()[3], b2.logits()[0]
    assert float((lx - ly).abs().max()) <= 5e-2
    assert len(x) == 4 and len(y) == 1
    for o in (b, b2, m):
        o.close()


def cache_tensors(qw, b):
    """Views of a batch's cache in its workspace: K, V (and scales) [seq][layer][head][position][...]."""
    c = b.model.cfg
    shape = (b.max_batch, c.n_layers, c.n_kv_heads, b.max_ctx, c.head_dim)
    elems = int(np.prod(shape))
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    ws, at, out = b.workspace, 0, []
    sizes = [1, 1, 2 / 32, 2 / 32] if b.kv_format == qw.KV_INT8_G32 else [4, 4]
    for k, sz in enumerate(sizes):
        nbytes = int(elems * sz)
        dt = torch.float32 if sz == 4 else torch.int8 if sz == 1 else torch.float16
        last = 4 if k >= 2 else c.head_dim
        out.append(ws[at:at + nbytes].view(dt).view(*shape[:4], last))
        at += up(nbytes)
    return out


def values(codes, scales):
    return codes.float() * scales.float().repeat_interleave(32, -1)


@pytest.mark.parametrize("chunks", [[37], [20, 17]])
def test_int8_prompt_rows_are_the_quantised_rows(qw, chunks):
    wl = qi.WORKLOADS["tiny"]
    host, m, b8 = setup(qw, wl, 2, 80, 2)
    bf = qw.Batch(m, 2, 80)
    prompt = np.random.default_rng(1).integers(0, wl.vocab, size=sum(chunks))
    at = 0
    for n in chunks:
        p8 = b8.prefill(1, prompt[at:at + n])
        pf = bf.prefill(1, prompt[at:at + n])
        at += n
    k8, v8, ks, vs = cache_tensors(qw, b8)
    kf, vf = cache_tensors(qw, bf)
    # layer 0's rows come from the same projections: the 8-bit batch holds their groups, quantised
    for c8, s8, f in ((k8, ks, kf), (v8, vs, vf)):
        rows = f[1, 0, :, :at].contiguous()
        codes = torch.zeros((1, 8, at, 128), dtype=torch.int8, device="cuda")
        scale = torch.zeros((1, 8, at, 4), dtype=torch.float16, device="cuda")
        view = qw.KvView(codes, codes.clone(), scale, scale.clone())
        qw.kv_append(view, rows[None], rows[None], torch.zeros(1, dtype=torch.int32, device="cuda"))
        assert torch.equal(c8[1, 0, :, :at], codes[0])
        assert torch.equal(s8[1, 0, :, :at], scale[0])
        # every layer: within the noise of 8-bit rows behind attention over 8-bit rows
        for l in range(wl.n_layers):
            assert rel_l2(values(c8[1, l, :, :at], s8[1, l, :, :at]).cpu().numpy(), f[1, l, :, :at].cpu().numpy()) <= 2 * Q8_ROW
    assert p8 >= 0 and pf >= 0
    for o in (b8, bf, m):
        o.close()


@pytest.mark.parametrize("tree", [None, [-1, 0, 0, 1]])
def test_int8_step_is_the_f32_step_over_the_values(qw, tree):
    wl = qi.WORKLOADS["tiny"]
    host, m, b8 = setup(qw, wl, 4, 200, 2)
    bf = qw.Batch(m, 4, 200)
    g = np.random.default_rng(2)
    lens = [150, 3, 64, 129]
    for s, n in enumerate(lens):
        p = g.integers(0, wl.vocab, size=n)
        b8.prefill(s, p)
        bf.prefill(s, p)
    for step in range(3):
        k8, v8, ks, vs = cache_tensors(qw, b8)
        kf, vf = cache_tensors(qw, bf)
        kf.copy_(values(k8, ks))
        vf.copy_(values(v8, vs))
        toks = g.integers(0, wl.vocab, size=4)
        if tree:
            b8.tree_step(3, toks, tree)
            bf.tree_step(3, toks, tree)
        else:
            b8.step(4, toks)
            bf.step(4, toks)
        l8, lf = b8.logits().cpu().numpy(), bf.logits().cpu().numpy()
        h8, hf = b8.debug_hidden().cpu().numpy(), bf.debug_hidden().cpu().numpy()
        assert np.isfinite(l8).all()
        for i in range(4):
            for l in range(wl.n_layers + 1):
                # a short sequence's new row is a large part of what it attends to; a tree node sees up to three new rows
                assert rel_l2(h8[l, i], hf[l, i]) <= HIDDEN_REL_L2 + Q8_ROW, (step, i, l)
        if tree:
            b8.tree_accept(3, [0, 1, 3])
            bf.tree_accept(3, [0, 1, 3])
            assert b8.length(3) == 129 + 3 * (step + 1) == bf.length(3)
    for o in (b8, bf, m):
        o.close()


def test_int8_full_shape(qw):
    wl = qi.WORKLOADS["qwen3_0p6b_decode"]
    host, m, b8 = setup(qw, wl, 8, 96, 2)
    bf = qw.Batch(m, 8, 96)
    g = np.random.default_rng(4)
    prompt = g.integers(0, wl.vocab, size=40)
    b8.prefill(0, prompt)
    bf.prefill(0, prompt)
    k8, v8, ks, vs = cache_tensors(qw, b8)
    kf, vf = cache_tensors(qw, bf)
    kf.copy_(values(k8, ks))
    vf.copy_(values(v8, vs))
    parents = [-1, 0, 1, 1, 0, 4, 4, 6]
    toks = g.integers(0, wl.vocab, size=8)
    b8.tree_step(0, toks, parents)
    bf.tree_step(0, toks, parents)
    h8, hf = b8.debug_hidden().cpu().numpy(), bf.debug_hidden().cpu().numpy()
    for i in range(8):
        assert rel_l2(h8[-1, i], hf[-1, i]) <= HIDDEN_REL_L2 + Q8_ROW
    for o in (b8, bf, m):
        o.close()


def test_tree_after_preparing_its_logits(qw):
    """The nodes' logits under a grammar mask and penalties, then sampled greedily: as a user checks a draft."""
    wl = qi.WORKLOADS["tiny"]
    host, m, b = setup(qw, wl, 4, 64)
    prompt = np.arange(12) * 7 + 1
    b.prefill(0, prompt)
    b.tree_step(0, [5, 6, 7], [-1, 0, 0])
    lg = b.logits()
    V = wl.vocab
    words = torch.zeros((1, (V + 31) // 32), dtype=torch.int32, device="cuda")
    words[0, 2], words[0, 40] = 0b110, 1 << 30  # tokens 65, 66, 1310
    hist = torch.from_numpy(prompt.astype(np.int32)).cuda()
    qw.process_logits(lg, history=hist, history_range=torch.tensor([[0, 12]] * 3, dtype=torch.int32, device="cuda"),
                      path=torch.tensor([[5, -1], [5, 6], [5, 7]], dtype=torch.int32, device="cuda"),
                      penalties=torch.tensor([[1.2, 0.1, 0.1]] * 3, device="cuda"), mask=words,
                      mask_index=torch.zeros(3, dtype=torch.int32, device="cuda"))
    tok, rng = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([1, 3], dtype=torch.int64, device="cuda")
    for r in range(3):
        qw.sample_logits(lg[r], qw.Sampling(0.0, 1, 1.0, 1.0), rng, tok)
        assert int(tok) in (65, 66, 1310)
        assert int(tok) == int(lg[r].argmax())
    b.close()
    m.close()


def test_refusals(qw):
    wl = qi.WORKLOADS["tiny"]
    host, m, b = setup(qw, wl, 4, 16)
    L = qw.lib()

    def code(call, *a):
        with pytest.raises(qw.QwError) as e:
            call(*a)
        return e.value.code
    with pytest.raises(qw.QwError):
        qw.Batch(m, 2, 16, 1)  # bf16 caches for a model with f32 ones
    with pytest.raises(qw.QwError):
        qw.Batch(m, 2, 16, 3)
    h = ctypes.c_void_p()
    n = L.qw_batch_workspace_bytes_kv(m.handle, 2, 16, 2)
    assert n > L.qw_batch_workspace_bytes_kv(m.handle, 1, 16, 2) > 0
    assert L.qw_batch_create_kv(m.handle, 2, 16, 1, b.workspace.data_ptr(), n, ctypes.byref(h)) == qw.INVALID_ARGUMENT
    assert L.qw_batch_create_kv(m.handle, 2, 16, 2, b.workspace.data_ptr(), n - 1, ctypes.byref(h)) == qw.OUT_OF_MEMORY
    assert L.qw_batch_create_kv(None, 2, 16, 2, b.workspace.data_ptr(), n, ctypes.byref(h)) == qw.INVALID_HANDLE
    assert L.qw_batch_tree_step(0x1234560, 0, 1, None, None, None) == qw.INVALID_HANDLE
    assert L.qw_batch_tree_accept(0x1234560, 0, 0, None) == qw.INVALID_HANDLE
    b.prefill(0, [1, 2, 3])
    bad = [(4, [1], [-1]), (-1, [1], [-1]), (0, [], []), (0, [1] * 5, [-1] * 5), (0, [1, 2], [-1, 1]), (0, [1, 2], [-2, 0]),
           (0, [1, -1], [-1, 0]), (0, [1, wl.vocab], [-1, 0]), (1, [-1], [-1])]
    for a in bad:
        assert code(b.tree_step, *a) == qw.INVALID_ARGUMENT, a
    with pytest.raises(ValueError):
        b.tree_step(0, [1, 2], [-1])
    assert code(b.tree_accept, 0, [0]) == qw.INVALID_ARGUMENT  # no tree waits
    b.tree_step(0, [4, 5, 6], [-1, 0, 1])
    for nodes in ([1], [0, 2], [0, 1, 1], [3], [-1], [0, 1, 2, 0]):
        assert code(b.tree_accept, 0, nodes) == qw.INVALID_ARGUMENT, nodes
    assert code(b.tree_accept, 1, [0]) == qw.INVALID_ARGUMENT
    b.tree_accept(0, [0, 1])
    assert b.length(0) == 5
    assert code(b.tree_accept, 0, [0]) == qw.INVALID_ARGUMENT  # accepted once
    b.tree_step(0, [4], [-1])
    b.step(1, [2])  # forgets the tree
    assert code(b.tree_accept, 0, [0]) == qw.INVALID_ARGUMENT
    b.tree_step(0, [4], [-1])
    b.reset(0)
    assert code(b.tree_accept, 0, [0]) == qw.INVALID_ARGUMENT
    b.prefill(0, list(range(13)))
    assert code(b.tree_step, 0, [1, 2, 3, 4], [-1, 0, 1, 2]) == qw.CONTEXT_EXCEEDED
    b.tree_step(0, [1, 2, 3], [-1, 0, 1])
    b.tree_accept(0, [0, 1, 2])
    assert b.length(0) == 16
    assert code(b.tree_step, 0, [1], [-1]) == qw.CONTEXT_EXCEEDED
    b.close()
    m.close()
