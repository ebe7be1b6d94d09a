"""Attention of batches that share a prefix (qw_prefix_attention) against its definition in 64 bits: the same
attention with the prefix written before every sequence's own positions.  Tolerances are tree attention's
(tests/test_gpu_ops.py): the arithmetic is the same, over as many keys."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import (BF16, F16, F32, TYPES, U, gen, i32, make_cache, random_tree, tolerance,  # noqa: E402
                          tree_reference, widen)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from runtime_qwen3_decode_gb300 import build, qw as binding
    build.build()
    return binding


ROOM = 60000  # the hint of a prefix of this length sends 16-bit queries to the tensor cores


def make_prefix(kind, shape, g, tc):
    """A prefix's cache; tc: with room for the hint of a long one."""
    return make_cache(kind, (shape[0], shape[1], max(shape[2], ROOM) if tc else shape[2], shape[3]), g)


def joined(pre, own, P):
    """The caches [prefix | own] of every sequence."""
    B = own[0].shape[0]
    return [None if o is None else torch.cat([p[:, :, :P].expand(B, -1, -1, -1), o], 2) for p, o in zip(pre, own)]


def run(qw, B, H, G, D, n, P, lens, counts, dt, kind, seed=0, layout="head", max_len=None, max_prefix=None, chain=False,
        room=7, ctx=None):
    g, rng = gen(300 + seed), np.random.default_rng(seed)
    ctx = ctx or max(lens) + n
    pre = make_cache(kind, (1, H, P + room, D), g, layout)
    own = make_cache(kind, (B, H, ctx, D), g, layout)
    q = (2 * torch.randn((B, n, H * G, D), generator=g, device="cuda")).to(dt)
    trees = [list(range(-1, n - 1)) if chain else random_tree(n, rng) for _ in range(B)]
    mask = torch.from_numpy(np.stack([qw.tree_mask(t) for t in trees]).view(np.int64)).cuda()
    out = torch.full_like(q, 55.0)
    qw.prefix_attention(qw.KvView(*pre), qw.KvView(*own), q, i32(*lens), i32(P), mask=None if chain else mask, out=out,
                        counts=None if counts is None else i32(*counts), max_len=max(lens) if max_len is None else max_len,
                        max_prefix=P if max_prefix is None else max_prefix)
    counts = counts or [n] * B
    total = [P + x for x in lens]
    ref, mag, vmax = tree_reference(q, joined(pre, own, P), mask, total, counts, D ** -0.5)
    tol = tolerance(dt, kind, mag, vmax, max(total) + n, D)
    for b in range(B):
        c = counts[b]
        err = (out[b, :c].double() - ref[b, :c]).abs()
        assert (err <= tol[b, :c]).all(), f"sequence {b}: {float((err - tol[b, :c]).max())} over, worst {float(err.max())}"
        assert (out[b, c:] == 55.0).all()
    return out


@pytest.mark.parametrize("dt,kind", TYPES)
@pytest.mark.parametrize("H,G,D", [(8, 2, 128), (2, 7, 64), (3, 1, 128), (8, 2, 64), (1, 64, 64)])
@pytest.mark.parametrize("max_prefix", [None, 20000])
def test_types_and_heads(qw, dt, kind, H, G, D, max_prefix):
    run(qw, 3, H, G, D, 5, 260, [130, 0, 77], [5, 2, 1], dt, kind, max_prefix=max_prefix, room=20000 if max_prefix else 7)


@pytest.mark.parametrize("dt,kind", TYPES)
@pytest.mark.parametrize("P,L", [(0, 0), (0, 5), (1, 0), (1, 1), (63, 1), (64, 64), (65, 127), (127, 128), (128, 129), (500, 0), (2100, 300)])
@pytest.mark.parametrize("max_prefix", [None, 40000])
def test_lengths(qw, dt, kind, P, L, max_prefix):
    run(qw, 4, 2, 2, 128, 1, P, [L, 0, L // 2, L], None, dt, kind, chain=True, max_prefix=max_prefix, room=40000 if max_prefix else 7)


@pytest.mark.parametrize("max_prefix", [None, 30000])  # the hint of a long prefix sends 16-bit queries to the tensor cores
@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (F16, "int8"), (F16, "f32"), (F16, "bf16"), (BF16, "int8"), (BF16, "f32")])
@pytest.mark.parametrize("B,n", [(1, 1), (2, 1), (63, 1), (64, 1), (65, 1), (130, 1), (5, 13), (7, 64), (43, 3), (3, 33)])
def test_rows_over_tiles(qw, dt, kind, B, n, max_prefix):
    """Rows of a sequence within one tile of rows, across two and across many."""
    rng = np.random.default_rng(B * n)
    run(qw, B, 2, 2, 64, n, 333, rng.integers(0, 200, B).tolist(), rng.integers(0, n + 1, B).tolist(), dt, kind, seed=n,
        max_prefix=max_prefix, room=30000 if max_prefix else 7)


@pytest.mark.parametrize("dt,kind", TYPES)
def test_long_prefix_many_sequences(qw, dt, kind):
    rng = np.random.default_rng(3)
    run(qw, 40, 4, 2, 128, 1, 9001, rng.integers(0, 700, 40).tolist(), None, dt, kind, chain=True)


@pytest.mark.parametrize("dt,kind", TYPES[3:])
@pytest.mark.parametrize("B,n,P,L", [(1, 1, 9000, 50), (8, 1, 600, 60), (8, 1, 4096, 300), (32, 1, 512, 400), (8, 4, 64, 16), (3, 2, 20000, 1)])
def test_both_sides_of_the_small_call(qw, dt, kind, B, n, P, L):
    run(qw, B, 8, 2, 128, n, P, [L] * B, None, dt, kind, chain=True)


# Most positions the sequences' own (tiles of 128 for fp16 over 8 bits), or the prefix's (of 64); ends on both sides of tiles and blocks.
@pytest.mark.parametrize("dt,kind,D", [(F16, "int8", 128), (F16, "int8", 64), (F16, "f32", 128), (F16, "f32", 64), (BF16, "f32", 128)])
@pytest.mark.parametrize("B,P,L", [(70, 0, 511), (70, 33, 450), (66, 129, 640), (40, 4033, 31), (70, 1985, 97)])
def test_tiles_of_both_sizes(qw, dt, kind, D, B, P, L):
    rng = np.random.default_rng(B + P + L)
    lens = [int(x) for x in rng.integers(0, L + 1, B)]
    lens[0], lens[-1], lens[7] = L, 64, 63
    run(qw, B, 8, 2, D, 1, P, lens, None, dt, kind, seed=L)


@pytest.mark.parametrize("dt,kind", [(F32, "int8"), (BF16, "bf16"), (F16, "int8"), (BF16, "f32")])
def test_token_major_caches(qw, dt, kind):
    run(qw, 9, 2, 4, 128, 4, 900, [0, 1, 900, 17, 300, 64, 129, 5, 128], [4, 0, 3, 4, 1, 2, 4, 2, 4], dt, kind, layout="token")


@pytest.mark.parametrize("dt,kind", TYPES)
@pytest.mark.parametrize("max_len,max_prefix", [(0, 0), (600, 0), (0, 1500)])
def test_longer_than_the_given_bounds(qw, dt, kind, max_len, max_prefix):
    run(qw, 3, 2, 2, 128, 2, 1500, [600, 3, 0], None, dt, kind, max_len=max_len, max_prefix=max_prefix)


@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (F16, "int8")])
def test_without_a_prefix_it_is_tree_attention(qw, dt, kind):
    g = gen(7)
    own, pre = make_cache(kind, (5, 2, 300, 128), g), make_cache(kind, (1, 2, 16, 128), g)
    q = torch.randn((5, 6, 4, 128), generator=g, device="cuda").to(dt)
    mask = torch.from_numpy(np.stack([qw.tree_mask([-1, 0, 0, 1, 2, 4])] * 5).view(np.int64)).cuda()
    lens = i32(290, 0, 7, 128, 255)
    a = qw.tree_attention(qw.KvView(*own), q, mask, lens).double()
    b = qw.prefix_attention(qw.KvView(*pre), qw.KvView(*own), q, lens, i32(0), mask=mask).double()
    # two roundings of the result and the same sums split in another way
    assert ((a - b).abs() <= 2 * U[dt] * a.abs() + (2 * U[dt] + 300 * 2.0 ** -24) * float(a.abs().max())).all()


@pytest.mark.parametrize("tc", [False, True])
@pytest.mark.parametrize("dt,kind", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_sequences_do_not_reach_one_another(qw, tc, dt, kind, bad):
    """What one sequence holds, and what stands behind the prefix and the sequences, reaches no other."""
    B, H, D, n, P = 6, 2, 128, 3, 200
    g = gen(11)
    pre, own = make_prefix(kind, (1, H, P + 60, D), g, tc), make_cache(kind, (B, H, 340, D), g)
    q = torch.randn((B, n, 4, D), generator=g, device="cuda").to(dt)
    lens, counts = [300, 0, 150, 128, 64, 333], [3, 3, 2, 3, 1, 3]
    mask = torch.from_numpy(np.stack([qw.tree_mask([-1, 0, 0])] * B).view(np.int64)).cuda()
    args = (qw.KvView(*pre), qw.KvView(*own), q, i32(*lens), i32(P))
    clean = qw.prefix_attention(*args, mask=mask, counts=i32(*counts)).clone()
    for t in (own[2:] if kind == "int8" else own[:2]):
        t[2, :, 17] = bad        # a cached row of sequence 2
        t[0, :, 301] = bad       # a drafted row of sequence 0: node 1's
        for b in range(B):
            t[b, :, lens[b] + counts[b]:] = bad
    for t in (pre[2:] if kind == "int8" else pre[:2]):
        t[:, :, P:] = bad
    got = qw.prefix_attention(*args, mask=mask, counts=i32(*counts))
    for b in range(B):
        for i in range(counts[b]):
            if b == 2 or (b == 0 and i == 1):
                assert not torch.isfinite(got[b, i]).all(), (b, i)
            else:
                assert torch.equal(got[b, i], clean[b, i]), (b, i)


@pytest.mark.parametrize("tc", [False, True])
@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (BF16, "int8"), (F16, "f32"), (F16, "int8")])
def test_one_bad_value_of_a_cached_v_row(qw, tc, dt, kind):
    """An element of one sequence's V that is not finite: the others keep their results, its own rows lose that element."""
    g = gen(12)
    pre, own = make_prefix(kind, (1, 1, 300, 128), g, tc), make_cache(kind, (3, 1, 200, 128), g)
    q = torch.randn((3, 1, 2, 128), generator=g, device="cuda").to(dt)
    args = (qw.KvView(*pre), qw.KvView(*own), q, i32(190, 150, 20), i32(290))
    clean = qw.prefix_attention(*args).clone()
    t = own[3] if kind == "int8" else own[1]
    t[1, 0, 40, 1] = float("nan")
    where = slice(32, 64) if kind == "int8" else slice(1, 2)
    got = qw.prefix_attention(*args)
    assert torch.isnan(got[1, 0, :, where]).all()
    keep = torch.ones(128, dtype=torch.bool, device="cuda")
    keep[where] = False
    assert torch.equal(got[1, 0][:, keep], clean[1, 0][:, keep])
    assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])


@pytest.mark.parametrize("tc", [False, True])
@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (BF16, "int8"), (F16, "f32")])
def test_rows_that_see_nothing(qw, tc, dt, kind):
    g = gen(13)
    pre, own = make_prefix(kind, (1, 2, 40, 128), g, tc), make_cache(kind, (3, 2, 70, 128), g)
    q = torch.randn((3, 4, 4, 128), device="cuda").to(dt)
    mask = torch.zeros((3, 4), dtype=torch.int64, device="cuda")
    mask[:, 2] = 0b0100
    mask[1, 3] = -(1 << 63)  # a bit behind the count: ignored
    got = qw.prefix_attention(qw.KvView(*pre), qw.KvView(*own), q, i32(0, 0, 0), i32(0), mask=mask)
    for i in (0, 1, 3):
        assert (got[:, i] == 0).all()
    v = widen(own[1][:, :, 2], None if own[3] is None else own[3][:, :, 2]).repeat_interleave(2, 1)
    assert ((got[:, 2].double() - v).abs() <= v.abs() * 2 * U[dt]).all()  # one row: its own v, rounded (twice at most)
    # with a prefix, such a row sees the prefix alone
    got = qw.prefix_attention(qw.KvView(*pre), qw.KvView(*own), q, i32(0, 0, 0), i32(1), mask=mask)
    v = widen(pre[1][0, :, 0], None if pre[3] is None else pre[3][0, :, 0]).repeat_interleave(2, 0)
    for i in (0, 1, 3):
        assert ((got[:, i].double() - v).abs() <= v.abs() * 2 * U[dt]).all()


@pytest.mark.parametrize("tc", [False, True])
@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (BF16, "int8"), (F16, "f32")])
def test_lengths_that_do_not_fit_give_nan(qw, tc, dt, kind):
    g = gen(14)
    pre, own = make_prefix(kind, (1, 2, 40, 128), g, tc), make_cache(kind, (6, 2, 40, 128), g)
    q = torch.randn((6, 4, 4, 128), device="cuda").to(dt)
    a = (qw.KvView(*pre), qw.KvView(*own), q, i32(-1, 37, 2**31 - 1, 0, 0, 36))
    got = qw.prefix_attention(*a, i32(40), counts=i32(4, 4, 4, 5, -1, 4), max_len=36)
    assert torch.isnan(got[:5]).all() and torch.isfinite(got[5]).all()
    for bad in (-1, pre[0].shape[2] + 1, 2**31 - 1):
        assert torch.isnan(qw.prefix_attention(*a, i32(bad), counts=i32(4, 4, 4, 5, -1, 4), max_len=36)).all()


@pytest.mark.parametrize("tc", [False, True])
@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (F16, "int8"), (BF16, "int8")])
@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
def test_scales(qw, tc, dt, kind, scale):
    """Scores in the thousands (the maximum moves from tile to tile and most weights underflow), equal and negative ones."""
    B, H, D, n, P = 3, 2, 128, 2, 400
    g = gen(15)
    pre, own = make_prefix(kind, (1, H, P, D), g, tc), make_cache(kind, (B, H, 300, D), g)
    q = (torch.randn((B, n, 4, D), generator=g, device="cuda") * 3).to(dt)
    got = qw.prefix_attention(qw.KvView(*pre), qw.KvView(*own), q, i32(250, 3, 0), i32(P), scale=scale)
    mask = torch.full((B, n), 3, dtype=torch.int64, device="cuda")
    mask[:, 0] = 1
    ref, mag, vmax = tree_reference(q, joined(pre, own, P), mask, [P + 250, P + 3, P], [n] * B, scale)
    err = (got.double() - ref).abs()
    assert (err <= tolerance(dt, kind, mag.abs(), vmax, P + 300, D)).all()


def test_strided_queries_and_output(qw):
    g = gen(16)
    pre, own = make_cache("bf16", (1, 4, 300, 128), g), make_cache("bf16", (2, 4, 90, 128), g)
    views = qw.KvView(*pre), qw.KvView(*own)
    for dt in (F32, BF16, F16):
        big = torch.randn((2, 3, 8 + 5, 128), generator=g, device="cuda").to(dt)  # q | k | v rows of a fused projection
        q = big[:, :, :8]
        whole = torch.full((8, 2, 3, 136), 3.0, dtype=dt, device="cuda")
        out = whole.permute(1, 2, 0, 3)[..., :128]
        qw.prefix_attention(*views, q, i32(80, 7), i32(277), out=out)
        assert torch.equal(out, qw.prefix_attention(*views, q.contiguous(), i32(80, 7), i32(277)))
        assert (whole[..., 128:] == 3.0).all()


def test_a_layer_of_larger_caches(qw):
    """Views of one layer of [layer][sequence] planes, and a prefix that is the head of one of the sequences."""
    g = gen(17)
    k, v = (torch.randn((2, 3, 4, 400, 128), generator=g, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn((3, 1, 8, 128), generator=g, device="cuda").to(BF16)
    pre = qw.KvView(k[1, :1], v[1, :1])
    own = qw.KvView(k[1, :, :, 256:], v[1, :, :, 256:])
    got = qw.prefix_attention(pre, own, q, i32(100, 0, 143), i32(256))
    full_k, full_v = k[1].clone(), v[1].clone()
    full_k[:, :, :256], full_v[:, :, :256] = k[1, :1, :, :256], v[1, :1, :, :256]
    mask = torch.ones((3, 1), dtype=torch.int64, device="cuda")
    ref, mag, vmax = tree_reference(q, [full_k, full_v, None, None], mask, [356, 256, 399], [1] * 3, 128 ** -0.5)
    assert ((got.double() - ref).abs() <= tolerance(BF16, "bf16", mag, vmax, 400, 128)).all()


@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (F16, "int8"), (F16, "f32")])
def test_same_result_every_time_on_a_stream_and_in_a_graph(qw, dt, kind):
    B, H, D, n = 20, 8, 128, 1
    g = gen(18)
    pre, own = make_cache(kind, (1, H, 3000, D), g), make_cache(kind, (B, H, 400, D), g)
    views = qw.KvView(*pre), qw.KvView(*own)
    q = torch.randn((B, n, 16, D), device="cuda").to(dt)
    lens = torch.randint(0, 399, (B,), device="cuda", dtype=torch.int32)
    plen = i32(2900)
    want = qw.prefix_attention(*views, q, lens, plen).clone()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out, scratch = torch.zeros_like(q), qw.prefix_attention_scratch(*views, n, 16)
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        qw.prefix_attention(*views, q, lens, plen, out=out, scratch=scratch, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    graphs, outs = [], [torch.zeros_like(q) for _ in range(2)]
    for o in outs:  # two graphs that share one workspace, replayed one after the other
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            qw.prefix_attention(*views, q, lens, plen, out=o, scratch=scratch)
        graphs.append(gph)
    lens.copy_(torch.randint(0, 399, (B,), device="cuda", dtype=torch.int32))  # lengths are read when the graph runs
    plen.fill_(1234)
    for _ in range(3):
        for gph in graphs:
            gph.replay()
    now = qw.prefix_attention(*views, q, lens, plen)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], now) and torch.equal(outs[1], now) and not torch.equal(now, want)


@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (F16, "int8")])
@pytest.mark.parametrize("tc", [False, True])
def test_thousands_of_sequences_most_without_rows(qw, dt, kind, tc):
    """More sequences than the tables in shared memory hold, and row tiles without any key between ones with some."""
    B, D = 9001, 64
    g = gen(21)
    pre, own = make_prefix(kind, (1, 1, 30, D), g, tc), make_cache(kind, (B, 1, 9, D), g)
    q = torch.randn((B, 1, 2, D), generator=g, device="cuda").to(dt)
    counts = torch.zeros(B, dtype=torch.int32, device="cuda")
    there = [0, 1, 63, 64, 4095, 4096, 4097, 8999, 9000]
    counts[there] = 1
    lens = torch.randint(0, 8, (B,), generator=g, device="cuda", dtype=torch.int32)
    for P in (0, 30):
        out = torch.full_like(q, 7.0)
        qw.prefix_attention(qw.KvView(*pre), qw.KvView(*own), q, lens, i32(P), out=out, counts=counts, max_len=8,
                            max_prefix=ROOM if tc else 30)
        cache = [None if o is None else torch.cat([p[:, :, :P].expand(len(there), -1, -1, -1), o[there]], 2) for p, o in zip(pre, own)]
        n = [P + int(lens[b]) for b in there]
        mask = torch.ones((len(there), 1), dtype=torch.int64, device="cuda")
        ref, mag, vmax = tree_reference(q[there], cache, mask, n, [1] * len(there), D ** -0.5)
        assert ((out[there].double() - ref).abs() <= tolerance(dt, kind, mag, vmax, max(n) + 1, D)).all()
        rest = torch.ones(B, dtype=torch.bool, device="cuda")
        rest[there] = False
        assert (out[rest] == 7.0).all()


@pytest.mark.parametrize("tc", [False, True])
def test_offsets_past_32_bits(qw, tc):
    """Sequences and heads whose rows lie more than 2^32 bytes apart."""
    g = gen(22)
    far = (1 << 31) + 64
    big = torch.empty(3 * far + 200 * 64, dtype=BF16, device="cuda")

    def plane(shape, strides, at):
        t = big.as_strided(shape, (*strides, 1), at)
        t.copy_(torch.randn(shape, generator=g, device="cuda"))
        return t
    own = [plane((3, 2, 20, 64), (far, 32 * 64, 64), 0), plane((3, 2, 20, 64), (far, 32 * 64, 64), 100 * 64)]
    room = ROOM if tc else 40
    pre = [torch.randn((1, 2, room, 64), generator=g, device="cuda").to(BF16) for _ in range(2)]
    q = torch.randn((3, 1, 4, 64), generator=g, device="cuda").to(BF16)
    lens = i32(19, 0, 7)
    got = qw.prefix_attention(qw.KvView(*pre), qw.KvView(*own), q, lens, i32(33), max_len=19, max_prefix=room)
    mask = torch.ones((3, 1), dtype=torch.int64, device="cuda")
    own += [None, None]
    ref, mag, vmax = tree_reference(q, joined(pre + [None, None], own, 33), mask, [52, 33, 40], [1] * 3, 64 ** -0.5)
    assert ((got.double() - ref).abs() <= tolerance(BF16, "bf16", mag, vmax, 53, 64)).all()
    # and a prefix whose heads lie that far apart
    pre = [plane((1, 2, 40, 64), (far, far, 64), at) for at in (0, 50 * 64)]
    near = make_cache("bf16", (3, 2, 20, 64), g)
    got = qw.prefix_attention(qw.KvView(*pre), qw.KvView(*near), q, lens, i32(33), max_len=19, max_prefix=40)
    ref, mag, vmax = tree_reference(q, joined(pre + [None, None], near, 33), mask, [52, 33, 40], [1] * 3, 64 ** -0.5)
    assert ((got.double() - ref).abs() <= tolerance(BF16, "bf16", mag, vmax, 53, 64)).all()
