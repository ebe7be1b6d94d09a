"""The operators on caller-owned buffers against plain 64-bit definitions: cache rows written and read
back (qw_kv_append, qw_kv_read), attention of drafted trees (qw_tree_attention), logits made ready for
sampling (qw_process_logits), and a run of them together.

Tolerances count roundings: u = eps / 2 of a type is the largest relative error of rounding to it.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = {t: torch.finfo(t).eps / 2 for t in (F32, F16, BF16)}


@pytest.fixture(scope="module")
def qw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from runtime_qwen3_decode_gb300 import build, qw as binding
    build.build()
    return binding


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make_cache(kind, shape, g, layout="head"):
    """Tensors (k, v, k_scale, v_scale) of a cache with random contents."""
    B, H, C, D = shape

    def lay(t):
        return t if layout == "head" else t.transpose(1, 2).contiguous().transpose(1, 2)
    if kind == "int8":
        codes = [lay(torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)) for _ in range(2)]
        scales = [lay((0.005 + 0.02 * torch.rand((B, H, C, D // 32), generator=g, device="cuda")).half()) for _ in range(2)]
        return codes + scales
    dt = {"f32": F32, "bf16": BF16}[kind]
    return [lay(torch.randn(shape, generator=g, device="cuda").to(dt)) for _ in range(2)] + [None, None]


def widen(t, s):
    """Cache rows as f64 values."""
    return t.double() if s is None else t.double() * s.double().repeat_interleave(32, -1)


# ---------------------------------------------------------------- append and read

def quantise(x):
    """The definition on numpy f32 [..., 32 n]: (codes int8, scales fp16)."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32).astype(np.float32)
    d = (np.abs(b).max(-1, keepdims=True) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(d > 0, b / d, np.float32(0)).astype(np.float64)
    c = np.clip(np.sign(r) * np.floor(np.abs(r) + 0.5), -127, 127)
    return c.reshape(x.shape).astype(np.int8), d[..., 0].astype(np.float16)


def test_definition_is_the_oracles_q8_block():
    g = np.random.default_rng(3)
    for scale in (1.0, 1e-3, 300.0):
        x = (g.standard_normal((20, 32)) * scale).astype(np.float32)
        c, s = quantise(x)
        for row, cc, ss in zip(x, c, s):
            oc, os_ = oracle.quantize_q8_block(row)
            np.testing.assert_array_equal(cc, oc)
            assert ss.view(np.uint16)[0] == os_


@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("D,n", [(128, 1), (64, 1), (128, 37), (64, 130)])
@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("kind", ["int8", "bf16", "f32"])
def test_append_and_read(qw, kind, dt, D, n, layout):
    g = gen(7)
    B, H, C = 3, 5, n + 9
    k, v, ks, vs = make_cache(kind, (B, H, C, D), g, layout)
    view = qw.KvView(k, v, ks, vs)
    start, count = i32(0, 9, 4), i32(n, n, n // 2)
    new = [torch.randn((B, n, H, D), generator=g, device="cuda").to(dt).transpose(1, 2) for _ in range(2)]
    before = [None if t is None else t.clone() for t in (k, v, ks, vs)]
    qw.kv_append(view, *new, start, count)
    outs = [torch.full((B, H, n, D), 77.0, dtype=dt, device="cuda") for _ in range(2)]
    qw.kv_read(view, *outs, start, count)
    torch.cuda.synchronize()
    for x, c, s, old_c, old_s, out in zip(new, (k, v), (ks, vs), before[:2], before[2:], outs):
        want_c, want_s = old_c.clone(), None if old_s is None else old_s.clone()
        for b in range(B):
            at, m = int(start[b]), int(count[b])
            rows = x[b, :, :m].float()
            if kind == "int8":
                qc, qs = quantise(rows.cpu().numpy())
                want_c[b, :, at:at + m] = torch.from_numpy(qc).cuda()
                want_s[b, :, at:at + m] = torch.from_numpy(qs).cuda()
            else:
                want_c[b, :, at:at + m] = rows.to(c.dtype)
        assert torch.equal(c, want_c)  # and nothing else was written
        if s is not None:
            assert torch.equal(s, want_s)
        val = widen(want_c, want_s).float()  # a code times a scale is exact in f32
        for b in range(B):
            at, m = int(start[b]), int(count[b])
            assert torch.equal(out[b, :, :m], val[b, :, at:at + m].to(dt))
            assert (out[b, :, m:] == 77.0).all()


def test_append_values_at_the_edges(qw):
    D = 64
    x = torch.zeros((1, 1, 8, D), device="cuda")
    x[0, 0, 0, :32] = torch.arange(32, device="cuda") - 15.5          # ties: amax 16.5, d = 16.5 / 127
    x[0, 0, 1, :32] = (torch.arange(32, device="cuda") % 7 - 3) * 127  # whole codes
    x[0, 0, 2, 5] = float("nan")
    x[0, 0, 3, 6] = float("inf")
    x[0, 0, 4, 7] = 127 * 65504.0 * 1.01                              # the scale overflows fp16
    x[0, 0, 5, 8] = 1e-9                                              # the scale underflows to 0
    x[0, 0, 6, :32] = -0.0
    x[0, 0, 7, :32] = torch.linspace(-3e-5, 3e-5, 32)                 # a subnormal scale
    x[0, 0, :, 32:] = 1.0
    k, v, ks, vs = make_cache("int8", (1, 1, 8, D), gen(1))
    view = qw.KvView(k, v, ks, vs)
    qw.kv_append(view, x, x, i32(0))
    out = [torch.empty_like(x) for _ in range(2)]
    qw.kv_read(view, *out, i32(0))
    o = out[0].cpu()
    assert torch.equal(o, out[1].cpu()) or torch.isnan(o).any()
    qc, qs = quantise(x.cpu().numpy()[0, 0, [0, 1, 5, 6, 7]])
    np.testing.assert_array_equal(k[0, 0, [0, 1, 5, 6, 7]].cpu().numpy(), qc)
    np.testing.assert_array_equal(ks[0, 0, [0, 1, 5, 6, 7]].cpu().numpy(), qs)
    for r in (2, 3):
        assert torch.isnan(o[0, 0, r, :32]).all()
    assert not torch.isfinite(o[0, 0, 4, 7])
    one = np.float32(127) * np.float32(np.float16(np.float32(1) / np.float32(127)))
    assert (o[0, 0, :, 32:] == float(one)).all()  # the other group is untouched by its neighbour


@pytest.mark.parametrize("dt", [F32, F16, BF16])
def test_append_codes_near_the_halves(qw, dt):
    # elements within a few ulp of every half step of their group, at scales from subnormal to large
    D, n = 128, 400
    g = np.random.default_rng(12)
    amax = (10.0 ** g.uniform(-38 if dt != F16 else -4, 6 if dt != F16 else 4, size=(n, D // 32, 1))).astype(np.float32)
    d = amax / np.float32(127)
    x = (g.integers(-127, 127, size=(n, D // 32, 32)) + 0.5).astype(np.float32) * d
    x = np.nextafter(x, np.where(g.random(x.shape) < 0.5, np.inf, -np.inf).astype(np.float32))
    x[:, :, :1] = amax
    rows = torch.from_numpy(x.reshape(1, 1, n, D)).cuda().to(dt)
    rows = torch.where(torch.isfinite(rows), rows, torch.ones_like(rows))
    k, v, ks, vs = make_cache("int8", (1, 1, n, D), gen(1))
    qw.kv_append(qw.KvView(k, v, ks, vs), rows, -rows, i32(0))
    qc, qs = quantise(rows.float().cpu().numpy())
    np.testing.assert_array_equal(k.cpu().numpy(), qc)
    np.testing.assert_array_equal(v.cpu().numpy(), -qc)
    np.testing.assert_array_equal(ks.cpu().numpy(), qs)


def test_append_leaves_a_sequence_that_does_not_fit_alone(qw):
    k, v, ks, vs = make_cache("int8", (6, 2, 8, 64), gen(2))
    view = qw.KvView(k, v, ks, vs)
    before = [t.clone() for t in (k, v, ks, vs)]
    x = torch.ones((6, 2, 3, 64), device="cuda")
    start, count = i32(-1, 6, 0, 0, 2**31 - 1, 5), i32(3, 3, 4, -1, 3, 3)
    out = [torch.full_like(x, 5.0) for _ in range(2)]
    qw.kv_read(view, *out, start, count)
    qw.kv_append(view, x, x, start, count)
    for t, b in zip((k, v, ks, vs), before):
        assert torch.equal(t[:5], b[:5])
        assert torch.equal(t[5, :, :5], b[5, :, :5]) and not torch.equal(t[5, :, 5:], b[5, :, 5:])
    assert (out[0][:5] == 5.0).all() and not (out[0][5] == 5.0).any()
    empty = torch.empty((6, 2, 0, 64), device="cuda")
    qw.kv_append(view, empty, empty, start)  # no rows: nothing to do


def test_append_twice_what_was_read_back_is_the_same(qw):
    g = gen(11)
    k, v, ks, vs = make_cache("int8", (1, 4, 50, 128), g)
    view = qw.KvView(k, v, ks, vs)
    x = [torch.randn((1, 4, 50, 128), generator=g, device="cuda") for _ in range(2)]
    qw.kv_append(view, *x, i32(0))
    first = [t.clone() for t in (k, v)]
    back = [torch.empty_like(t) for t in x]
    qw.kv_read(view, *back, i32(0))
    qw.kv_append(view, *back, i32(0))
    assert torch.equal(k, first[0]) and torch.equal(v, first[1])


# ---------------------------------------------------------------- tree attention

def random_tree(n, g):
    parents = [-1 if i == 0 or g.random() < 0.15 else int(g.integers(0, i)) for i in range(n)]
    return parents


def tree_reference(q, cache, mask, lens, counts, scale):
    """f64 [B, n, heads, D] (0 where a node sees nothing or is not there), and the bound of the scores'
    sum of magnitudes and of |v| that tolerances are made of."""
    k, v, ks, vs = cache
    B, n, heads, D = q.shape
    G = heads // k.shape[1]
    out = torch.zeros((B, n, heads, D), dtype=torch.float64, device="cuda")
    mag, vmax = torch.zeros((B, n, heads), dtype=torch.float64, device="cuda"), 0.0
    for b in range(B):
        L, c = int(lens[b]), int(counts[b])
        if c == 0:
            continue
        kk = widen(k[b, :, :L + c], None if ks is None else ks[b, :, :L + c]).repeat_interleave(G, 0)
        vv = widen(v[b, :, :L + c], None if vs is None else vs[b, :, :L + c]).repeat_interleave(G, 0)
        sees = torch.ones((c, L + c), dtype=torch.bool, device="cuda")
        for i in range(c):
            m = int(mask[b, i]) & ((1 << 64) - 1)
            sees[i, L:] = torch.tensor([(m >> j) & 1 for j in range(c)], device="cuda").bool()
        qq = q[b, :c].double().transpose(0, 1)                     # [heads, c, D]
        s = (qq @ kk.transpose(1, 2)) * scale
        s = s.masked_fill(~sees, -float("inf"))
        m = s.amax(-1, keepdim=True)
        p = torch.where(sees, torch.exp(s - torch.where(m.isinf(), 0.0, m)), 0.0)
        den = p.sum(-1, keepdim=True)
        vz = torch.nan_to_num(vv)
        o = p @ vz / torch.where(den == 0, 1.0, den)
        out[b, :c] = o.transpose(0, 1)
        mag[b, :c] = ((qq.abs() @ torch.nan_to_num(kk).abs().transpose(1, 2)).amax(-1) * scale).transpose(0, 1)
        vmax = max(vmax, float(vz.abs().max()))
    return out, mag, vmax


def tolerance(dt, kind, mag, vmax, keys, D):
    """Largest error of one output, from the roundings.  Scores are off by the D roundings of an f32 sum
    and, where K is rounded to 16 bits (an 8-bit or wider cache under 16-bit queries), by its u; a score
    error e changes a weight by a factor e^e, a weighted mean of v by at most 2 e max|v|.  The weights
    and V are rounded to 16 bits (u each), exp2 is off by 2^-21, sums of `keys` f32 terms by keys 2^-24,
    the output by its own u."""
    u = 0.0 if dt == F32 else U[BF16 if kind == "bf16" and dt == BF16 else dt]
    k_rounds = dt != F32 and not (kind == "bf16" and dt == BF16)
    score = mag * ((D + 4) * 2.0 ** -24 + (u if k_rounds else 0.0))
    rel = 2 * score + 2 * u + U[dt] + 2.0 ** -20 + keys * 2.0 ** -24
    return (rel * vmax)[..., None]


def run_tree(qw, B, H, G, D, n, lens, counts, dt, kind, seed=0, layout="head", max_len=None, ctx=None):
    g, rng = gen(100 + seed), np.random.default_rng(seed)
    ctx = ctx or max(lens) + n
    cache = make_cache(kind, (B, H, ctx, D), g, layout)
    view = qw.KvView(*cache)
    q = (2 * torch.randn((B, n, H * G, D), generator=g, device="cuda")).to(dt)
    mask = torch.from_numpy(np.stack([qw.tree_mask(random_tree(n, rng)) for _ in range(B)]).view(np.int64)).cuda()
    out = torch.full_like(q, 55.0)
    got = qw.tree_attention(view, q, mask, i32(*lens), out, counts=None if counts is None else i32(*counts),
                            max_len=max(lens) if max_len is None else max_len)
    counts = counts or [n] * B
    ref, mag, vmax = tree_reference(q, cache, mask, lens, counts, D ** -0.5)
    tol = tolerance(dt, kind, mag, vmax, max(lens) + n, D)
    for b in range(B):
        c = counts[b]
        err = (got[b, :c].double() - ref[b, :c]).abs()
        assert (err <= tol[b, :c]).all(), f"sequence {b}: {float((err - tol[b, :c]).max())} over, worst {float(err.max())}"
        assert (got[b, c:] == 55.0).all()
    return got


TYPES = [(F32, "f32"), (F32, "bf16"), (F32, "int8"), (F16, "f32"), (F16, "bf16"), (F16, "int8"), (BF16, "f32"),
         (BF16, "bf16"), (BF16, "int8")]


@pytest.mark.parametrize("dt,kind", TYPES)
@pytest.mark.parametrize("H,G,D", [(8, 2, 128), (2, 7, 64), (3, 1, 128)])
def test_tree_types_and_heads(qw, dt, kind, H, G, D):
    run_tree(qw, 3, H, G, D, 9, [130, 0, 77], [9, 5, 1], dt, kind)


@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (F16, "int8"), (BF16, "f32")])
@pytest.mark.parametrize("n,L", [(1, 0), (1, 1), (1, 63), (1, 64), (1, 65), (2, 127), (3, 128), (8, 511), (33, 1), (63, 95),
                                 (64, 0), (64, 64), (64, 1500)])
def test_tree_lengths(qw, dt, kind, n, L):
    run_tree(qw, 1, 2, 2, 128, n, [L], None, dt, kind, seed=n)


@pytest.mark.parametrize("dt,kind", [(F32, "int8"), (BF16, "bf16"), (F16, "int8"), (F16, "f32")])
def test_tree_ragged_batch_token_major(qw, dt, kind):
    lens = [0, 1, 900, 17, 2047, 300, 64, 129, 1024]
    run_tree(qw, 9, 2, 4, 128, 17, lens, [17, 0, 3, 17, 1, 9, 16, 2, 17], dt, kind, layout="token")


@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (BF16, "int8")])
def test_tree_many_rows_per_kv_head(qw, dt, kind):
    run_tree(qw, 1, 1, 9, 128, 61, [333], None, dt, kind)  # 549 query rows share a KV head
    run_tree(qw, 2, 1, 64, 64, 3, [100, 7], None, dt, kind)


@pytest.mark.parametrize("dt,kind", [(F32, "bf16"), (BF16, "bf16"), (BF16, "int8")])
def test_tree_longer_than_the_given_bound(qw, dt, kind):
    run_tree(qw, 2, 2, 2, 128, 5, [700, 3], None, dt, kind, max_len=1)
    run_tree(qw, 2, 2, 2, 128, 5, [700, 3], None, dt, kind, max_len=700)


@pytest.mark.parametrize("dt,kind", TYPES)
def test_tree_long_contexts_of_many_tiles(qw, dt, kind):
    # every CTA works through several tiles of several items, whole and cut ones
    run_tree(qw, 3, 8, 2, 128, 21, [9000, 1, 4321], [21, 20, 3], dt, kind, ctx=9100)


@pytest.mark.parametrize("dt,kind", TYPES[3:])
@pytest.mark.parametrize("B,n,L", [(1, 1, 3600), (1, 1, 5000), (4, 1, 500), (4, 1, 1200), (1, 4, 900), (1, 4, 2500), (1, 5, 100), (1, 8, 1000), (1, 8, 1400)])
def test_tree_few_rows_on_both_sides_of_the_small_call(qw, dt, kind, B, n, L):
    run_tree(qw, B, 8, 2, 128, n, [L] * B, None, dt, kind)


@pytest.mark.parametrize("dt,kind", [(F32, "int8"), (BF16, "bf16"), (F16, "int8")])
def test_tree_more_sequences_than_a_warp(qw, dt, kind):
    rng = np.random.default_rng(5)
    lens, counts = rng.integers(0, 500, 70).tolist(), rng.integers(0, 5, 70).tolist()
    run_tree(qw, 70, 2, 2, 64, 4, lens, counts, dt, kind)


def test_tree_one_node_is_decode_attention(qw):
    # a chain of one: softmax over the cache and the node's own row
    run_tree(qw, 8, 8, 2, 128, 1, [511, 0, 1, 130, 200, 64, 65, 400], None, F32, "f32")
    run_tree(qw, 8, 8, 2, 128, 1, [511, 0, 1, 130, 200, 64, 65, 400], None, BF16, "bf16")


@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (F16, "int8"), (BF16, "bf16"), (BF16, "int8"), (F16, "f32")])
def test_tree_rows_that_see_nothing(qw, dt, kind):
    cache = make_cache(kind, (2, 2, 70, 128), gen(3))
    q = torch.randn((2, 6, 4, 128), device="cuda").to(dt)
    mask = torch.zeros((2, 6), dtype=torch.int64, device="cuda")
    mask[:, 3] = 0b1000
    mask[0, 4] = -(1 << 63)  # a bit behind the count: ignored
    got = qw.tree_attention(qw.KvView(*cache), q, mask, i32(0, 0))
    for i in (0, 1, 2, 4, 5):
        assert (got[:, i] == 0).all()
    v = widen(cache[1][:, :, 3], None if cache[3] is None else cache[3][:, :, 3]).repeat_interleave(2, 1)
    assert ((got[:, 3].double() - v).abs() <= v.abs() * 2 * U[dt]).all()  # one row: its own v, rounded (twice at most)


@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (F32, "int8"), (BF16, "bf16"), (BF16, "int8"), (F16, "f32"), (F16, "bf16")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_tree_what_is_not_seen_does_not_reach(qw, dt, kind, bad):
    B, H, D, n, L = 2, 2, 128, 12, 150
    cache = make_cache(kind, (B, H, L + 40, D), gen(4))
    view = qw.KvView(*cache)
    q = torch.randn((B, n, 4, D), device="cuda").to(dt)
    lens, counts = [L, 90], [n, 7]
    parents = [-1, 0, 0, 1, 1, 2, 2, 3, 4, 5, 6, 7]
    mask = torch.from_numpy(np.stack([qw.tree_mask(parents)] * B).view(np.int64)).cuda()
    clean = qw.tree_attention(view, q, mask, i32(*lens), counts=i32(*counts)).clone()
    # behind the drafted rows, and in the drafted node 4 (seen by 4 and 8 only)
    hit = cache[2:] if kind == "int8" else cache[:2]
    for t in hit:
        for b in range(B):
            t[b, :, lens[b] + counts[b]:] = bad
            t[b, :, lens[b] + 4] = bad
    got = qw.tree_attention(view, q, mask, i32(*lens), counts=i32(*counts))
    for b in range(B):
        for i in range(counts[b]):
            if i in (4, 8):
                assert not torch.isfinite(got[b, i]).any()
            else:
                assert torch.equal(got[b, i], clean[b, i]), (b, i)


@pytest.mark.parametrize("dt,kind", [(F32, "bf16"), (BF16, "bf16"), (BF16, "int8")])
def test_tree_one_bad_value_of_a_drafted_v_row(qw, dt, kind):
    cache = make_cache(kind, (1, 1, 140, 128), gen(5))
    q = torch.randn((1, 4, 2, 128), device="cuda").to(dt)
    mask = torch.from_numpy(qw.tree_mask([-1, 0, -1, 2]).view(np.int64)).cuda()[None]
    view = qw.KvView(*cache)
    clean = qw.tree_attention(view, q, mask, i32(133)).clone()
    t = cache[3] if kind == "int8" else cache[1]
    t[0, 0, 134, 1] = float("nan")  # node 1's V: element 1, or its second group
    where = slice(32, 64) if kind == "int8" else slice(1, 2)
    got = qw.tree_attention(view, q, mask, i32(133))
    assert torch.isnan(got[0, 1, :, where]).all()
    keep = torch.ones(128, dtype=torch.bool, device="cuda")
    keep[where] = False
    assert torch.equal(got[0, 1][:, keep], clean[0, 1][:, keep])
    for i in (0, 2, 3):
        assert torch.equal(got[0, i], clean[0, i])


@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (BF16, "int8")])
def test_tree_lengths_that_do_not_fit_give_nan(qw, dt, kind):
    cache = make_cache(kind, (6, 2, 40, 128), gen(6))
    q = torch.randn((6, 4, 4, 128), device="cuda").to(dt)
    mask = torch.full((6, 4), 15, dtype=torch.int64, device="cuda")
    got = qw.tree_attention(qw.KvView(*cache), q, mask, i32(-1, 37, 2**31 - 1, 0, 0, 36), counts=i32(4, 4, 4, 5, -1, 4), max_len=36)
    assert torch.isnan(got[:5]).all() and torch.isfinite(got[5]).all()


@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (F16, "int8")])
def test_tree_large_scores(qw, dt, kind):
    # scores in the thousands: the maximum moves from tile to tile and most weights underflow
    B, H, D, n, L = 1, 2, 128, 5, 400
    cache = make_cache(kind, (B, H, L + n, D), gen(8))
    q = (torch.randn((B, n, 4, D), generator=gen(9), device="cuda") * 40).to(dt)
    mask = torch.from_numpy(qw.tree_mask(range(-1, n - 1)).view(np.int64)).cuda()[None]
    got = qw.tree_attention(qw.KvView(*cache), q, mask, i32(L))
    ref, mag, vmax = tree_reference(q, cache, mask, [L], [n], D ** -0.5)
    assert torch.isfinite(got).all()
    err = (got.double() - ref).abs()
    assert (err <= tolerance(dt, kind, mag, vmax, L + n, D)).all()


def test_tree_strided_queries_and_output(qw):
    g = gen(10)
    cache = make_cache("bf16", (2, 4, 90, 128), g)
    view = qw.KvView(*cache)
    mask = torch.full((2, 3), 7, dtype=torch.int64, device="cuda")
    for dt in (F32, BF16, F16):
        big = torch.randn((2, 3, 8 + 5, 128), generator=g, device="cuda").to(dt)  # q | k | v rows of a fused projection
        q = big[:, :, :8]
        whole = torch.full((8, 2, 3, 136), 3.0, dtype=dt, device="cuda")
        out = whole.permute(1, 2, 0, 3)[..., :128]
        qw.tree_attention(view, q, mask, i32(80, 7), out)
        want = qw.tree_attention(view, q.contiguous(), mask, i32(80, 7))
        assert torch.equal(out, want)
        assert (whole[..., 128:] == 3.0).all()


@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (BF16, "bf16"), (F16, "int8")])
def test_tree_same_result_every_time_on_a_stream_and_in_a_graph(qw, dt, kind):
    B, H, D, n = 4, 8, 128, 16
    cache = make_cache(kind, (B, H, 1200, D), gen(12))
    view = qw.KvView(*cache)
    q = torch.randn((B, n, 16, D), device="cuda").to(dt)
    mask = torch.from_numpy(np.stack([qw.tree_mask(range(-1, n - 1))] * B).view(np.int64)).cuda()
    lens = i32(1100, 3, 640, 1024)
    want = qw.tree_attention(view, q, mask, lens).clone()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out, scratch = torch.zeros_like(q), qw.tree_attention_scratch(view, n, 16)
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        qw.tree_attention(view, q, mask, lens, out, scratch=scratch, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    graphs, outs = [], [torch.zeros_like(q) for _ in range(2)]
    for o in outs:  # two graphs that share one workspace, replayed one after the other
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            qw.tree_attention(view, q, mask, lens, o, scratch=scratch)
        graphs.append(gph)
    lens.copy_(i32(900, 77, 0, 1184))  # the lengths are read when the graph runs
    for _ in range(3):
        for gph in graphs:
            gph.replay()
    now = qw.tree_attention(view, q, mask, lens)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], now) and torch.equal(outs[1], now) and not torch.equal(now, want)


def test_tree_makes_its_result_on_the_stream_that_it_runs_on(qw):
    view = qw.KvView(*make_cache("int8", (2, 2, 300, 64), gen(13)))
    q = torch.randn((2, 5, 4, 64), device="cuda").to(BF16)
    mask = torch.full((2, 5), 31, dtype=torch.int64, device="cuda")
    lens = i32(290, 0)
    want = qw.tree_attention(view, q, mask, lens).clone()
    busy = torch.ones(1 << 26, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(100):  # some 10 ms of work on the current stream, which the call does not wait for
        busy.mul_(1.0)
    out = qw.tree_attention(view, q, mask, lens, stream=st)
    st.synchronize()
    early = torch.empty_like(out)
    with torch.cuda.stream(st):
        early.copy_(out)
    torch.cuda.synchronize()
    assert torch.equal(early, want) and torch.equal(out, want)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_cache_offsets_past_32_bits(qw, dt):
    D, C = 64, (1 << 26) + 100  # 4.3 GB of codes per plane
    k, v = (torch.zeros((1, 1, C, D), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((1, 1, C, D // 32), dtype=F16, device="cuda") for _ in range(2))
    view = qw.KvView(k, v, ks, vs)
    x = [torch.randn((1, 1, 4, D), generator=gen(1), device="cuda") for _ in range(2)]
    L = C - 4
    qw.kv_append(view, *x, i32(L))
    back = [torch.empty_like(t) for t in x]
    qw.kv_read(view, *back, i32(L))
    qc, qs = quantise(x[0].cpu().numpy())
    np.testing.assert_array_equal(back[0].cpu().numpy(), qc.astype(np.float32) * np.repeat(qs.astype(np.float32), 32, -1))
    # every cached row is zero: score 0 and value 0; node i sees itself alone of the drafted rows.  Its
    # query makes its own score large, so that the row's weight is not lost among 2^26 zeros.
    q = torch.zeros((1, 4, 1, D), device="cuda", dtype=dt)
    kr = back[0][0, 0]
    q[0, :, 0] = (kr / kr.norm(dim=-1, keepdim=True) ** 2 * 40 * D ** 0.5).to(dt)
    mask = torch.tensor([[1, 2, 4, 8]], dtype=torch.int64, device="cuda")
    got = qw.tree_attention(view, q, mask, i32(L))
    # weight of the own row: e^40 / (e^40 + 2^26), 1 within 2^-24
    tol = 2 * U[dt] + (2.0 ** -9 if dt != F32 else 2.0 ** -18)
    assert ((got[0, :, 0].double() - back[1][0, 0].double()).abs() <= tol * back[1].abs().max()).all()


# ---------------------------------------------------------------- logits

def logits_reference(x, pen, hist, hrange, path, bids, bias, brange, mask, mindex):
    R, V = x.shape
    out = x.double().cpu().numpy().copy()
    for r in range(R):
        ids = []
        if hist is not None:
            ids += hist[max(0, hrange[r][0]):max(0, min(len(hist), hrange[r][1]))].tolist()
        if path is not None:
            ids += path[r].tolist()
        if pen is not None:
            rep, pres, freq = (float(t) for t in pen[r])
            for t in set(i for i in ids if 0 <= i < V):
                z = out[r, t]
                z = z / rep if z > 0 else z * rep
                out[r, t] = z - pres - freq * ids.count(t)
        if bids is not None:
            for i in range(max(0, brange[r][0]), min(len(bids), brange[r][1])):
                if 0 <= bids[i] < V:
                    out[r, bids[i]] += float(bias[i])
        if mask is not None:
            m = r if mindex is None else int(mindex[r])
            if m >= mask.shape[0]:
                out[r] = -np.inf
            elif m >= 0:
                bits = np.unpackbits(mask[m].view(np.uint8), bitorder="little")[:V]
                out[r, bits == 0] = -np.inf
    return out


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make_logits(R, V, seed, n_hist=60, n_bias=20, n_masks=2):
    g = np.random.default_rng(seed)
    hist = g.integers(-3, V + 3, size=n_hist).astype(np.int32)
    hist[: n_hist // 2] = g.integers(0, min(V, 9), size=n_hist // 2)
    b = g.integers(0, n_hist, size=R)
    hr = np.stack([b, b + g.integers(0, n_hist, size=R)], 1).astype(np.int32)  # some run past the array
    path = g.integers(-1, V, size=(R, 5)).astype(np.int32)
    pen = np.stack([1 + g.random(R), g.random(R), 0.3 * g.random(R)], 1).astype(np.float32)
    bids = g.integers(-2, V + 2, size=n_bias).astype(np.int32)
    bids[::3] = bids[0]  # one id many times
    bias = (3 * g.standard_normal(n_bias)).astype(np.float32)
    bb = g.integers(0, n_bias // 2, size=R)
    br = np.stack([bb, bb + n_bias // 2 + 4], 1).astype(np.int32)
    mask = g.integers(-2**31, 2**31, size=(n_masks, (V + 31) // 32)).astype(np.int32)
    mi = g.integers(-1, n_masks, size=R).astype(np.int32)
    return pen, hist, hr, path, bids, bias, br, mask, mi


def call_logits(qw, x, parts, out=None):
    pen, hist, hr, path, bids, bias, br, mask, mi = parts
    return qw.process_logits(x, out, penalties=dev(pen), history=dev(hist), history_range=dev(hr), path=dev(path),
                             bias_ids=dev(bids), bias=dev(bias), bias_range=dev(br), mask=dev(mask), mask_index=dev(mi))


def check_logits(got, ref, x, parts, dt):
    """Every value takes at most five f32 roundings (the penalty's product or quotient, the frequency's
    product, two sums, each bias) of terms no larger than the sum of magnitudes, then the output's own."""
    big = x.double().abs().cpu().numpy() * 2 + 2 + 0.3 * 70 + 3 * 6 * 30
    big = np.where(np.isfinite(big), big, 0)
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf])
    ok = np.isfinite(ref)
    tol = 30 * 2.0 ** -24 * big + np.abs(np.where(ok, ref, 0)) * (0 if dt == F32 else U[dt])
    assert (np.abs(got - ref)[ok] <= tol[ok]).all()


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("R,V", [(1, 1), (3, 31), (2, 100), (4, 2048), (3, 2049), (5, 8191), (2, 8193), (1, 30001), (40, 151936)])
def test_logits(qw, dt, R, V):
    x = (3 * torch.randn((R, V), generator=gen(V), device="cuda")).to(dt)
    parts = make_logits(R, V, V + R)
    keep = x.clone()
    out = torch.empty_like(x)
    call_logits(qw, x, parts, out)
    assert torch.equal(x, keep)
    check_logits(out, logits_reference(keep, *parts), keep, parts, dt)
    assert call_logits(qw, x, parts) is x  # in place: the same values
    assert torch.equal(x, out)


@pytest.mark.parametrize("drop", ["pen", "hist", "path", "bias", "mask", "mindex", "all"])
def test_logits_optional_parts(qw, drop):
    R, V = 3, 9001
    pen, hist, hr, path, bids, bias, br, mask, mi = make_logits(R, V, 5, n_masks=3)
    if drop in ("pen", "all"):
        pen = None
    if drop in ("hist", "all"):
        hist = hr = None
    if drop in ("path", "all"):
        path = None
    if drop in ("bias", "all"):
        bids = bias = br = None
    if drop in ("mask", "all"):
        mask = mi = None
    if drop == "mindex":
        mi = None
    parts = (pen, hist, hr, path, bids, bias, br, mask, mi)
    x = torch.randn((R, V), generator=gen(3), device="cuda")
    keep = x.clone()
    check_logits(call_logits(qw, x, parts), logits_reference(keep, *parts), keep, parts, F32)


def test_logits_special_values_and_masks(qw):
    V = 300
    x = torch.randn((4, V), device="cuda")
    x[:, 3], x[:, 4], x[:, 5] = float("nan"), float("inf"), -float("inf")
    x[:, 6], x[:, 7] = -0.0, 0.0
    g = np.random.default_rng(1)
    hist = np.arange(0, 10, dtype=np.int32)
    hr = np.array([[0, 10]] * 4, np.int32)
    pen = np.array([[1.5, 0.0, 0.0]] * 4, np.float32)
    bids, bias = np.array([8, 9, 8], np.int32), np.array([-np.inf, 2.0, 5.0], np.float32)
    br = np.array([[0, 3]] * 4, np.int32)
    mask = g.integers(-2**31, 2**31, size=(2, 10)).astype(np.int32)
    mask[1] = 0  # forbids everything
    mi = np.array([-1, 0, 1, 2], np.int32)  # 2: past the masks
    parts = (pen, hist, hr, None, bids, bias, br, mask, mi)
    keep = x.clone()
    got = call_logits(qw, x, parts)
    check_logits(got, logits_reference(keep, *parts), keep, parts, F32)
    assert (got[2:] == -float("inf")).all()
    assert (got[0, 8] == -float("inf")).all()


def test_logits_ranges_outside_the_lists(qw):
    V, top = 3000, 2**31 - 1
    pen, hist, hr, path, bids, bias, br, mask, mi = make_logits(6, V, 8)
    hr[:] = [[-5, 10], [top, top], [top, -top], [0, top], [-top, 7], [59, 58]]
    br[:] = [[-1, 3], [top, top], [4, top], [-top, -3], [19, 20], [20, 5]]
    parts = (pen, hist, hr, path, bids, bias, br, mask, mi)
    x = torch.randn((6, V), generator=gen(3), device="cuda")
    keep = x.clone()
    check_logits(call_logits(qw, x, parts), logits_reference(keep, *parts), keep, parts, F32)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_logits_rows_off_vector_boundaries(qw, dt):
    R, V = 3, 5000
    whole = torch.randn((R, V + 7), generator=gen(2), device="cuda").to(dt)
    parts = make_logits(R, V, 9)
    for off, at, wide in ((0, 2, 9), (1, 2, 9), (3, 2, 9), (1, 1, 7), (2, 2, 7), (3, 3, 7), (2, 6, 11)):
        x = whole[:, off:off + V]
        dst = torch.full((R, V + wide), 9.0, dtype=dt, device="cuda")
        out = dst[:, at:at + V]
        call_logits(qw, x, parts, out)
        check_logits(out, logits_reference(x.clone(), *parts), x.clone(), parts, dt)
        assert (dst[:, :at] == 9.0).all() and (dst[:, at + V:] == 9.0).all()


def test_logits_a_bias_named_many_times_is_summed_in_order(qw):
    V, n = 64, 1500
    g = np.random.default_rng(4)
    bids = g.integers(0, 3, size=n).astype(np.int32)
    bias = (1e3 * g.standard_normal(n)).astype(np.float32)
    br = np.array([[0, n]], np.int32)
    want = np.zeros(V, np.float32)
    for i, b in zip(bids, bias):
        want[i] = np.float32(want[i] + b) if want[i] != 0 else b
    for _ in range(3):
        x = torch.zeros((1, V), device="cuda")
        qw.process_logits(x, bias_ids=dev(bids), bias=dev(bias), bias_range=dev(br))
        np.testing.assert_array_equal(x[0].cpu().numpy(), want)


@pytest.mark.parametrize("R,V,n_hist,n_bias", [(3, 40000, 6000, 20), (2, 5000, 20, 3000), (70, 17000, 1500, 700)])
def test_logits_long_lists(qw, R, V, n_hist, n_bias):
    # more entries for a CTA's tokens than it keeps apart
    x = 3 * torch.randn((R, V), generator=gen(V), device="cuda")
    pen, hist, hr, path, bids, bias, br, mask, mi = make_logits(R, V, R, n_hist=n_hist, n_bias=n_bias)
    hr[:, 0], hr[:, 1] = 0, n_hist
    bias = (bias / 100).astype(np.float32)
    br[:, 0], br[:, 1] = 0, n_bias
    parts = (pen, hist, hr, path, bids, bias, br, mask, mi)
    keep = x.clone()
    got = call_logits(qw, x, parts)
    ref = logits_reference(keep, *parts)
    # frequency * count grows with the list: counts up to n_hist, each product and sum rounded once;
    # a bias sum of n_bias terms up to 0.15 each is off by at most n_bias^2 0.15 2^-24
    got = got.double().cpu().numpy()
    ok = np.isfinite(ref)
    assert np.array_equal(got[~ok], ref[~ok])
    tol = 8 * 2.0 ** -24 * (40 + 0.3 * n_hist) + n_bias ** 2 * 0.15 * 2.0 ** -24
    assert np.abs(got[ok] - ref[ok]).max() <= tol


def test_logits_captured(qw):
    x = torch.randn((4, 20000), device="cuda")
    parts = make_logits(4, 20000, 21)
    names = ("penalties", "history", "history_range", "path", "bias_ids", "bias", "bias_range", "mask", "mask_index")
    args = {k: dev(p) for k, p in zip(names, parts)}
    want = qw.process_logits(x, torch.empty_like(x), **args)
    out = torch.zeros_like(x)
    torch.cuda.synchronize()
    gph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gph):
        qw.process_logits(x, out, **args)
    for _ in range(2):
        gph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ---------------------------------------------------------------- refusals of the binding

def test_binding_refusals(qw):
    k, v, ks, vs = make_cache("int8", (2, 2, 16, 64), gen(1))
    with pytest.raises(ValueError):
        qw.KvView(k, v)
    with pytest.raises(ValueError):
        qw.KvView(k.cpu(), v.cpu(), ks, vs)
    with pytest.raises(ValueError):
        qw.KvView(k, v, ks.float(), vs.float())
    with pytest.raises(ValueError):
        qw.KvView(k, v[:, :, :8], ks, vs)
    with pytest.raises(ValueError):
        qw.KvView(k.float(), v.float(), ks, vs)
    with pytest.raises(ValueError):
        qw.KvView(k.half(), v.half())
    view = qw.KvView(k, v, ks, vs)
    x = torch.zeros((2, 2, 3, 64), device="cuda")
    for bad in ((x.double(), x.double()), (x, x.half()), (x[:1], x[:1]), (x[..., :32], x[..., :32]), (x.cpu(), x.cpu())):
        with pytest.raises(ValueError):
            qw.kv_append(view, *bad, i32(0, 0))
    for bad in (i32(0), torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(ValueError):
            qw.kv_append(view, x, x, bad)
        with pytest.raises(ValueError):
            qw.kv_read(view, x, x, i32(0, 0), bad)
    q = torch.zeros((2, 3, 4, 64), device="cuda")
    m = torch.zeros((2, 3), dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        qw.tree_attention(view, q, m[:, :2], i32(0, 0))
    with pytest.raises(ValueError):
        qw.tree_attention(view, q[:1], m, i32(0, 0))
    with pytest.raises(ValueError):
        qw.tree_attention(view, q, m, i32(0, 0), out=q.half())
    with pytest.raises(qw.QwError) as e:
        qw.tree_attention(view, q, m, i32(0, 0), scratch=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == qw.OUT_OF_MEMORY
    with pytest.raises(qw.QwError) as e:
        qw.tree_attention(view, torch.zeros((2, 3, 3, 64), device="cuda"), m, i32(0, 0))
    assert e.value.code == qw.UNSUPPORTED_SHAPE
    y = torch.zeros((2, 50), device="cuda")
    for bad in (dict(history=i32(1)), dict(penalties=torch.ones((1, 3), device="cuda")), dict(mask_index=i32(0, 0)),
                dict(mask=torch.zeros((1, 1), dtype=torch.int32, device="cuda")), dict(bias_ids=i32(1)), dict(path=i32(1))):
        with pytest.raises(ValueError):
            qw.process_logits(y, **bad)


def test_results_over_one_another_and_empty_masks_are_refused(qw):
    view = qw.KvView(*make_cache("int8", (2, 2, 16, 64), gen(1)))
    x = torch.zeros((2, 2, 3, 64), device="cuda")
    wide = x[:, :1].expand(2, 2, 3, 64)
    qw.kv_append(view, wide, wide, i32(0, 0))  # one row for every head is a source like another
    with pytest.raises(qw.QwError) as e:
        qw.kv_read(view, wide, wide, i32(0, 0))
    assert e.value.code == qw.INVALID_ARGUMENT
    q = torch.zeros((2, 3, 4, 64), device="cuda")
    with pytest.raises(qw.QwError) as e:
        qw.tree_attention(view, q, torch.zeros((2, 3), dtype=torch.int64, device="cuda"), i32(0, 0), out=q[:1].expand(2, 3, 4, 64))
    assert e.value.code == qw.INVALID_ARGUMENT
    with pytest.raises(ValueError):
        qw.process_logits(torch.zeros((2, 50), device="cuda"), mask=torch.zeros((0, 2), dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dt,kind", [(F32, "int8"), (BF16, "int8"), (BF16, "bf16")])
def test_a_tree_gives_what_each_of_its_paths_gives(qw, dt, kind):
    """Append a tree and attend, against appending each node's path as a chain on its own copy of the
    cache; the nodes' logits are then prepared and sampled."""
    g = gen(31)
    B, H, G, D, n, L = 2, 2, 2, 128, 7, 140
    parents = [-1, 0, 0, 1, 2, 4, -1]
    cache = make_cache(kind, (B, H, L + n, D), g)
    rows = [torch.randn((B, n, H, D), generator=g, device="cuda").to(dt) for _ in range(2)]
    q = torch.randn((B, n, H * G, D), generator=g, device="cuda").to(dt)
    view = qw.KvView(*cache)
    lens = i32(L, 33)
    before = [None if t is None else t.clone() for t in cache]
    qw.kv_append(view, rows[0].transpose(1, 2), rows[1].transpose(1, 2), lens)
    mask = torch.from_numpy(np.stack([qw.tree_mask(parents)] * B).view(np.int64)).cuda()
    tree = qw.tree_attention(view, q, mask, lens)
    ref, mag, vmax = tree_reference(q, cache, mask, [L, 33], [n, n], D ** -0.5)
    tol = tolerance(dt, kind, mag, vmax, L + n, D)
    for i in range(n):
        path, j = [], i
        while j >= 0:
            path.insert(0, j)
            j = parents[j]
        copy = [None if t is None else t.clone() for t in before]
        chain = qw.KvView(*copy)
        qw.kv_append(chain, rows[0][:, path].transpose(1, 2), rows[1][:, path].transpose(1, 2), lens)
        m = torch.from_numpy(np.stack([qw.tree_mask(range(-1, len(path) - 1))] * B).view(np.int64)).cuda()
        one = qw.tree_attention(chain, q[:, path].contiguous(), m, lens)
        assert ((one[:, -1].double() - tree[:, i].double()).abs() <= 2 * tol[:, i]).all()
    V = 500
    logits = (tree.float().reshape(B * n, -1) @ torch.randn((H * G * D, V), generator=g, device="cuda") / 10).contiguous()
    allowed = torch.full((1, (V + 31) // 32), 0, dtype=torch.int32, device="cuda")
    allowed[0, 3] = 0b1010  # tokens 97 and 99
    qw.process_logits(logits, mask=allowed, mask_index=torch.zeros(B * n, dtype=torch.int32, device="cuda"))
    rng = torch.tensor([1, 3], dtype=torch.int64, device="cuda")
    tok = i32(-1)
    for r in range(B * n):
        qw.sample_logits(logits[r], qw.Sampling(0.0, 1, 1.0, 1.0), rng, tok)
        assert int(tok) in (97, 99)
