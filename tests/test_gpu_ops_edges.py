"""The operators on caller-owned buffers where their types, strides and lengths end: rows on the smallest
alignment, values at the edges of the types, long contexts, and errors no larger than the number formats of
the operands leave.

Tolerances count roundings: u = eps / 2 of a type is the largest relative error of rounding to it.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import BF16, F16, F32, U, gen, i32, make_cache, quantise, tree_reference, widen  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from runtime_qwen3_decode_gb300 import build, qw as binding
    build.build()
    return binding


# ---------------------------------------------------------------- append and read

@pytest.mark.parametrize("kind", ["f32", "bf16", "int8"])
@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("D,n", [(128, 3), (64, 300)])
def test_rows_on_16_byte_boundaries_and_no_larger_ones(qw, kind, dt, D, n):
    # the cache and the rows begin 16 bytes behind a larger boundary, and their rows are 16 bytes longer
    B, H, C = 2, 3, n + 5
    ct = {"f32": F32, "bf16": BF16, "int8": torch.int8}[kind]

    def off(shape, t):
        unit = 16 // torch.empty((), dtype=t).element_size()
        whole = torch.zeros(int(np.prod(shape[:-1])) * (shape[-1] + unit) + unit, dtype=t, device="cuda")
        x = whole[unit:].view(*shape[:-1], shape[-1] + unit)[..., :shape[-1]]
        assert x.data_ptr() % 32 == 16
        return x
    k, v = off((B, H, C, D), ct), off((B, H, C, D), ct)
    ks, vs = (torch.zeros((B, H, C, D // 32), dtype=F16, device="cuda") for _ in range(2)) if kind == "int8" else (None, None)
    view = qw.KvView(k, v, ks, vs)
    rows = [off((B, H, n, D), dt) for _ in range(2)]
    for i, r in enumerate(rows):
        r.copy_(torch.randn((B, H, n, D), generator=gen(40 + i), device="cuda").to(dt))
    outs = [off((B, H, n, D), dt) for _ in range(2)]
    start = i32(5, 2)
    qw.kv_append(view, *rows, start)
    qw.kv_read(view, *outs, start)
    for r, c, s, o in zip(rows, (k, v), (ks, vs), outs):
        for b, at in enumerate((5, 2)):
            x = r[b].float()
            if kind == "int8":
                qc, qs = quantise(x.cpu().numpy())
                want = torch.from_numpy(qc).cuda(), torch.from_numpy(qs).cuda()
                assert torch.equal(s[b, :, at:at + n], want[1])
                val = widen(*want).float()
            else:
                want = (x.to(ct),)
                val = want[0].float()
            assert torch.equal(c[b, :, at:at + n], want[0])
            assert torch.equal(o[b], val.to(dt))


@pytest.mark.parametrize("dt", [F32, F16, BF16])
def test_edge_values_of_k_and_v_each_in_their_plane(qw, dt):
    n, D = 9, 64
    x = torch.zeros((2, 1, 1, n, D), device="cuda")              # K and V
    ramp = torch.arange(32, device="cuda")
    x[:, 0, 0, 0, :32] = ramp - 15.5                             # ties: amax 16.5, d = 16.5 / 127
    x[:, 0, 0, 1, :32] = (ramp % 7 - 3.0) * 127                  # whole codes
    x[:, 0, 0, 2, 5], x[:, 0, 0, 3, 6] = float("nan"), float("inf")
    x[:, 0, 0, 4, 7] = 127 * 65504.0 * 1.01 if dt is not F16 else float("inf")  # the scale overflows fp16
    x[:, 0, 0, 5, 8] = 1e-9                                      # the scale underflows to 0
    x[:, 0, 0, 6, :32] = -0.0
    x[:, 0, 0, 7, :32] = torch.linspace(-3e-5, 3e-5, 32)         # a subnormal scale
    x[:, ..., 32:] = 1.0
    x[1] *= -3                                                   # V's own values: a mixed-up plane shows
    x[1, 0, 0, 8, :32] = 40 + ramp
    x = x.to(dt)
    k, v, ks, vs = make_cache("int8", (1, 1, n, D), gen(1))
    view = qw.KvView(k, v, ks, vs)
    qw.kv_append(view, x[0], x[1], i32(0))
    out = [torch.empty_like(x[0]) for _ in range(2)]
    qw.kv_read(view, *out, i32(0))
    fin = [0, 1, 5, 6, 7, 8]
    for rows, codes, scales, o in zip(x, (k, v), (ks, vs), out):
        qc, qs = quantise(rows.float().cpu().numpy()[0, 0, fin])
        np.testing.assert_array_equal(codes[0, 0, fin].cpu().numpy(), qc)
        np.testing.assert_array_equal(scales[0, 0, fin].cpu().numpy(), qs)
        val = torch.from_numpy(qc.astype(np.float32) * np.repeat(qs.astype(np.float32), 32, -1)).cuda().to(dt)
        assert torch.equal(o[0, 0, fin], val)
        assert torch.isnan(o[0, 0, 2:4, :32]).all() and not torch.isfinite(o[0, 0, 4, 7])
        assert torch.equal(o[0, 0, 2:5, 32:], o[0, 0, :1, 32:].expand(3, 32))  # a bad group leaves its neighbour alone


# ---------------------------------------------------------------- tree attention

@pytest.mark.parametrize("dt,kind", [(F16, "int8"), (F16, "f32"), (F16, "bf16"), (BF16, "int8"), (BF16, "f32"), (BF16, "bf16")])
def test_a_long_tail_of_small_weights_counts(qw, dt, kind):
    # One key stands out; each of the 2^17 others weighs 2^-25.2 of it, together 0.34% of the whole.  Their
    # values are 1 and the key's own is 0, so the result is the tail's share.  max_len keeps the positions together.
    C, D, n, heads = 1 << 17, 64, 16, 2
    ct = {"f32": F32, "bf16": BF16, "int8": torch.int8}[kind]
    k, v = (torch.zeros((1, 1, C + n, D), dtype=ct, device="cuda") for _ in range(2))
    ks = vs = None
    k[:, :, 12345, 0] = 64
    v[:, :, :C] = 1
    v[:, :, 12345] = 0
    if kind == "int8":
        ks, vs = (torch.ones((1, 1, C + n, D // 32), dtype=F16, device="cuda") for _ in range(2))
    q = torch.zeros((1, n, heads, D), device="cuda")
    q[..., 0] = 2.1875                                   # the key's score is 140 scale: exact in every type
    scale = 25.2 * float(np.log(2)) / 140
    mask = torch.zeros((1, n), dtype=torch.int64, device="cuda")  # nodes that see the cached positions only
    got = qw.tree_attention(qw.KvView(k, v, ks, vs), q.to(dt), mask, i32(C), scale=scale, max_len=0).double()
    tail = (C - 1) * 2.0 ** -25.2
    want = tail / (1 + tail)
    # Relative to the result: the score (an f32 product, 2^-24 of 25.2) and exp2 (2^-21) change a weight by under
    # 2^-18 of it; its 16 bits by 2^-8 in bf16, and in fp16, held 2^9 above their reference, by 2^-25 of
    # 2^-16.2; V is exact; a running f32 sum takes up to 2^15 additions of 2^-24 each; the result's own rounding.
    weight = U[BF16] if dt is BF16 and kind != "int8" else 2.0 ** -8.8
    tol = 2.0 ** -18 + weight + 2.0 ** -9 + U[dt]
    assert ((got - want).abs() <= tol * want).all(), (float(got.min()), float(got.max()), want)


@pytest.mark.parametrize("kind", ["f32", "int8"])
@pytest.mark.parametrize("drafted", [False, True])
def test_what_fp16_operands_cannot_hold_is_infinite(qw, kind, drafted):
    # fp16 queries, 16 x 2 rows: 16-bit operands.  Cached magnitudes above 65504 are infinite: not NaN, and the same
    # for cached rows and drafted ones.
    n, L, D = 16, 200, 128
    ct = F32 if kind == "f32" else torch.int8
    k, v = (torch.zeros((1, 1, L + n, D), dtype=ct, device="cuda") for _ in range(2))
    ks = vs = None
    if kind == "int8":
        ks, vs = (torch.ones((1, 1, L + n, D // 32), dtype=F16, device="cuda") for _ in range(2))
    v[:] = 1
    at = L + 3 if drafted else 77
    if kind == "f32":
        v[0, 0, at, 5], v[0, 0, at, 6] = 1e5, -float("inf")
        v[0, 0, at, 70] = -65504.0 * 1.5
        k[0, 0, at - 2, 9] = 1e6
    else:
        vs[0, 0, at, 0], vs[0, 0, at, 2] = 1000, 1000        # groups of dims 0-31 and 64-95
        v[0, 0, at, :32] = 0
        v[0, 0, at, 64:96] = 0
        v[0, 0, at, 5], v[0, 0, at, 6], v[0, 0, at, 70] = 100, -127, -66
        ks[0, 0, at - 2, 0] = 60000
        k[0, 0, at - 2, 9] = 100
    q = torch.zeros((1, n, 2, D), dtype=F16, device="cuda")
    q[..., 9] = -1                                           # -inf for that key: weight 0
    mask = torch.full((1, n), (1 << n) - 1, dtype=torch.int64, device="cuda")
    got = qw.tree_attention(qw.KvView(k, v, ks, vs), q, mask, i32(L))[0].float()
    inf = float("inf")
    assert (got[..., 5] == inf).all() and (got[..., 6] == -inf).all() and (got[..., 70] == -inf).all()
    keep = torch.ones(D, dtype=torch.bool, device="cuda")
    keep[[5, 6, 70]] = False
    if kind == "int8":                                       # the bad row's zeros beside 214 ones
        keep[:32] = keep[64:96] = False
        rest = torch.cat([got[..., 7:32], got[..., 71:96]], -1)
        assert ((rest - 214 / 215).abs() <= 2 * U[F16]).all()
    # equal weights of 215 keys on ones: exact but for the weights' sum and the quotient in f32, then one rounding
    assert ((got[..., keep] - 1).abs() <= U[F16]).all()


@pytest.mark.parametrize("max_len", [0, 300])
@pytest.mark.parametrize("n,heads", [(16, 2), (1, 2)])
@pytest.mark.parametrize("sk,sv", [(1.0, 1e-8), (1.0, 1e6), (1e-9, 1e30), (1e8, 1e-30)])
def test_bf16_queries_over_f32_rows_keep_their_range(qw, sk, sv, n, heads, max_len):
    # the result can hold what f32 rows hold; how long the caller thinks that the sequences are changes nothing
    L, D = 300, 128
    g = gen(50)
    k, v = (torch.randn((1, 1, L + n, D), generator=g, device="cuda") * s for s in (sk, sv))
    q = torch.randn((1, n, heads, D), generator=g, device="cuda").to(BF16)
    scale = D ** -0.5 / sk
    mask = torch.from_numpy(qw.tree_mask(range(-1, n - 1)).view(np.int64)).cuda()[None]
    got = qw.tree_attention(qw.KvView(k, v), q, mask, i32(L), scale=scale, max_len=max_len)
    ref, mag, vmax = tree_reference(q, (k, v, None, None), mask, [L], [n], scale)
    # K and V are two bf16 terms (2^-16 at most); a score error e changes the mean of v by at most 2 e max|v|; f32
    # sums of D and of L + n terms; exp2; weights in bf16, and the result
    score = mag * (2.0 ** -16 + (D + 4) * 2.0 ** -24)
    tol = (2 * score + U[BF16] + 2.0 ** -16 + 2.0 ** -20 + (L + n) * 2.0 ** -24) * vmax
    assert ((got.double() - ref).abs() <= tol[..., None] + ref.abs() * U[BF16]).all()


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("dt,kind", [(F16, "int8"), (F16, "f32"), (F16, "bf16"), (BF16, "f32"), (BF16, "bf16")])
@pytest.mark.parametrize("D,L", [(128, 900), (64, 2000)])
def test_errors_are_those_of_the_weights_and_the_result(qw, dt, kind, D, L):
    # Scores of tens, where one rounding of K to 16 bits would be most of the error.
    n, H, G = 17, 2, 4
    g = gen(60)
    cache = make_cache(kind, (1, H, L + n, D), g)
    q = (8 * torch.randn((1, n, H * G, D), generator=g, device="cuda")).to(dt)
    mask = torch.from_numpy(qw.tree_mask(range(-1, n - 1)).view(np.int64)).cuda()[None]
    got = qw.tree_attention(qw.KvView(*cache), q, mask, i32(L))
    ref, _, _ = tree_reference(q, cache, mask, [L], [n], D ** -0.5)
    # Independent roundings of a relative error of at most u are u / sqrt(3) or less in the mean square: the
    # weights', the result's.  Two-term K: 2^-16 (bf16) of q k, whose mean square over the D terms, scaled, is
    # 8 times K's rms of 1.2 or less; f32 sums of D terms, some 2^-19 of scores up to 100.
    u = U[dt]
    bound = u * (2 / 3) ** 0.5 + 10 * 2.0 ** -16 * (dt is BF16 and kind == "f32") + 100 * 2.0 ** -19
    assert rel(got, ref) <= bound
    if kind != "bf16":  # and the bound would not have let one-term operands pass
        one = [widen(t, s).to(dt).double() for t, s in ((cache[0], cache[2]), (cache[1], cache[3]))]
        far, _, _ = tree_reference(q, one + [None, None], mask, [L], [n], D ** -0.5)
        assert rel(far, ref) > bound


@pytest.mark.parametrize("dt,kind", [(F16, "int8"), (F16, "f32"), (BF16, "f32")])
def test_values_that_nearly_cancel_keep_their_second_term(qw, dt, kind):
    # every node sees two keys of equal weight whose values differ in sign and a few of their last bits
    n, D = 16, 128
    g = gen(61)
    if kind == "f32":
        v = torch.randn((1, 1, n, D), generator=g, device="cuda")
        v[:, :, 1::2] = -v[:, :, ::2] * (1 + 2.0 ** -12 * torch.rand((1, 1, n // 2, D), generator=g, device="cuda"))
        cache = [torch.randn_like(v), v, None, None]
    else:
        cache = make_cache("int8", (1, 1, n, D), g)
        cache[1][:, :, 1::2] = -cache[1][:, :, ::2]
        bits = cache[3].view(torch.int16)
        bits[:, :, 1::2] = bits[:, :, ::2] + 1               # the next fp16 scale
    q = torch.zeros((1, n, 2, D), dtype=dt, device="cuda")
    mask = torch.tensor([[3 << (i // 2 * 2) for i in range(n)]], dtype=torch.int64, device="cuda")
    got = qw.tree_attention(qw.KvView(*cache), q, mask, i32(0))
    ref, _, vmax = tree_reference(q, cache, mask, [0], [n], 1.0)
    # what two terms leave of V, and four f32 operations, of max|v|; the result's rounding
    left = 2.0 ** -22 if dt is F16 else 2.0 ** -16
    tol = (left + 4 * 2.0 ** -24) * vmax + ref.abs() * U[dt]
    assert ((got.double() - ref).abs() <= tol).all()
    one = [None, widen(cache[1], cache[3]).to(dt).double()]
    far, _, _ = tree_reference(q, [cache[0] if kind == "f32" else widen(cache[0], cache[2]), one[1], None, None], mask, [0], [n], 1.0)
    assert ((far - ref).abs() > tol).any()  # one-term values would not have passed


@pytest.mark.parametrize("dt,kind", [(F32, "f32"), (F16, "int8"), (BF16, "int8"), (F16, "f32"), (BF16, "bf16")])
def test_a_cache_that_is_only_read_may_overlap(qw, dt, kind):
    # windows of one long row of positions, a few positions apart: sequences that share a prefix's end
    B, L, n, D, step = 3, 100, 5, 64, 20
    whole = make_cache(kind, (1, 1, (B - 1) * step + L + n, D), gen(62))
    cut = [None if t is None else t.as_strided((B, 1, L + n, t.shape[-1]), (step * t.shape[-1], t.stride(1), t.shape[-1], 1))
           for t in whole]
    q = torch.randn((B, n, 8, D), generator=gen(63), device="cuda").to(dt)
    mask = torch.full((B, n), 31, dtype=torch.int64, device="cuda")
    got = qw.tree_attention(qw.KvView(*cut), q, mask, i32(L, L, 7))
    want = qw.tree_attention(qw.KvView(*[None if t is None else t.contiguous() for t in cut]), q, mask, i32(L, L, 7))
    assert torch.equal(got, want)
    out = [torch.empty((B, 1, L + n, D), device="cuda") for _ in range(2)]
    qw.kv_read(qw.KvView(*cut), *out, i32(0, 0, 0))
    assert torch.equal(out[1], widen(cut[1], cut[3]).float())
    with pytest.raises(qw.QwError) as e:
        qw.kv_append(qw.KvView(*cut), *out, i32(0, 0, 0))
    assert e.value.code == qw.INVALID_ARGUMENT


# ---------------------------------------------------------------- logits

@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("V,off,in_place", [(5000, 0, True), (5000, 0, False), (4099, 3, False), (4099, 3, True), (40, 0, True)])
def test_biases_of_a_token_are_added_one_after_the_other(qw, dt, V, off, in_place):
    # behind the penalties, each sum rounded: large logits swallow biases that would count if they were added up first
    R = 3
    g = np.random.default_rng(V)
    named = [t for t in (0, 1, 2, 31, 39, 2047, 2048, V - 1) if t < V]
    x0 = (g.choice([-1.0, 1.0], size=(R, V)) * g.choice([0.5, 3.0, 60.0], size=(R, V))).astype(np.float32)
    big = np.float32(2.0 ** 25 if dt != F16 else 2.0 ** 15)
    x0[:, named] = big * g.choice([-1.0, 1.0], size=(R, len(named)))
    ids = np.array(named * 5 + [-1, V, V + 1], dtype=np.int32)
    g.shuffle(ids)
    bias = g.choice([-3.0, -1.0, 1.0, 3.0, 2.0 ** -12], size=ids.size).astype(np.float32)
    bias[0] = -big
    whole = torch.zeros((R, V + off + 1), dtype=dt, device="cuda")
    x = whole[:, off:off + V]
    x.copy_(torch.from_numpy(x0).cuda())
    x0 = x.float().cpu().numpy()
    hist = np.array([named[0], named[1], named[1], 5], np.int32)
    want = x0.copy()
    for r in range(R):
        for t in set(hist.tolist()):
            c = int((hist == t).sum())
            z = want[r, t]
            z = z / np.float32(2) if z > 0 else z * np.float32(2)
            want[r, t] = z - (np.float32(0.25) + np.float32(0.5) * np.float32(c))
        for i, b in zip(ids, bias):
            if 0 <= i < V:
                want[r, i] = np.float32(want[r, i] + b)
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    out = x if in_place else torch.empty_like(whole)[:, off:off + V]
    qw.process_logits(x, out, penalties=cu(np.array([[2, 0.25, 0.5]] * R, np.float32)), history=cu(hist),
                      history_range=cu(np.array([[0, 4]] * R, np.int32)), bias_ids=cu(ids), bias=cu(bias),
                      bias_range=cu(np.array([[0, ids.size]] * R, np.int32)))
    assert torch.equal(out.float(), cu(want).to(dt).float())
