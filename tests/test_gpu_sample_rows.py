"""The draw of many rows' next tokens (qw_sample_rows) against its definition in 64 bits.

Whole numbers (token, how many were kept) have to be those of the definition unless the border that decides
them lies within the weights' error of a running sum.  A weight is 2^(q / 32) 2^r, |r| <= 1/64: r is rounded to half a place of
2^-30 (3.2e-10 of the weight), 2^r - 1 <= 0.011 too (4.7e-10), the table's f32 and the product with it to 2^-24 of
0.011 (6.5e-10 each), the table's whole number to 2^-32 (2.3e-10): 2.4e-9 together.  A border compares a running sum
with a part of another one, so a row may differ only where the definition's own border is within 5e-9 of the sum.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NEAR = 5e-9


@pytest.fixture(scope="module")
def qw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from runtime_qwen3_decode_gb300 import build, qw as binding
    build.build()
    return binding


def define(x, t, k, p, m, u):
    """(token, kept, probability, sure) of one row of logits (numpy, any float type)."""
    x = x.astype(np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, float(np.finfo(np.float32).max))) + 0.0
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    if len(order) == 0:
        return -1, 0, 0.0, True
    if t == 0:
        return int(order[0]), 1, 1.0, True
    sure = True
    if 0 < k < len(order):
        order = order[:k]
    w = np.exp((x[order] - x[order[0]]) / t)
    cum = np.cumsum(w.astype(np.longdouble))
    n = len(order)
    if p < 1:
        goal = np.longdouble(p) * cum[-1]
        n = min(n, int(np.searchsorted(cum, goal)) + 1)
        sure &= _clear(cum, goal, w)
    n_m = int((w >= m).sum())
    if m > 0:
        z = (x[order] - x[order[0]]) / t - math.log(m)
        sure &= not bool(((np.abs(z) < 1e-12) & (z != 0)).any())
    n = min(n, n_m)
    goal = np.longdouble(u) * cum[n - 1]
    j = min(int(np.searchsorted(cum[:n], goal, side="right")), n - 1)
    sure &= _clear(cum[:n], goal, w[:n])
    return int(order[j]), n, float(w[j] / cum[n - 1]), sure


def _clear(cum, goal, w):
    """Whether no running sum is within the weights' error of goal (sums of equal weights are exact)."""
    if (w == 1).all():
        return True
    return bool(np.abs(cum - goal).min() > NEAR * cum[-1])


def check(qw, x, u, t=None, k=None, p=None, m=None, out_sure=0.98):
    R = x.shape[0]
    f = lambda v, d: None if v is None else torch.tensor(np.broadcast_to(np.asarray(v), (R,)).copy(), dtype=d, device="cuda")
    uu = f(u, F32)
    kept, probs = torch.full((R,), -7, dtype=torch.int32, device="cuda"), torch.full((R,), -7.0, device="cuda")
    tok = qw.sample_rows(x, uu, f(t, F32), f(k, torch.int32), f(p, F32), f(m, F32), probs=probs, kept=kept)
    again = qw.sample_rows(x, uu, f(t, F32), f(k, torch.int32), f(p, F32), f(m, F32))
    assert torch.equal(tok, again)
    tok, kept, probs, uu = tok.cpu().numpy(), kept.cpu().numpy(), probs.cpu().numpy(), uu.cpu().numpy()
    val = lambda v, d, r: d if v is None else np.float32(np.broadcast_to(np.asarray(v), (R,))[r]).astype(np.float64)
    xs = x.float().cpu().numpy()
    n_sure = 0
    for r in range(R):
        want = define(xs[r], val(t, 1.0, r), int(val(k, 0, r)), val(p, 1.0, r), val(m, 0.0, r), float(uu[r]))
        if not want[3]:
            continue
        n_sure += 1
        assert (tok[r], kept[r]) == want[:2], (r, tok[r], kept[r], want)
        # W and S off by 2.4e-9 each, an f32 quotient (2^-24, its parts' roundings 2^-24 more)
        assert abs(probs[r] - want[2]) <= 5e-9 * want[2] + 2 ** -23 * want[2]
    assert n_sure >= out_sure * R
    return tok


def peaked(g, R, V, dt=F32):
    x = 2.0 * torch.randn((R, V), generator=g, device="cuda")
    n = min(V, 40)
    x[:, :n] += 10 - 2 * torch.log1p(torch.arange(n, device="cuda").float())
    return x[:, torch.randperm(V, generator=g, device="cuda")].contiguous().to(dt)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("R,V", [(1, 1), (3, 2), (5, 31), (2, 1000), (4, 8192), (7, 9001), (3, 32768), (2, 151936), (40, 20011)])
def test_settings(qw, R, V, dt):
    g = gen(R * V)
    x = peaked(g, R, V, dt)
    u = torch.rand((R,), generator=g, device="cuda").cpu().numpy()
    for t, k, p, m in ((None, None, None, None), (0.7, 40, 0.9, None), (0.7, None, 0.95, None), (1.3, 300, 1.0, 0.02), (1.8, None, 0.99, None),
                       (0.0, 5, 0.3, 0.5), (2.5, 5000, 0.999, 0.001), (1.0, 1, 1.0, 0.0), (0.9, 3000, None, None), (3.0, V, 1.0, 1e-7)):
        # logits of 16 bits tie, but their running sums are as the others
        check(qw, x, u, t, k, p, m, out_sure=0.5)


@pytest.mark.parametrize("V", [10000, 151936])
def test_borders_far_down(qw, V):
    """Sets of kept tokens that no list holds: each border is searched for."""
    g = gen(V)
    x = torch.randn((6, V), generator=g, device="cuda")
    u = np.array([0.0, 0.3, 0.9, 0.999, 1 - 2 ** -24, 0.5], np.float32)
    for t, k, p, m in ((1.0, None, None, None), (5.0, None, 0.9, None), (1.0, V // 2, 0.8, None), (0.8, V // 3, 0.9, 0.05),
                       (1e6, None, None, None), (1.0, V - 1, None, 1e-3), (2.0, 2048, None, None), (2.0, 2049, None, None)):
        check(qw, x, u, t, k, p, m, out_sure=0.3)


@pytest.mark.parametrize("V", [5, 2048, 2049, 70001])
def test_equal_logits(qw, V):
    """Every logit alike: running sums are whole multiples and borders are met exactly."""
    x = torch.full((8, V), -3.25, device="cuda")
    u = np.array([0, 0.25, 0.5, 0.75, 1 - 2 ** -24, 0.125, 0.3, 0.9], np.float32)
    check(qw, x, u, out_sure=1.0)
    check(qw, x, u, 0.37, None, 0.5, out_sure=1.0)
    check(qw, x, u, 3.0, max(1, V // 2), 0.25, 1.0, out_sure=1.0)


def test_nucleus_border_is_at_least(qw):
    x = torch.zeros((4, 4), device="cuda")
    p = np.array([0.25, 0.5, 0.75, 0.5000001], np.float32)
    kept = torch.zeros(4, dtype=torch.int32, device="cuda")
    qw.sample_rows(x, torch.zeros(4, device="cuda"), top_p=torch.tensor(p, device="cuda"), kept=kept)
    assert kept.tolist() == [1, 2, 3, 3]


@pytest.mark.parametrize("V", [40, 4097, 100003])
def test_masked_and_unusual_logits(qw, V):
    g = gen(V)
    x = peaked(g, 12, V)
    x[0] = -math.inf                                    # nothing to draw
    x[1] = math.nan
    x[2, 1:] = -math.inf                                # one candidate
    x[3, torch.rand(V, generator=g, device="cuda") < 0.9] = -math.inf
    x[4, ::3] = math.nan
    x[5, V // 2] = math.inf                             # the greatest finite number
    x[5, V // 3] = math.inf
    x[6] = torch.finfo(F32).min                         # the type's lowest value as a mask
    x[6, 7:19] = torch.linspace(-1, 1, 12, device="cuda")
    x[7] = torch.finfo(F32).min
    x[8] *= 1e30
    x[9] *= -1e-30
    x[10, :] = 0.0
    x[10, 5] = -0.0
    x[11] += 30000.0
    u = torch.rand((12,), generator=g, device="cuda").cpu().numpy()
    for t, k, p, m in ((None, None, None, None), (0.5, 20, 0.9, 0.0), (1e-6, None, 0.9, None), (0.0, None, None, None), (7.0, 30, None, 0.1),
                       (1e6, None, 0.4, None)):
        check(qw, x, u, t, k, p, m, out_sure=0.3)


def test_row_strides_and_alignments(qw):
    g = gen(5)
    for dt in (F32, F16, BF16):
        wide = peaked(g, 6, 5003, dt)
        for off in range(4):
            x = wide[::2, off:off + 4097]
            u = torch.rand((3,), generator=g, device="cuda").cpu().numpy()
            check(qw, x, u, 0.8, 100, 0.9, None, out_sure=0.5)
    one = peaked(g, 1, 3001).expand(5, 3001)            # one row drawn from five times
    check(qw, one, np.linspace(0, 0.99, 5).astype(np.float32), 1.5, out_sure=0.5)


def test_vocabulary_beyond_shared_memory(qw):
    g = gen(9)
    x = peaked(g, 2, 1 << 20, BF16)
    check(qw, x, np.array([0.2, 0.8], np.float32), 1.0, 200, 0.9, out_sure=0.0)
    x = torch.randn((2, 700001), generator=g, device="cuda")
    check(qw, x, np.array([0.2, 0.8], np.float32), 1.0, None, 0.9, out_sure=0.0)


def test_parameters_outside_their_ranges(qw):
    x = torch.randn((9, 50), device="cuda")
    ok = torch.full((9,), 0.5, device="cuda")

    def with_(row, v):
        t = ok.clone()
        t[row] = v
        return t
    t = with_(0, -1.0)
    t[1], t[2] = math.nan, 1e7
    p = with_(3, 0.0)
    p[4] = 1.5
    m = with_(5, -0.1)
    u = with_(6, 1.0)
    u[7] = math.nan
    kept, probs = torch.full((9,), 9, dtype=torch.int32, device="cuda"), torch.ones(9, device="cuda")
    tok = qw.sample_rows(x, u, t, None, p, m, probs=probs, kept=kept)
    assert tok[:8].tolist() == [-1] * 8 and kept[:8].tolist() == [0] * 8 and probs[:8].tolist() == [0.0] * 8
    assert tok[8] >= 0 and kept[8] >= 1


def test_many_draws_follow_the_probabilities(qw):
    """Every border of the definition hit by an even grid of u: the picks are its inverse distribution function."""
    g = gen(1)
    x = peaked(g, 1, 3000)
    n = 4000
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    check(qw, x.expand(n, 3000), u, 0.8, 50, 0.97, 0.001, out_sure=0.99)


def test_captured_and_on_another_stream(qw):
    g = gen(2)
    x = peaked(g, 5, 30011)
    u = torch.rand((5,), generator=g, device="cuda")
    k = torch.full((5,), 30, dtype=torch.int32, device="cuda")
    want = qw.sample_rows(x, u, top_k=k)
    tok = torch.zeros(5, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        qw.sample_rows(x, u, top_k=k, tokens=tok, stream=st)
    st.synchronize()
    assert torch.equal(tok, want)
    with torch.cuda.graph(graph, stream=st):
        qw.sample_rows(x, u, top_k=k, tokens=tok)
    x.copy_(peaked(g, 5, 30011))
    u.copy_(torch.rand((5,), generator=g, device="cuda"))
    tok.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(tok, qw.sample_rows(x, u, top_k=k))


def test_top_k_order_is_qw_sample_logits(qw):
    """With u of PCG32's word the token is the one-row sampler's."""
    g = gen(3)
    for seed in range(5):
        x = peaked(g, 1, 8192)
        state = torch.tensor([1234567 + seed, 2 * seed + 1], dtype=torch.int64, device="cuda")
        st = int(state[0])
        word = oracle_word(st)
        tok = torch.zeros(1, dtype=torch.int32, device="cuda")
        qw.sample_logits(x[0], qw.Sampling(0.8, 50, 0.9, 1.0), state, tok)
        u = torch.tensor([(word >> 8) / 2 ** 24], dtype=F32, device="cuda")
        f = lambda v: torch.full((1,), v, device="cuda")
        ours = qw.sample_rows(x, u, f(0.8), torch.full((1,), 50, dtype=torch.int32, device="cuda"), f(0.9))
        assert int(ours) == int(tok)


def oracle_word(old):
    x = (((old >> 18) ^ old) >> 27) & 0xFFFFFFFF
    rot = old >> 59
    return ((x >> rot) | (x << ((32 - rot) & 31))) & 0xFFFFFFFF


def test_the_largest_vocabulary_and_rows_far_apart(qw):
    """2^24 tokens, all of one CTA's in the same part of a pass; rows more than 2^32 bytes apart."""
    V = 1 << 24
    x = torch.zeros((1, V), dtype=F16, device="cuda")
    kept = torch.zeros(1, dtype=torch.int32, device="cuda")
    for u in (0.0, 0.3, 1 - 2 ** -24):
        tok = qw.sample_rows(x, torch.tensor([u], device="cuda"), kept=kept)
        # equal weights: token j is drawn for u in [j / V, (j + 1) / V); u is an f32
        assert int(tok) == int(np.float64(np.float32(u)) * V) and int(kept) == V
    tok = qw.sample_rows(x, torch.tensor([0.5], device="cuda"), top_p=torch.tensor([0.25], device="cuda"), kept=kept)
    assert int(kept) == V // 4 and int(tok) == V // 8
    far = (1 << 31) + 5
    big = torch.empty(2 * far, dtype=F16, device="cuda")
    rows = big.as_strided((2, 5000), (far, 1), 3)
    rows.copy_(peaked(gen(4), 2, 5000))
    check(qw, rows, np.array([0.4, 0.7], np.float32), 0.9, 50, 0.9, None, out_sure=0.5)


@pytest.mark.parametrize("R", [300, 2100])
def test_many_rows_with_settings_of_their_own(qw, R):
    """Rows that take the short way and the long one in one call, in more than one wave."""
    g = gen(R)
    x = peaked(g, R, 3001)
    r = np.random.default_rng(R)
    t = np.where(r.random(R) < 0.2, 0, r.uniform(0.3, 3, R)).astype(np.float32)
    k = np.where(r.random(R) < 0.5, 0, r.integers(1, 3000, R)).astype(np.int32)
    p = np.where(r.random(R) < 0.5, 1, r.uniform(0.2, 1, R)).astype(np.float32)
    m = np.where(r.random(R) < 0.5, 0, r.uniform(0, 0.2, R)).astype(np.float32)
    check(qw, x, r.random(R).astype(np.float32), t, k, p, m, out_sure=0.9)
