"""Edges of the draw of many rows' next tokens (qw_sample_rows): logits about zero, small weights, calls of other sizes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_sample_rows import check, gen, peaked, qw  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("many", [False, True])  # passes of 32 and of 8 parts
@pytest.mark.parametrize("zeros,below,bits,above", [(10000, 30000, 22, 0), (10328, 38399, 21, 0), (3000, 5000, 8, 300), (700, 20000, 12, 0),
                                                    (12000, 0, 1, 2000)])
def test_zeros_beside_numbers_next_to_zero(qw, zeros, below, bits, above, many):  # noqa: F811
    """Borders on both sides of the place between the greatest negative number and 0.  Every weight is 1, so that
    the running sums are exact."""
    r = np.random.default_rng(zeros)
    x = np.concatenate([np.zeros(zeros, np.float32), -r.integers(1, 1 << bits, below).astype(np.uint32).view(np.float32),
                        r.integers(1, 1000, above).astype(np.uint32).view(np.float32)])
    x[: zeros // 2] *= -1.0                             # -0 is 0
    x = x[r.permutation(len(x))]
    n = 8 if not many else 160 if len(x) > 24000 else 320
    share = np.array([zeros + above, above + 1, zeros + above + 1, (zeros + above) // 2, len(x) - 1], np.float64) / len(x)
    p = np.tile(np.concatenate([[0.26, 0.5, 0.9], share[share < 1]]), n)[:n].astype(np.float32)
    u = np.resize(np.array([0.0, 0.3, 0.77, 0.9999], np.float32), n)
    rows = torch.from_numpy(x).cuda().expand(n, len(x))
    check(qw, rows, u, None, None, p, out_sure=1.0)
    k = np.resize(np.array([1500, max(1, zeros + above - 1), zeros + above, zeros + above + 1, len(x) - 1], np.int32), n)
    check(qw, rows, u, None, k, None, out_sure=1.0)
    check(qw, rows, u, 1e6, k, p, out_sure=1.0)


@pytest.mark.parametrize("V", [8192, 20011, 40000, 65000])
def test_a_row_draws_the_same_alone_and_among_many(qw, V):  # noqa: F811
    """The number of rows decides how many CTAs a row has; tokens of 2^-29 of the first one's weight show in their
    probabilities what unit weights have."""
    g = gen(V)
    x = (-20.0 + 0.5 * torch.randn((1, V), generator=g, device="cuda")).contiguous()
    x[0, V // 3] = 0.0
    n = 24
    u = torch.cat([torch.rand((n // 2,), generator=g, device="cuda"), 1 - 2.0 ** -24 * torch.arange(1, 13, device="cuda") * V / 4096])
    many = 320 // n * n + n

    def draw(rows, u, k, p, m):
        f = lambda v, d: torch.full((rows,), v, dtype=d, device="cuda")  # noqa: E731
        kept, probs = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, device="cuda")
        tok = qw.sample_rows(x.expand(rows, V), u, f(1.0, torch.float32), f(k, torch.int32), f(p, torch.float32), f(m, torch.float32),
                             probs=probs, kept=kept)
        return torch.stack([tok.double(), kept.double(), probs.double()])
    for k, p, m in ((0, 1.0, 0.0), (0, 0.99999, 0.0), (3000, 1.0, 0.0), (900, 1.0, 0.0), (0, 0.99999, 1e-9), (0, 1.0, 2e-9)):
        alone = torch.cat([draw(1, u[i:i + 1], k, p, m) for i in range(n)], 1)
        assert alone[0].unique().numel() > 1
        for rows in (n, many):
            assert torch.equal(draw(rows, u.repeat(rows // n), k, p, m), alone.repeat(1, rows // n)), (k, p, m, rows)


def unit_bits(V):
    return 44 if V <= 1 << 18 else 62 - (V - 1).bit_length()


@pytest.mark.parametrize("V", [151936, 1 << 20, 1 << 22])
@pytest.mark.parametrize("units", [0.49, 0.51, 1.45, 1.55, 3.4, 30.45])
def test_long_tails_of_small_weights(qw, V, units):  # noqa: F811
    """One sure token and V - 1 whose weights are `units` of the unit: each is off by 2.4e-9 of itself and half a unit at
    most, so any running sum by `off`, and what is drawn is what the definition draws within that of its border."""
    unit = 2.0 ** -unit_bits(V)
    tail = np.float32(np.log(units * unit))
    x = torch.full((1, V), float(tail), device="cuda")
    x[0, 0] = 0.0
    w = np.exp(np.float64(tail))
    S = 1 + (V - 1) * w
    off = 2.4e-9 * S + (V - 1) * unit / 2
    u = (1 - np.arange(1, 9) * 2.0 ** -24).astype(np.float32)
    kept, probs = torch.zeros(8, dtype=torch.int32, device="cuda"), torch.zeros(8, device="cuda")
    tok = qw.sample_rows(x.expand(8, V), torch.from_numpy(u).cuda(), kept=kept, probs=probs).cpu().numpy()
    assert (kept == V).all()                            # all of them are candidates, whatever they weigh
    for t, uu, pr in zip(tok, u.astype(np.float64), probs.cpu().numpy().astype(np.float64)):
        before, upto = (0 if t == 0 else 1 + (t - 1) * w), 1 + t * w
        # the sums that are compared are those before and up to the token, and u times the last one
        assert before - 2 * off <= uu * S < upto + 2 * off
        wt = 1.0 if t == 0 else w
        assert abs(pr - wt / S) <= (2.4e-9 * wt + unit / 2 + pr * off) / S * (1 + 1e-6) + 2 ** -23 * (wt / S + pr)
    p = (1 - np.arange(1, 9) * 2.0 ** -24).astype(np.float32)
    qw.sample_rows(x.expand(8, V), torch.zeros(8, device="cuda"), top_p=torch.from_numpy(p).cuda(), kept=kept)
    for n, pp in zip(kept.tolist(), p.astype(np.float64)):
        assert 1 + (n - 2) * w - 2 * off < pp * S <= 1 + (n - 1) * w + 2 * off or (n == 1 and pp * S <= 1 + 2 * off)


@pytest.mark.parametrize("dt,V", [(torch.bfloat16, 1 << 20), (torch.float32, 700001), (torch.float16, 400003)])
def test_rows_that_shared_memory_does_not_hold(qw, dt, V):  # noqa: F811
    """Rows that are read again in every pass, at random logits whose borders are clear: all but a few are compared."""
    g = gen(V)
    R = 8
    x = peaked(g, R, V, dt)
    u = torch.rand((R,), generator=g, device="cuda").cpu().numpy()
    for t, k, p, m in ((1.0, 200, 0.9, None), (0.8, 5000, 0.95, None), (1.0, None, None, 0.01), (0.0, None, None, None)):
        check(qw, x, u, t, k, p, m, out_sure=0.9)
    flat = torch.randn((R, V), generator=g, device="cuda").to(dt)
    # a running sum passes a border by a weight of some 1e-6, next to which 5e-9 are seldom
    for t, k, p, m in ((1.0, None, 0.9, None), (1.3, V // 2, None, None), (1.0, None, 0.99, 0.001)):
        check(qw, flat, u, t, k, p, m, out_sure=0.75)
