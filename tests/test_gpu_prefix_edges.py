"""Edges of the attention of batches that share a prefix (qw_prefix_attention)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import BF16, F16, F32, U, gen, i32, make_cache, tolerance, tree_reference  # noqa: E402, F401
from test_gpu_prefix import ROOM, joined, make_prefix, qw, run  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,P,L", [(3, 60000, 5), (130, 9000, 700), (64, 4096, 257)])
def test_long_runs_of_tiles(qw, B, P, L, D):  # noqa: F811
    """Shares of many tiles, of the prefix alone and of many sequences' own: stages of V are filled again while the
    warps that look some of them through are behind or ahead.  The same result every time."""
    g = gen(B)
    pre, own = make_cache("bf16", (1, 2, P, D), g), make_cache("bf16", (B, 2, L + 1, D), g)
    q = torch.randn((B, 1, 4, D), generator=g, device="cuda").to(BF16)
    lens = torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    views = qw.KvView(*pre), qw.KvView(*own)
    scratch = qw.prefix_attention_scratch(*views, 1, 4)
    want = qw.prefix_attention(*views, q, lens, i32(P), scratch=scratch)
    for _ in range(30):
        assert torch.equal(qw.prefix_attention(*views, q, lens, i32(P), scratch=scratch), want)
    mask = torch.ones((B, 1), dtype=torch.int64, device="cuda")
    some = [0, B // 2, B - 1]
    at = [None if o is None else o[some] for o in own]
    ref, mag, vmax = tree_reference(q[some], joined(pre, at, P), mask[some], [P + int(lens[b]) for b in some], [1] * 3, D ** -0.5)
    assert ((want[some].double() - ref).abs() <= tolerance(BF16, "bf16", mag, vmax, P + L + 1, D)).all()


@pytest.mark.parametrize("tc", [False, True])
@pytest.mark.parametrize("dt,kind,D", [(BF16, "int8", 128), (BF16, "int8", 64), (BF16, "bf16", 128), (F16, "f32", 128), (F32, "f32", 64)])
def test_scores_that_underflow(qw, tc, dt, kind, D):  # noqa: F811
    """Queries near the type's smallest numbers and a small scale: every score rounds to 0, and a row is the mean of what it
    sees.  The factor of a row's scores underflows, and what is hidden must not become 0 x -inf."""
    B, H, n, P = 3, 2, 4, 300
    g = gen(30)
    pre, own = make_prefix(kind, (1, H, P, D), g, tc), make_cache(kind, (B, H, 200, D), g)
    tiny = float(torch.finfo(dt).tiny)
    q = (tiny * torch.randn((B, n, 2 * H, D), generator=g, device="cuda")).to(dt)
    lens = [150, 0, 31]
    mask = torch.tensor([[1, 3, 5, 9]] * B, dtype=torch.int64, device="cuda")
    scale = 1e-9
    got = qw.prefix_attention(qw.KvView(*pre), qw.KvView(*own), q, i32(*lens), i32(P), mask=mask, scale=scale)
    ref, mag, vmax = tree_reference(q, joined(pre, own, P), mask, [P + x for x in lens], [n] * B, scale)
    assert ((got.double() - ref).abs() <= tolerance(dt, kind, mag, vmax, P + 200, D)).all()


@pytest.mark.parametrize("tc", [False, True])
@pytest.mark.parametrize("dt,kind", [(BF16, "bf16"), (BF16, "int8"), (BF16, "f32"), (F16, "int8"), (F16, "f32"), (F16, "bf16")])
@pytest.mark.parametrize("where", ["prefix", "own"])
def test_a_row_that_sees_one_key_is_its_value(qw, tc, dt, kind, where):  # noqa: F811
    """One score some 50 above all others: whatever its weight is rounded to, the result is that position's V.  The others
    are at most 700 e^-45 = 2e-17 of it; the result's rounding leaves u, f32 sums and quotients 2^-20, V as the products
    hold it 2^-21 (two fp16 terms) or 2^-16 (two of bf16).  8-bit rows beside bf16 queries: V and the weight, which the sum
    takes unrounded, are one fp16 number each, 2^-11."""
    B, H, D, P = 64, 2, 128, 500
    g = gen(31)
    pre, own = make_prefix(kind, (1, H, P, D), g, tc), make_cache(kind, (B, H, 200, D), g)
    u = torch.randint(0, 2, (D,), generator=g, device="cuda") * 2.0 - 1.0
    for t, at in ((pre, (0, slice(None), 77)), (own, (slice(None), slice(None), 33))):
        k = t[0]
        if kind == "int8":
            k.copy_(torch.randint(-3, 4, k.shape, generator=g, device="cuda").to(k.dtype))
            t[2].fill_(0.01)
        else:
            k.mul_(0.03)
        if (t is pre) == (where == "prefix"):
            k[at] = (100 * u).to(k.dtype) if kind == "int8" else u.to(k.dtype)
    # every row another score of the one key: its weight lies anywhere between two powers of two
    a = (4.0 + 3.0 * torch.rand((B, 1, H, 1), generator=g, device="cuda")).to(dt)
    q = (a.float() * u).to(dt)
    lens = i32(*[40 + 2 * b for b in range(B)])
    got = qw.prefix_attention(qw.KvView(*pre), qw.KvView(*own), q, lens, i32(P)).double()
    at = (pre, (slice(None), slice(None), 77)) if where == "prefix" else (own, (slice(None), slice(None), 33))
    v = at[0][1][at[1]].double()
    if kind == "int8":
        v = v * at[0][3][at[1]].double().repeat_interleave(32, -1)
    v = v.expand(B, H, D).unsqueeze(1)
    tol = U[dt] + (2 * 2.0 ** -11 if dt is BF16 and kind == "int8" else 2.0 ** -16 if dt is BF16 else 2.0 ** -21) + 2.0 ** -20
    assert ((got - v).abs() <= tol * v.abs() + 1e-7).all(), float(((got - v).abs() / v.abs().clamp(min=1e-3)).max())
