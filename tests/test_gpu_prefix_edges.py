"""Edges of the attention of batches that share a prefix (qw_prefix_attention)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import BF16, F16, F32, gen, i32, make_cache, tolerance, tree_reference  # noqa: E402, F401
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
