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
