"""The same prompt leaves the same bits every time: the softmax warps of the prefill's attention may be a block apart."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import qw_inputs as qi  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,times", [(2048, 500), (4001, 250), (300, 500)])
def test_rows_of_a_repeated_prompt(n, times):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from runtime_qwen3_decode_gb300 import build, qw
    build.build()
    wl = qi.WORKLOADS["tiny"]
    ctx = 4200
    m = qw.Model(wl, qw.weights_to_device(qi.make_weights(wl), int8=False), max_ctx=ctx)
    b = qw.Batch(m, 1, ctx)
    planes = 2 * wl.n_layers * wl.n_kv_heads
    rows = b.workspace[:planes * ctx * wl.head_dim * 4].view(torch.float32).view(planes, ctx, wl.head_dim)[:, :n]  # K and V
    p = np.random.default_rng(n).integers(0, wl.vocab, n).astype(np.int32)
    token = b.prefill(0, p)
    want = rows.clone()
    assert want.abs().amax((1, 2)).min() > 0
    for k in range(times):
        b.reset()
        assert b.prefill(0, p) == token
        assert torch.equal(rows, want), f"time {k}"
    b.close()
    m.close()
