"""Drafted trees and 8-bit batches where tests/test_gpu_tree.py does not reach: caller memory that changes behind a call,
and contexts long enough that the steps attend on the tensor cores."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import qw_inputs as qi  # noqa: E402
from test_gpu_tree import setup  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from runtime_qwen3_decode_gb300 import build, qw as binding
    build.build()
    return binding


def test_a_tree_step_is_done_with_the_callers_memory_when_it_returns(qw):
    wl = qi.WORKLOADS["tiny"]
    host, m, b = setup(qw, wl, 4, 64, flags=False)
    b.prefill(1, [3, 1, 4, 1, 5])
    toks, parents = [9, 2, 6, 5], [-1, 0, 0, 1]
    b.tree_step(1, toks, parents)
    want = b.logits().clone()
    t = torch.tensor(toks, dtype=torch.int32).pin_memory()
    p = torch.tensor(parents, dtype=torch.int32).pin_memory()
    i32p = ctypes.POINTER(ctypes.c_int32)
    busy = torch.ones(1 << 26, device="cuda")
    torch.cuda.synchronize()
    for _ in range(100):  # some 10 ms before the step's turn comes
        busy.mul_(1.0)
    rc = qw.lib().qw_batch_tree_step(b._h, 1, 4, ctypes.cast(t.data_ptr(), i32p), ctypes.cast(p.data_ptr(), i32p), None)
    t.fill_(7)
    p.fill_(-1)
    assert rc == qw.OK
    b.last_n = 4
    assert torch.equal(b.logits(), want)
    b.close()
    m.close()
