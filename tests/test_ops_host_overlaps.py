"""Calls whose results lie over what they read: refused before the device is touched, so these run without a GPU."""
import ctypes

import pytest

from test_ops_host import P, qw  # noqa: F401
from test_ops_host_prefix import call, sample


def apart(**kw):
    """Arrays of eight rows, 64 bytes apart."""
    names = ("u", "temperature", "top_k", "top_p", "min_p", "tokens", "probs", "kept")
    return {**{n: P + 4096 + 64 * i for i, n in enumerate(names)}, "n_rows": 8, **kw}


@pytest.mark.parametrize("out", ["tokens", "probs", "kept"])
@pytest.mark.parametrize("other", ["temperature", "top_k", "top_p", "min_p", "tokens", "probs", "kept"])
@pytest.mark.parametrize("shift", [-28, -4, 0, 4, 28])
def test_results_over_settings_or_one_another(qw, out, other, shift):  # noqa: F811
    if out == other:
        return
    d = apart()
    a = sample(qw, **{**d, out: d[other] + shift})
    assert qw.lib().qw_sample_rows(ctypes.byref(a), None) == qw.INVALID_ARGUMENT


def test_prefix_attention_in_place(qw):  # noqa: F811
    assert call(qw, args=dict(q=P + 4096, out=P + 4096)) == qw.INVALID_ARGUMENT
