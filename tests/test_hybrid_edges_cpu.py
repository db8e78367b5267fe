"""Host-side checks of the operators around the layer, beside those of test_hybrid_cpu.py: descriptors
of which only the documented fields are filled, sizes that overflow, tensors the binding refuses."""
import ctypes

import pytest

from tests.test_hybrid_cpu import _at, _conv, _rg, dsa  # noqa: F401  (a fixture)


def test_conv_does_not_judge_max_q_len(dsa):  # noqa: F811
    """What comes back for an unset max_q_len is what comes back for a right one."""
    for max_q_len in (0, -1, -(1 << 31)):
        rg = _rg(dsa, max_q_len=max_q_len)
        assert _conv(dsa, rg=rg, width=5) == dsa.DSA_ERR_UNSUPPORTED
        assert _conv(dsa, rg=rg, ptrs=dict(weight=None)) == dsa.DSA_ERR_INVALID_ARG
