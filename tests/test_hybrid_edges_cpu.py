"""Host-side checks of the operators around the layer, beside those of test_hybrid_cpu.py: descriptors
of which only the documented fields are filled, sizes that overflow, tensors the binding refuses."""
import ctypes

import pytest

from tests.test_hybrid_cpu import _at, _conv, _rg, _rope, dsa  # noqa: F401  (a fixture)


def test_conv_does_not_judge_max_q_len(dsa):  # noqa: F811
    """What comes back for an unset max_q_len is what comes back for a right one."""
    for max_q_len in (0, -1, -(1 << 31)):
        rg = _rg(dsa, max_q_len=max_q_len)
        assert _conv(dsa, rg=rg, width=5) == dsa.DSA_ERR_UNSUPPORTED
        assert _conv(dsa, rg=rg, ptrs=dict(weight=None)) == dsa.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("shape", [(5, 64), (5, 4, 128)])
def test_binding_refuses_repeated_and_overlapping_rows(dsa, shape):  # noqa: F811
    """A row stride of 0 means packed rows to the library, so a broadcast tensor must not reach it; nor
    rows that overlap.  (get_device() of a CPU tensor is -1.)"""
    import torch
    row = torch.zeros(1, *shape[1:], dtype=torch.bfloat16)
    rows = lambda t: dsa._rows("call", "x", t, torch.bfloat16, shape, -1)  # noqa: E731
    width = row.numel()
    for bad in (row.expand(shape), torch.zeros(4096, dtype=torch.bfloat16).as_strided(shape, (8, *row.stride()[1:])),
                row.expand(9, *shape[1:])):
        with pytest.raises(dsa.DsaError):
            rows(bad)
    wide = torch.zeros(5, width + 8, dtype=torch.bfloat16)
    assert rows(wide[:, :width].view(shape)) == (wide.data_ptr(), width + 8)
    assert rows(torch.zeros(shape, dtype=torch.bfloat16))[1] == 0
    # one row or none: there is nothing to repeat
    one = (1, *shape[1:])
    assert dsa._rows("call", "x", row.expand(shape)[:1], torch.bfloat16, one, -1) == (row.data_ptr(), 0)
    assert dsa._rows("call", "x", row.expand(shape), torch.bfloat16, one, -1) == (row.data_ptr(), 0)


def test_binding_refuses_a_workspace_smaller_than_it_says(dsa):  # noqa: F811
    import torch
    ws = torch.zeros(64, dtype=torch.int32)
    take = lambda t, n=None: dsa._workspace("call", t, n, -1)  # noqa: E731
    assert take(ws) == (ws.data_ptr(), 256) and take(ws, 100) == (ws.data_ptr(), 100)
    assert take(None) == (None, 0) and take(None, 64) == (None, 0)
    for t, n in ((ws[:1].expand(64), None), (ws[::2], None), (ws, 257), (ws, -1)):
        with pytest.raises(dsa.DsaError):
            take(t, n)
    with pytest.raises(dsa.DsaError):
        dsa._workspace("call", ws, None, 0)


@pytest.mark.parametrize("kw", [dict(rot_dim=16, rot_offset=(1 << 31) - 8), dict(rot_dim=128, rot_offset=(1 << 31) - 128),
                                dict(rot_dim=(1 << 31) - 16, rot_offset=(1 << 31) - 8),
                                dict(idx_rot_dim=64, idx_rot_offset=(1 << 31) - 64)])
def test_rope_offsets_whose_end_overflows(dsa, kw):  # noqa: F811
    """offset + dimensions beyond 2^31 is past the head, not negative."""
    none = {n: None for n, _ in dsa.RopeBuffers._fields_}
    for buffers in (dict(none, q=_at(0), q_out=_at(5)), dict(none, q_idx=_at(3), q_idx_out=_at(8))):
        if ("rot_dim" in kw) == (buffers["q"] is not None):
            assert _rope(dsa, rg=_rg(dsa, total_q=0), buffers=buffers, **kw) == dsa.DSA_ERR_INVALID_ARG
