"""Host-side checks of the operators around the layer (rotary append, short convolution, gated
delta rule): argument errors come back before any CUDA call, and sizes are planned on the host."""
import ctypes

import pytest

A = 0x10000000  # aligned stand-in addresses, never dereferenced on these paths
STEP = 1 << 32  # apart from one another by more than any buffer here


def _at(i):
    return A + i * STEP


@pytest.fixture(scope="module")
def dsa():
    import indexer_top_gated_b200 as m
    return m


def _rg(dsa, batch=2, q=8, kv=64, **kw):
    rg = dsa.Ragged(batch, 0x1000, 0x2000, q, kv, q * batch, kv * batch)
    for k, v in kw.items():
        setattr(rg, k, v)
    return rg


# ---------------------------------------------------------------- rotary append

def _rope(dsa, rg=None, shape=None, rope=None, buffers=None, **kw):
    o = dict(layout=0, scaling=0, rot_dim=128, rot_offset=0, idx_rot_dim=64, idx_rot_offset=0,
             theta=1e4, factor=1.0, orig_len=4096.0, beta_fast=32.0, beta_slow=1.0, magnitude=0.0)
    o.update(kw)
    rp = dsa.RopeParams(**o)
    names = [n for n, _ in dsa.RopeBuffers._fields_]
    b = dsa.RopeBuffers(*[_at(i) for i in range(len(names))])
    for k, v in (buffers or {}).items():
        setattr(b, k, v)
    p = (shape or dsa.LayerShape(top_k=4)).params()
    rg = rg or _rg(dsa)
    return dsa.lib.dsa_rope_append(ctypes.byref(p), ctypes.byref(rg), ctypes.byref(rp),
                                   ctypes.byref(b), None, None, None)


@pytest.mark.parametrize("kw", [
    dict(layout=2), dict(layout=-1), dict(scaling=4), dict(scaling=-1), dict(rot_dim=144),
    dict(rot_dim=-16), dict(rot_dim=64, rot_offset=72), dict(rot_offset=-8), dict(idx_rot_dim=80),
    dict(theta=0.0), dict(theta=float("nan")), dict(theta=float("inf")), dict(magnitude=float("nan")),
    dict(scaling=1, factor=0.0), dict(scaling=2, factor=-1.0), dict(scaling=1, factor=float("inf")),
    dict(scaling=3, orig_len=0.0), dict(scaling=3, beta_fast=1.0, beta_slow=1.0),
    dict(scaling=3, beta_fast=float("nan")), dict(q_row_stride=64), dict(k_row_stride=516),
    dict(v_row_stride=-512),
    dict(theta=1e-300, scaling=1, factor=1e-300),
])
def test_rope_invalid_parameters(dsa, kw):
    assert _rope(dsa, **kw) == dsa.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(rot_dim=24), dict(idx_rot_dim=8), dict(rot_dim=64, rot_offset=4)])
def test_rope_unsupported_parameters(dsa, kw):
    assert _rope(dsa, **kw) == dsa.DSA_ERR_UNSUPPORTED


def test_rope_shapes_and_buffers(dsa):
    inv, uns = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    S = dsa.LayerShape
    assert _rope(dsa, shape=S(top_k=4, head_dim=64)) == uns
    assert _rope(dsa, shape=S(top_k=4, idx_dim=32)) == uns
    assert _rope(dsa, shape=S(top_k=4, n_idx_heads=5)) == uns
    assert _rope(dsa, shape=S(top_k=4, n_q_heads=0)) == inv
    assert _rope(dsa, shape=S(top_k=4, idx_dtype=7)) == inv
    assert _rope(dsa, shape=S(top_k=4, idx_scale_k=0.0)) == inv
    for name in ("q_out", "k_cache", "v_cache", "q_idx_out", "k_idx_cache"):
        assert _rope(dsa, buffers={name: None}) == inv, name     # an input without its output
        assert _rope(dsa, buffers={name: _at(40) + 8}) == inv, name
    assert _rope(dsa, buffers=dict(k_cache=_at(7))) == inv       # two outputs in one place
    assert _rope(dsa, buffers=dict(q_out=_at(0) + 256)) == inv   # shifted over its input
    assert _rope(dsa, buffers=dict(q_out=_at(0)), q_row_stride=8192) == inv  # in place, not packed
    assert _rope(dsa, buffers=dict(k_cache=_at(0))) == inv       # over another input
    fp8 = S(top_k=4, idx_dtype=dsa.DSA_FP8_E4M3)
    assert _rope(dsa, shape=fp8, buffers=dict(q_idx_out=_at(3))) == inv  # in place, other type
    # pages
    for kw in (dict(page_size=100), dict(page_size=64), dict(max_pages=0), dict(page_size=128, total_kv=200)):
        rg = _rg(dsa, **dict(dict(block_table=_at(30), max_pages=4, page_size=128, total_kv=1024), **kw))
        assert _rope(dsa, rg=rg) == inv, kw
    # nothing to do: no rows, or no inputs
    assert _rope(dsa, rg=_rg(dsa, total_q=0)) == 0
    none = {n: None for n, _ in dsa.RopeBuffers._fields_}
    assert _rope(dsa, buffers=none) == 0
    assert _rope(dsa, rg=_rg(dsa, kv_offsets=None)) == inv
    assert _rope(dsa, rg=_rg(dsa, total_q=1 << 31)) == uns


# ---------------------------------------------------------------- short convolution

def _conv(dsa, rg=None, channels=64, width=4, n_states=3, sx=0, so=0, ptrs=None):
    p = dsa.ConvParams(channels, width, 1, n_states, sx, so)
    a = dict(x=_at(0), weight=_at(1), bias=_at(2), state_in=_at(3), state_out=_at(4),
             state_index=_at(5), out=_at(6))
    a.update(ptrs or {})
    rg = rg or _rg(dsa)
    return dsa.lib.dsa_short_conv(ctypes.byref(p), ctypes.byref(rg), *a.values(), None)


def test_conv_refusals(dsa):
    inv, uns = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    for kw in (dict(channels=0), dict(channels=12), dict(n_states=0), dict(n_states=-1), dict(sx=32),
               dict(sx=68), dict(so=56), dict(sx=-64)):
        assert _conv(dsa, **kw) == inv, kw
    for kw in (dict(width=1), dict(width=5), dict(channels=1 << 25)):
        assert _conv(dsa, **kw) == uns, kw
    for name in ("x", "weight", "out"):
        assert _conv(dsa, ptrs={name: None}) == inv
    for name in ("x", "weight", "bias", "state_in", "state_out", "out"):
        assert _conv(dsa, ptrs={name: _at(50) + 2}) == inv
    assert _conv(dsa, ptrs=dict(out=_at(0))) == inv                # a row's window is read after it
    assert _conv(dsa, ptrs=dict(state_out=_at(3) + 16)) == inv     # shifted over state_in
    assert _conv(dsa, ptrs=dict(out=_at(4))) == inv
    for name in ("out", "state_out"):                              # over the weights, the bias
        assert _conv(dsa, ptrs={name: _at(1)}) == inv and _conv(dsa, ptrs={name: _at(2)}) == inv
    assert _conv(dsa, rg=_rg(dsa, batch=0)) == inv
    assert dsa.lib.dsa_short_conv(None, ctypes.byref(_rg(dsa)), *([_at(0)] * 7), None) == inv


# ---------------------------------------------------------------- gated delta rule

def _delta(dsa, rg=None, decode=False, ptrs=None, ws=None, nbytes=1 << 40, **kw):
    o = dict(n_k_heads=2, n_v_heads=4, head_dim=128, qk_norm=1, norm_eps=1e-6, scale=0.0, n_states=3)
    o.update(kw)
    p = dsa.DeltaParams(**o)
    a = dict(q=_at(0), k=_at(1), v=_at(2), g=_at(3), beta=_at(4), state_in=_at(5), state_out=_at(6),
             state_index=_at(7), out=_at(8))
    a.update(ptrs or {})
    rg = rg or _rg(dsa, q=1 if decode else 64)
    if decode:
        return dsa.lib.dsa_gated_delta_decode(ctypes.byref(p), ctypes.byref(rg), *a.values(), None)
    return dsa.lib.dsa_gated_delta_prefill(ctypes.byref(p), ctypes.byref(rg), *a.values(), ws, nbytes, None)


@pytest.mark.parametrize("decode", [False, True])
def test_delta_refusals(dsa, decode):
    inv, uns = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    call = lambda **kw: _delta(dsa, decode=decode, **kw)  # noqa: E731
    for kw in (dict(n_k_heads=0), dict(n_v_heads=0), dict(n_v_heads=3), dict(norm_eps=0.0),
               dict(norm_eps=float("nan")), dict(scale=-1.0), dict(scale=float("inf")),
               dict(n_states=0), dict(n_states=-2), dict(reserved=1), dict(q_row_stride=128),
               dict(k_row_stride=260), dict(v_row_stride=256)):
        assert call(**kw) == inv, kw
    for kw in (dict(head_dim=64), dict(head_dim=256), dict(n_v_heads=1 << 17)):
        assert call(**kw) == uns, kw
    for name in ("q", "k", "v", "g", "beta", "out"):
        assert call(ptrs={name: None}) == inv, name
    for name in ("q", "k", "v", "g", "beta", "state_in", "state_out", "out"):
        assert call(ptrs={name: _at(60) + 4}) == inv, name
    for name in ("q", "k", "v", "g", "beta", "state_in", "state_out"):
        at = [n for n in ("q", "k", "v", "g", "beta", "state_in", "state_out")].index(name)
        assert call(ptrs=dict(out=_at(at))) == inv, name
    assert call(ptrs=dict(state_out=_at(5) + 128 * 128 * 4)) == inv
    assert call(rg=_rg(dsa, q=1, q_offsets=None)) == inv


def test_absent_inputs_are_not_checked(dsa):
    """Rotary append of q alone: the other heads' counts and the indexer's scales say nothing."""
    only_q = {n: None for n, _ in dsa.RopeBuffers._fields_ if n not in ("q", "q_out")}
    shape = dsa.LayerShape(top_k=4, n_kv_heads=-5, idx_dim=7, idx_scale_q=0.0)
    rg = _rg(dsa, total_q=0)
    assert _rope(dsa, rg=rg, shape=shape, buffers=only_q) == 0
    shape = dsa.LayerShape(top_k=4, n_q_heads=1 << 20)
    assert _rope(dsa, rg=rg, shape=shape, buffers=only_q) == dsa.DSA_ERR_UNSUPPORTED


def test_delta_batches_too_large(dsa):
    big = _rg(dsa, batch=1 << 24, q=1)
    assert _delta(dsa, decode=True, rg=big, n_v_heads=64, n_k_heads=64) == dsa.DSA_ERR_UNSUPPORTED
    assert _delta(dsa, rg=big, n_v_heads=64, n_k_heads=64) == dsa.DSA_ERR_UNSUPPORTED


def test_delta_decode_is_one_token_per_sequence(dsa):
    assert _delta(dsa, decode=True, rg=_rg(dsa, q=2)) == dsa.DSA_ERR_INVALID_ARG
    assert _delta(dsa, decode=True, rg=_rg(dsa, q=1, total_q=3)) == dsa.DSA_ERR_INVALID_ARG


def test_delta_workspace(dsa):
    shape = dsa.DeltaShape(2, 4)
    mn, rec = dsa.dsa_gated_delta_workspace_size(shape, _rg(dsa, batch=3, q=1000))
    # per chunk and head: three pieces of the inverse and P, ten 16 x 16 bf16 blocks each, and the
    # scalars
    assert mn == (3000 // 64 + 3) * (4 * 10 * 512 + 1024) and rec == 4 * mn
    assert dsa.dsa_gated_delta_workspace_size(shape, _rg(dsa, batch=3, q=24)) == (0, 0)
    W = dsa.DSA_ERR_WORKSPACE
    assert _delta(dsa, ws=None) == W
    assert _delta(dsa, ws=_at(9) + 16) == W
    need = dsa.dsa_gated_delta_workspace_size(dsa.DeltaShape(2, 4), _rg(dsa, q=64))[0]
    assert _delta(dsa, ws=_at(9), nbytes=need - 1) == W


def test_structures_match_the_header(dsa):
    """Sizes of the binding's structures, as the C layout rules give them."""
    assert ctypes.sizeof(dsa.RopeParams) == 6 * 4 + 6 * 8 + 5 * 8
    assert ctypes.sizeof(dsa.RopeBuffers) == 80
    assert ctypes.sizeof(dsa.ConvParams) == 32
    assert ctypes.sizeof(dsa.DeltaParams) == 56
