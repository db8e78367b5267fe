"""GPU checks of the operators around the layer where they can go wrong besides sizes: extreme values,
infinities and NaN, descriptors of which only the documented fields are filled, batches of single
tokens, captured calls and streams.  Plain 64-bit computations are the reference."""
import numpy as np
import pytest
import torch

from tests import test_gpu_hybrid as T

pytestmark = pytest.mark.gpu

dsa = None
BF16 = torch.bfloat16
U = 2.0 ** -8  # half a step of bf16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    global dsa
    import indexer_top_gated_b200 as m
    dsa = T.dsa = m
    torch.cuda.init()
    yield
    assert dsa.dsa_device_status(clear=True) == 0


def _offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _randn(seed, *shape, scale=1.0, dtype=BF16):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).cuda()


# ---------------------------------------------------------------- short convolution

LOWEST = float(torch.finfo(BF16).min)
EXTREMES = [LOWEST, -1e30, -1e20, -1e17, -1e6, -1000.0, -128.0, -104.0, -96.0, -89.0, -88.0, -87.0, -80.0, -64.0,
            -50.0, -41.0, -40.0, -20.0, -1.0, -1e-30, 0.0, 1e-30, 1.0, 20.0, 100.0, 1e20, -LOWEST, float("inf"),
            float("-inf"), float("nan")]


@pytest.mark.parametrize("lens", [[1], [9], [30000]])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_conv_activation_of_extreme_values(lens, width):
    """y / (1 + e^-y) of every pair of extreme values in neighbouring channels (they share registers).
    The last tap is 1 and the others 0, so y is x itself.  Tolerance: the output's rounding, 2^-15 of
    the value (an exponent of up to 127 in fp32 is off by 127 half steps, twice that with its factor
    log2 e) and 2^-119, above 88 * 2^-126, for what a reciprocal flushed to zero leaves out."""
    pairs = torch.tensor([v for a in EXTREMES for b in EXTREMES for v in (a, b)], dtype=BF16)
    c = len(pairs)
    n = sum(lens)
    x = torch.zeros(n, c, dtype=BF16, device="cuda")
    rows = sorted({0, n // 2, n - 1})  # alone in their windows
    x[rows] = pairs.cuda()
    weight = torch.zeros(c, width, dtype=BF16, device="cuda")
    weight[:, -1] = 1.0
    out = torch.full_like(x, 7.0)
    off = _offsets(lens)
    dsa.dsa_short_conv(dsa.ConvShape(c, width), dsa.ragged(off, off, lens, lens), x, weight, out)
    y = pairs.double()
    ref = y / (1 + torch.exp(-y))
    for r in rows:
        got = out[r].double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref)), r
        wild = torch.isnan(ref) | torch.isinf(ref)
        assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)])
        over = ((got - ref).abs() > (U + 2.0 ** -15) * ref.abs() + 2.0 ** -119) & ~wild
        assert not over.any(), (r, [(float(y[i]), float(got[i]), float(ref[i])) for i in torch.nonzero(over)[:4, 0]])


@pytest.mark.parametrize("max_q_len", [0, 1, -7, 1 << 30])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_conv_results_do_not_depend_on_max_q_len(max_q_len, width):
    """Of the descriptor only batch, q_offsets and total_q are filled; max_q_len is whatever it is."""
    lens, c = [70, 0, 1, 33, 2], 264
    n, slots = sum(lens), len(lens)
    x, weight, state = _randn(1, n, c), _randn(2, c, width), _randn(3, slots, width - 1, c)
    off = _offsets(lens)
    conv = dsa.ConvShape(c, width)
    want, want_state = torch.empty_like(x), torch.empty_like(state)
    dsa.dsa_short_conv(conv, dsa.ragged(off, off, lens, lens), x, weight, want, state_in=state, state_out=want_state)
    rg = dsa.Ragged(slots, off.data_ptr(), None, max_q_len, 0, n, 0)
    out, st = torch.full_like(x, 7.0), torch.full_like(state, 7.0)
    dsa.dsa_short_conv(conv, rg, x, weight, out, state_in=state, state_out=st)
    assert torch.equal(out, want) and torch.equal(st, want_state)


# ---------------------------------------------------------------- gated delta rule

def _delta_states(d):
    """States after token after token, 64 bits, on the GPU: [sequence, Hv, dv, dk]."""
    n, rep = d.n, d.hv // d.hk
    k, v = d.k[:n].double(), d.v[:n].double()
    if d.norm:
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    k = k.repeat_interleave(rep, 1)
    alpha, beta = torch.exp(d.g[:n].double()), d.beta[:n].double()
    S = d.state[d.index.long()].double()
    at = 0
    for b, m in enumerate(d.lens):
        s = S[b]
        for t in range(at, at + m):
            s *= alpha[t][:, None, None]
            u = beta[t][:, None] * (v[t] - (s @ k[t][..., None])[..., 0])
            s += u[..., None] * k[t][:, None, :]
        at += m
    return S


# few heads; 32 columns a CTA; whole heads (of 40, and of 148: one for each SM)
@pytest.mark.parametrize("hk,hv,lens", [(1, 2, [1300]), (2, 24, [1300]), (2, 40, [1300]), (4, 148, [1300, 5])])
def test_delta_decays_of_each_chunk_its_own(hk, hv, lens):
    """Chunks of 64 whose decays differ by factors from one to the next and to the one after it (which
    takes its place in shared memory).  A chunk's decay in another's place moves the state by more than
    a tenth of itself; tolerance 1e-5 of each head's."""
    d = T._Delta(lens, hk, hv, rate=0.0)
    n = sum(lens)
    per_chunk = torch.tensor([0.0, -0.4, -1.2, 0.0, -2.5])[torch.arange(n) // 64 % 5]
    per_head = torch.linspace(0.5, 1.0, hv)
    d.g = (per_chunk[:, None] * per_head / 64).cuda().contiguous()
    _, st = d.call()
    want = _delta_states(d)
    off = (st[d.index.long()].double() - want).flatten(2).norm(dim=-1)
    assert (off <= 1e-5 * want.flatten(2).norm(dim=-1)).all(), float((off / want.flatten(2).norm(dim=-1)).max())


# few heads (16 value columns a CTA); 32 columns; whole heads
@pytest.mark.parametrize("hk,hv", [(1, 2), (2, 24), (2, 40)])
def test_delta_state_is_of_fp32_quality(hk, hv):
    """Every third bf16 piece is there.  Two pieces round a value to 2.7e-6 of itself (rms: 1.6e-3 for
    a piece, of a remainder of 1.6e-3).  In S of K S^T alone (by design) that moves the next state by
    sqrt(64 tokens / 128 columns) * 0.54 (write strength) * 0.63 (mean decay inside a chunk) * 2.7e-6 =
    6.5e-7 of the old one, less what decays (e^-1 a chunk).  In T, X or U it moves what a chunk writes,
    most of the state here, by 2.7e-6.  Hence 1e-6."""
    d = T._Delta([640], hk, hv, rate=0.02)
    _, st = d.call()
    want = _delta_states(d)
    got = st[d.index.long()].double()
    assert (got - want).norm() <= 1e-6 * want.norm(), float((got - want).norm() / want.norm())


@pytest.mark.parametrize("hv", [2, 24, 40])
@pytest.mark.parametrize("kscale", [0.5, 1.2])
@pytest.mark.parametrize("lens", [[300, 9]])
def test_delta_keys_of_other_lengths(lens, kscale, hv):
    """qk_norm = 0 with keys that are not of unit length (beta |k|^2 < 2: the rule still contracts)."""
    d = T._Delta(lens, 2, hv, norm=False, kscale=kscale)
    d.check(*d.call())


# ---------------------------------------------------------------- single tokens

@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("lens", [[1, 0, 1, 1, 0], [1] * 256])
def test_conv_single_tokens(lens, width):
    """Decode batches: one token or none for each sequence, slots in any order, some of them not kept."""
    c, n, slots = 1096, sum(lens), len(lens) + 7
    x, weight, bias = _randn(1, n, c), _randn(2, c, width), _randn(3, c)
    state = _randn(4, slots, width - 1, c)
    index = torch.randperm(slots, generator=torch.Generator().manual_seed(5))[:len(lens)].to(torch.int32)
    index[1], index[2] = -1, slots  # of an empty sequence (or a token), and of a token
    off = _offsets(lens)
    rg = dsa.ragged(off, off, lens, lens)
    assert rg.max_q_len == 1
    conv = dsa.ConvShape(c, width)
    out, st = torch.full_like(x, 7.0), torch.full_like(state, 7.0)
    dsa.dsa_short_conv(conv, rg, x, weight, out, bias=bias, state_in=state, state_out=st, state_index=index.cuda())
    ref, mag, states = T._conv_ref(x, lens, weight, bias, True, state, index.tolist(), slots)
    T._near(out, ref, U * ref.abs() + 2.0 ** -20 * 1.1 * mag, "out")
    for s in range(slots):
        want = states[s] if s in states else torch.full((width - 1, c), 7.0, dtype=torch.float64)
        assert torch.equal(st[s].double().cpu(), want), s
    inplace, again = state.clone(), torch.full_like(x, 7.0)
    dsa.dsa_short_conv(conv, rg, x, weight, again, bias=bias, state_in=inplace, state_out=inplace, state_index=index.cuda())
    assert torch.equal(again, out)
    for s in range(slots):
        assert torch.equal(inplace[s], st[s] if s in states else state[s]), s


# ---------------------------------------------------------------- infinities, NaN, lowest values

def _same(got, ref, tol, what):
    """NaN where the reference has it, the same infinities, the rest within tol."""
    got, ref, tol = got.double().cpu(), ref.double().cpu(), tol.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), what
    rest = ~inf & ~torch.isnan(ref)
    assert ((got - ref).abs() <= tol)[rest].all(), (what, float((got - ref).abs()[rest].max()))


@pytest.mark.parametrize("width", [2, 4])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_infinities_and_nan_stay_in_their_windows(silu, width):
    lens, c = [9, 40], 64
    x, weight = _randn(1, sum(lens), c), _randn(2, c, width)
    state = _randn(3, 2, width - 1, c)
    x[2, 5], x[8, 6], x[20, 7], x[30, 8] = float("inf"), float("nan"), float("-inf"), float("nan")
    state[1, -1, 9] = float("inf")
    off = _offsets(lens)
    out, st = torch.empty_like(x), torch.empty_like(state)
    dsa.dsa_short_conv(dsa.ConvShape(c, width, silu=silu), dsa.ragged(off, off, lens, lens), x, weight, out,
                       state_in=state, state_out=st)
    ref, mag, states = T._conv_ref(x, lens, weight, None, silu, state, None, 2)
    _same(out, ref, U * ref.abs() + 2.0 ** -20 * 1.1 * mag, "out")
    for s in (0, 1):
        _same(st[s], states[s], torch.zeros_like(states[s]), "state")


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("fp8", [False, True])
def test_rope_extreme_values(layout, fp8):
    """In one element of a pair each (two lowest values together overflow): both elements of the pair
    follow the formula, the others do not notice.  e4m3 saturates infinities, keeps NaN."""
    rope = dsa.RopeShape(layout=layout, rot_dim=64, rot_offset=32, idx_rot_dim=32, idx_rot_offset=16)
    t = T._Rope([3, 6], [0, 70], heads=(2, 1, 2), fp8=fp8, page=128)
    wild = [LOWEST, -LOWEST, float("inf"), float("-inf"), float("nan")]
    for src, first, r in ((t.q, 32, 64), (t.k, 32, 64), (t.q_idx, 16, 32), (t.k_idx, 16, 32)):
        for i, w in enumerate(wild):
            pair = 3 + i
            src[i % 3::2, :, first + (pair if layout == 0 else 2 * pair + 1)] = w
        src[:, :, 1] = float("inf")     # outside the rotated part
        src[0, :, 2] = float("nan")
    t.v[:, 0, :5] = torch.tensor(wild, dtype=BF16, device="cuda")
    t.call(rope)
    rows = torch.arange(t.n)
    for src, name, at, r, o in ((t.q, "q_out", rows, 64, 32), (t.k, "k_cache", t.to, 64, 32),
                                (t.q_idx, "q_idx_out", rows, 32, 16), (t.k_idx, "k_idx_cache", t.to, 32, 16)):
        ref, mag = T._turned(src, t.pos, rope, r, o)
        if fp8 and "idx" in name:
            ref = ref.clamp(-448, 448)
            tol = 2.0 ** -4 * ref.abs() + 2.0 ** -10 + 2.0 ** -20 * mag
        else:
            tol = U * ref.abs() + 2.0 ** -20 * mag
        _same(t.out[name].float().cpu()[at], ref, tol, name)
    assert torch.equal(t.out["v_cache"].view(torch.int16)[t.to.cuda()], t.v.contiguous().view(torch.int16))


# ---------------------------------------------------------------- capture, replay, streams

def _captured(run):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    return graph


def test_rope_captured_decode_steps():
    """A captured call replayed as the caches grow: lengths and rows change on the device."""
    rope = dsa.RopeShape(theta=1e6)
    t = T._Rope([1, 1, 1], [130, 3, 250], page=128)
    fresh = T._Rope([1, 1, 1], [130, 3, 250], page=128, seed=50)
    graph = _captured(lambda: dsa.dsa_rope_append(t.shape, t.rg, rope, q=t.q, k=t.k, v=t.v, q_idx=t.q_idx,
                                                  k_idx=t.k_idx, **t.out))
    for step in range(4):
        for name in ("q", "k", "v", "q_idx", "k_idx"):
            getattr(t, name).copy_(getattr(fresh, name) * (step + 1))
        for o in t.out.values():
            o.copy_(torch.full_like(o, 7.0, dtype=torch.float32).to(o.dtype))
        t.keep[1].copy_(_offsets([n + step for n in t.kv_lens]))
        graph.replay()
        torch.cuda.synchronize()
        pos = t.pos + step
        to = torch.stack([t.table[b].long()[p // 128] * 128 + p % 128 for b, p in enumerate(pos.tolist())])
        t.check(rope, pos=pos, to=to)


@pytest.mark.parametrize("lens", [[1] * 9, [40, 3, 0, 17]])
def test_conv_captured_steps_hand_the_state_on(lens):
    c, w, n = 520, 4, sum(lens)
    xs, weight = [_randn(10 + i, n, c) for i in range(3)], _randn(2, c, w)
    off = _offsets(lens)
    rg, conv = dsa.ragged(off, off, lens, lens), dsa.ConvShape(c, w)
    want_state, want = _randn(3, len(lens), w - 1, c), []
    state, x, out = want_state.clone(), xs[0].clone(), torch.empty(n, c, dtype=BF16, device="cuda")
    for v in xs:
        y = torch.empty_like(out)
        dsa.dsa_short_conv(conv, rg, v, weight, y, state_in=want_state, state_out=want_state)
        want.append(y)
    start = state.clone()
    graph = _captured(lambda: dsa.dsa_short_conv(conv, rg, x, weight, out, state_in=state, state_out=state))
    state.copy_(start)
    for v, y in zip(xs, want):
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)
    assert torch.equal(state, want_state)


def test_two_streams_at_once():
    rope, conv = dsa.RopeShape(), dsa.ConvShape(2048, 4)
    lens = [700, 0, 900]
    off, x, weight = _offsets(lens), _randn(1, 1600, 2048), _randn(2, 2048, 4)
    rg = dsa.ragged(off, off, lens, lens)
    want = torch.empty_like(x)
    dsa.dsa_short_conv(conv, rg, x, weight, want)
    batches = [T._Rope(lens, [5, 9, 100], seed=i) for i in (0, 30)]
    outs = [torch.full_like(x, 7.0) for _ in range(2)]
    torch.cuda.synchronize()
    for s, t, o in zip((torch.cuda.Stream(), torch.cuda.Stream()), batches, outs):
        with torch.cuda.stream(s):
            for _ in range(3):
                dsa.dsa_rope_append(t.shape, t.rg, rope, q=t.q, k=t.k, v=t.v, q_idx=t.q_idx, k_idx=t.k_idx, **t.out)
                dsa.dsa_short_conv(conv, rg, x, weight, o)
    torch.cuda.synchronize()
    for t, o in zip(batches, outs):
        t.check(rope)
        assert torch.equal(o, want)


# ---------------------------------------------------------------- the binding

def test_every_operator_refuses_repeated_rows():
    t = T._Rope([4], [3])
    kw = dict(q=t.q, k=t.k, v=t.v, q_idx=t.q_idx, k_idx=t.k_idx, **t.out)
    for name in ("q", "k", "v", "q_idx", "k_idx"):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_rope_append(t.shape, t.rg, dsa.RopeShape(), **dict(kw, **{name: kw[name][:1].expand_as(kw[name])}))
    off, x, w = _offsets([6]), _randn(1, 6, 64), _randn(2, 64, 4)
    rg = dsa.ragged(off, off, [6], [6])
    for a, b in ((x[:1].expand_as(x), torch.empty_like(x)), (x, torch.empty_like(x)[:1].expand_as(x))):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_short_conv(dsa.ConvShape(64, 4), rg, a, w, b)
    d = T._Delta([7])
    out = torch.empty(7, 4, 128, dtype=BF16, device="cuda")
    args = dict(q=d.q, k=d.k, v=d.v, g=d.g, beta=d.beta, out=out)
    for name in args:
        with pytest.raises(dsa.DsaError):
            dsa.dsa_gated_delta_prefill(d.shape, d.rg, **dict(args, **{name: args[name][:1].expand_as(args[name])}))


# ---------------------------------------------------------------- nothing to do

def test_batches_without_tokens_hand_states_on():
    """Sequences without rows: tensors of no rows, states copied to where they are kept, nothing else."""
    lens, c = [0, 0, 0], 136
    off = _offsets(lens)
    rg = dsa.ragged(off, off, lens, lens)
    none = lambda *s: torch.empty(0, *s, dtype=BF16, device="cuda")  # noqa: E731
    index = torch.tensor([4, 0, 9], dtype=torch.int32, device="cuda")  # the last is not kept
    state = _randn(1, 5, 3, c)
    st = torch.full_like(state, 7.0)
    dsa.dsa_short_conv(dsa.ConvShape(c, 4), rg, none(c), _randn(2, c, 4), none(c), state_in=state, state_out=st, state_index=index)
    for s in range(5):
        assert torch.equal(st[s], state[s] if s in (0, 4) else torch.full_like(state[s], 7.0)), s
    state = _randn(3, 5, 2, 128, 128, dtype=torch.float32)
    gates = torch.empty(0, 2, device="cuda")
    for call in (dsa.dsa_gated_delta_prefill, dsa.dsa_gated_delta_decode):
        st = torch.full_like(state, 7.0)
        call(dsa.DeltaShape(1, 2), rg, none(1, 128), none(1, 128), none(2, 128), gates, gates, none(2, 128),
             state_in=state, state_out=st, state_index=index)
        for s in range(5):
            assert torch.equal(st[s], state[s] if s in (0, 4) else torch.full_like(state[s], 7.0)), s
        # from nothing: the state of no tokens is zero
        call(dsa.DeltaShape(1, 2), rg, none(1, 128), none(1, 128), none(2, 128), gates, gates, none(2, 128),
             state_out=st, state_index=index)
        assert not st[0].any() and not st[4].any() and (st[1:4] == 7.0).all()
    shape = dsa.LayerShape(n_idx_heads=1, n_q_heads=2, n_kv_heads=1, top_k=4)
    dsa.dsa_rope_append(shape, rg, dsa.RopeShape(), q=none(2, 128), q_out=none(2, 128), k=none(1, 128), k_cache=none(1, 128))


def test_calls_on_a_given_stream():
    """stream= takes precedence over the current one."""
    s = torch.cuda.Stream()
    x, w = _randn(1, 300, 2048), _randn(2, 2048, 4)
    off = _offsets([300])
    rg, conv = dsa.ragged(off, off, [300], [300]), dsa.ConvShape(2048, 4)
    want, out = torch.empty_like(x), torch.full_like(x, 7.0)
    dsa.dsa_short_conv(conv, rg, x, w, want)
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        late.copy_(x)
    dsa.dsa_short_conv(conv, rg, late, w, out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
