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
