"""GPU checks of the operators around the layer against plain 64-bit computations: rotary
positions with the append to the caches, the short convolution, the gated delta rule, and all of
them in front of the mixing attention.

Tolerances.  u = 2^-8 is half a step of bf16, 2^-24 of fp32, 2^-4 of e4m3.
 - Rotation and convolution are a few fp32 operations on exact inputs, rounded once: u |ref| plus
   2^-20 of the sum of the magnitudes that enter (16 fp32 half steps: two to four products, their
   sums, the angle's or the exponential's error).
 - Delta rule, token by token: fp32 sums of 128 terms, rounded once: u |ref| plus 2^-18 of the
   magnitudes.  In chunks: P enters its product with U rounded to bf16, hence also
   u sum_j |P_ij U_j|.
 - Its state: the two-piece form of S in K S^T leaves out at most 2^-16 of an element, 4.4e-6 rms
   (uniform), and a chunk replaces at most all of the state: 1e-5 of its 2-norm.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

dsa = None
BF16 = torch.bfloat16
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    global dsa
    import indexer_top_gated_b200 as m
    dsa = m
    torch.cuda.init()
    yield
    assert dsa.dsa_device_status(clear=True) == 0


def _offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _randn(seed, *shape, scale=1.0, dtype=BF16):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).cuda()


def _near(got, ref, tol, what):
    got, ref, tol = got.double().cpu(), ref.double().cpu(), tol.double().cpu()
    assert torch.isfinite(ref).all(), what
    over = ((got - ref).abs() > tol) | ~torch.isfinite(got)
    assert not over.any(), (what, int(over.sum()), float((got - ref).abs().max()))


# ---------------------------------------------------------------- rotary append

def _freqs(rope, r):
    i = torch.arange(r // 2, dtype=torch.float64)
    theta = rope.theta
    if rope.scaling == dsa.DSA_ROPE_SCALE_NTK and r > 2:
        theta *= rope.factor ** (r / (r - 2))
    f = theta ** (-2 * i / r)
    if rope.scaling == dsa.DSA_ROPE_SCALE_LINEAR:
        f = f / rope.factor
    if rope.scaling == dsa.DSA_ROPE_SCALE_BY_PARTS:
        y = ((rope.orig_len * f / (2 * math.pi) - rope.beta_slow) / (rope.beta_fast - rope.beta_slow)).clamp(0, 1)
        f = f * (y + (1 - y) / rope.factor)
    return f


def _turned(x, pos, rope, r, off):
    """(value, sum of the magnitudes that enter it), 64 bits."""
    x = x.double().cpu()
    y, mag = x.clone(), x.abs()
    if r:
        ang = pos.double().cpu()[:, None] * _freqs(rope, r)
        c, s = ang.cos()[:, None] * rope.magnitude, ang.sin()[:, None] * rope.magnitude
        h = x[..., off:off + r]
        a, b = (h[..., :r // 2], h[..., r // 2:]) if rope.layout == dsa.DSA_ROPE_HALF else (h[..., 0::2], h[..., 1::2])
        for d, fa, fb in ((y, a * c - b * s, a * s + b * c), (mag, (a.abs() + b.abs()) * rope.magnitude,) * 1 + ((a.abs() + b.abs()) * rope.magnitude,)):
            if rope.layout == dsa.DSA_ROPE_HALF:
                d[..., off:off + r // 2], d[..., off + r // 2:off + r] = fa, fb
            else:
                d[..., off:off + r:2], d[..., off + 1:off + r:2] = fa, fb
    return y, mag


class _Rope:
    """One batch: inputs as slices of fused rows, caches (contiguous or shuffled pages) of known
    contents, the expected cache row of each query row."""

    def __init__(self, q_lens, hists, heads=(8, 2, 4), page=0, fp8=False, seed=0, extra_rows=0, scale=(1.0, 1.0)):
        self.q_lens, self.kv_lens = q_lens, [h + n for h, n in zip(hists, q_lens)]
        self.hq, self.hkv, self.hi = heads
        self.n, self.total = sum(q_lens), sum(q_lens) + extra_rows
        t = self.total
        fused = _randn(seed, t, (self.hq + 2 * self.hkv) * 128)
        a, b = self.hq * 128, (self.hq + self.hkv) * 128
        self.q, self.k, self.v = (fused[:, :a].view(t, self.hq, 128), fused[:, a:b].view(t, self.hkv, 128),
                                  fused[:, b:].view(t, self.hkv, 128))
        fi = _randn(seed + 1, t, 2 * self.hi * 64)
        self.q_idx, self.k_idx = fi[:, :self.hi * 64].view(t, self.hi, 64), fi[:, self.hi * 64:].view(t, self.hi, 64)
        self.shape = dsa.LayerShape(n_idx_heads=self.hi, n_q_heads=self.hq, n_kv_heads=self.hkv, top_k=16,
                                    idx_dtype=dsa.DSA_FP8_E4M3 if fp8 else dsa.DSA_BF16,
                                    idx_scale_q=scale[0], idx_scale_k=scale[1])
        qo, ko = _offsets(q_lens), _offsets(self.kv_lens)
        self.keep = [qo, ko]
        pos = [torch.arange(L - n, L) for n, L in zip(q_lens, self.kv_lens)]
        self.pos = torch.cat(pos) if pos else torch.zeros(0, dtype=torch.long)
        if page:
            pages = [-(-L // page) for L in self.kv_lens]
            perm = torch.randperm(sum(pages) + 2, generator=torch.Generator().manual_seed(seed))
            self.table = torch.full((len(q_lens), max(1, max(pages))), -1, dtype=torch.int32)
            at = 0
            for s, c in enumerate(pages):
                self.table[s, :c] = perm[at:at + c].to(torch.int32)
                at += c
            self.rows = (sum(pages) + 2) * page
            self.to = torch.cat([self.table[s].long()[p // page] * page + p % page for s, p in enumerate(pos)])
            self.dev_table = self.table.cuda()
            self.rg = dsa.ragged(qo, ko, q_lens, self.kv_lens, block_table=self.dev_table, page_size=page,
                                 cache_rows=self.rows)
        else:
            self.rows = sum(self.kv_lens)
            self.to = torch.cat([int(o) + p for o, p in zip(ko.cpu(), pos)])
            self.rg = dsa.ragged(qo, ko, q_lens, self.kv_lens)
        self.rg.total_q = t
        idx_type = torch.float8_e4m3fn if fp8 else BF16
        self.out = dict(q_out=torch.full((t, self.hq, 128), 7.0, dtype=BF16, device="cuda"),
                        k_cache=torch.full((self.rows, self.hkv, 128), 7.0, dtype=BF16, device="cuda"),
                        v_cache=torch.full((self.rows, self.hkv, 128), 7.0, dtype=BF16, device="cuda"),
                        q_idx_out=torch.full((t, self.hi, 64), 7.0, device="cuda").to(idx_type),
                        k_idx_cache=torch.full((self.rows, self.hi, 64), 7.0, device="cuda").to(idx_type))
        self.fp8, self.scale = fp8, scale

    def call(self, rope, **kw):
        args = dict(q=self.q, k=self.k, v=self.v, q_idx=self.q_idx, k_idx=self.k_idx, **self.out)
        args.update(kw)
        dsa.dsa_rope_append(self.shape, self.rg, rope, **args)
        torch.cuda.synchronize()

    def check(self, rope, pos=None, to=None):
        pos = self.pos if pos is None else pos
        to = self.to if to is None else to
        rows = torch.arange(self.n)
        for src, name, at, r, off, sc in (
                (self.q, "q_out", rows, rope.rot_dim, rope.rot_offset, None),
                (self.k, "k_cache", to, rope.rot_dim, rope.rot_offset, None),
                (self.v, "v_cache", to, 0, 0, None),
                (self.q_idx, "q_idx_out", rows, rope.idx_rot_dim, rope.idx_rot_offset, self.scale[0]),
                (self.k_idx, "k_idx_cache", to, rope.idx_rot_dim, rope.idx_rot_offset, self.scale[1])):
            got = self.out[name].float().cpu()
            ref, mag = _turned(src[:self.n], pos, rope, r, off)
            if sc is not None and self.fp8:
                ref, mag = (ref / sc).clamp(-448, 448), mag / sc
                tol = 2.0 ** -4 * ref.abs() + 2.0 ** -10 + 2.0 ** -20 * mag  # 2^-10: half the smallest step
            else:
                tol = U * ref.abs() + 2.0 ** -20 * mag
            live = at >= 0
            _near(got[at[live]], ref[live], tol[live], name)
            rest = torch.ones(got.shape[0], dtype=torch.bool)
            rest[at[live]] = False
            assert (got[rest] == 7.0).all(), f"{name}: rows that are not the batch's were written"


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rot,off,irot,ioff", [(128, 0, 64, 0), (64, 64, 32, 32), (48, 8, 16, 40), (0, 0, 0, 0), (16, 0, 64, 0)])
@pytest.mark.parametrize("page", [0, 128])
def test_rope_layouts(layout, rot, off, irot, ioff, page):
    rope = dsa.RopeShape(layout=layout, rot_dim=rot, rot_offset=off, idx_rot_dim=irot, idx_rot_offset=ioff, magnitude=1.25)
    t = _Rope([1, 0, 130, 7], [300, 5, 0, 121], page=page)
    t.call(rope)
    t.check(rope)


@pytest.mark.parametrize("scaling", [0, 1, 2, 3])
@pytest.mark.parametrize("fp8", [False, True])
def test_rope_scaling_and_e4m3(scaling, fp8):
    rope = dsa.RopeShape(scaling=scaling, factor=7.5, theta=5e5, layout=scaling & 1)
    t = _Rope([3, 40], [100000, 9], heads=(6, 3, 3), fp8=fp8, scale=(0.25, 0.004), page=1024)
    t.call(rope)
    t.check(rope)


def test_rope_many_rows():
    """More rows than one per CTA is used for, and an odd number of them."""
    rope = dsa.RopeShape()
    t = _Rope([4801, 0, 2], [0, 3, 1], heads=(2, 1, 1))
    t.call(rope)
    t.check(rope)


def test_rope_positions_far_and_negative():
    rope = dsa.RopeShape(theta=1e4, layout=1)
    t = _Rope([9], [50])
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 30, 16777217, 123456789, 7], dtype=torch.int32)
    t.call(rope, positions=pos.cuda())
    t.check(rope, pos=pos)  # cache rows are those of the rows' own places


def test_rope_padded_batch_leaves_rows():
    rope = dsa.RopeShape()
    t = _Rope([2, 3], [4, 5], extra_rows=6)
    t.call(rope)
    t.check(rope)


def test_rope_bad_pages_are_counted():
    rope = dsa.RopeShape()
    t = _Rope([4, 4, 4], [254, 254, 254], page=128)
    t.dev_table[1, 2] = 10 ** 6
    t.dev_table[2, 1] = -3
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t.call(rope, err_count=err)
    to = t.to.clone()
    to[6:8] = -1   # positions 256, 257 of sequence 1
    to[8:10] = -1  # positions 254, 255 of sequence 2
    t.check(rope, to=to)
    assert int(err.item()) == 4


def test_rope_in_place_and_parts_of_the_call():
    rope = dsa.RopeShape()
    t = _Rope([5, 6], [7, 0])
    q, qi = t.q.contiguous(), t.q_idx.contiguous()
    want = _turned(q, t.pos, rope, 128, 0)[0], _turned(qi, t.pos, rope, 64, 0)[0]
    k0 = t.out["k_cache"].clone()
    dsa.dsa_rope_append(t.shape, t.rg, rope, q=q, q_out=q, q_idx=qi, q_idx_out=qi)
    torch.cuda.synchronize()
    for got, ref, mag in ((q, want[0], t.q), (qi, want[1], t.q_idx)):
        _near(got, ref, U * ref.abs() + 2.0 ** -18 * mag.double().cpu().abs().amax(), "in place")
    assert torch.equal(t.out["k_cache"], k0)
    # heads of a decode row only: k and v without q
    dsa.dsa_rope_append(t.shape, t.rg, rope, k=t.k, k_cache=t.out["k_cache"], v=t.v, v_cache=t.out["v_cache"])
    torch.cuda.synchronize()
    assert torch.equal(t.out["v_cache"].cpu()[t.to], t.v.cpu())


# ---------------------------------------------------------------- short convolution

def _conv_ref(x, lens, weight, bias, silu, state_in, index, n_states):
    """(out, magnitudes, {slot: new state}), 64 bits."""
    w = weight.shape[1]
    x, wt = x.double().cpu(), weight.double().cpu()
    out, mag, states, at = [], [], {}, 0
    for b, n in enumerate(lens):
        s = index[b] if index is not None else b
        kept = 0 <= s < n_states
        old = state_in[s].double().cpu() if kept and state_in is not None else torch.zeros(w - 1, x.shape[1], dtype=torch.float64)
        rows = torch.cat([old, x[at:at + n]])
        if n:
            win = rows.unfold(0, w, 1)
            y, m = (win * wt).sum(-1), (win * wt).abs().sum(-1)
            if bias is not None:
                y, m = y + bias.double().cpu(), m + bias.double().cpu().abs()
            out.append(y * torch.sigmoid(y) if silu else y)
            mag.append(m)
        if kept:
            states[s] = rows[n:]
        at += n
    return torch.cat(out), torch.cat(mag), states


@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("silu,bias", [(True, False), (False, True)])
@pytest.mark.parametrize("lens", [[1], [0, 1, 2, 3, 4], [8, 7, 9, 0, 33, 65], [31, 32, 97, 1]])
def test_conv(width, silu, bias, lens):
    c, slots = 1096, len(lens) + 4
    n = sum(lens)
    x = _randn(1, n + 5, c + 24)[:, 8:c + 8]  # rows inside wider ones, five behind the last sequence
    weight, b = _randn(2, c, width), _randn(3, c) if bias else None
    state_in = _randn(4, slots, width - 1, c)
    index = torch.randperm(slots, generator=torch.Generator().manual_seed(5))[:len(lens)].to(torch.int32)
    if len(lens) > 2:
        index[0], index[2] = -1, slots + 3  # not kept
    state_out = torch.full_like(state_in, 7.0)
    out = torch.full((n + 5, c), 7.0, dtype=BF16, device="cuda")
    off = _offsets(lens)
    rg = dsa.ragged(off, off, lens, lens)
    rg.total_q = n + 5
    conv = dsa.ConvShape(c, width, silu=silu)
    dsa.dsa_short_conv(conv, rg, x, weight, out, bias=b, state_in=state_in, state_out=state_out, state_index=index.cuda())
    ref, mag, states = _conv_ref(x[:n], lens, weight, b, silu, state_in, index.tolist(), slots)
    # |d silu / dy| <= 1.1
    _near(out[:n], ref, U * ref.abs() + 2.0 ** -20 * 1.1 * mag, "out")
    assert (out[n:] == 7.0).all()
    for s in range(slots):
        want = states[s] if s in states else torch.full((width - 1, c), 7.0, dtype=torch.float64)
        assert torch.equal(state_out[s].double().cpu(), want), s
    # in place, the same
    again, state = torch.empty_like(out), state_in.clone()
    dsa.dsa_short_conv(conv, rg, x, weight, again, bias=b, state_in=state, state_out=state, state_index=index.cuda())
    assert torch.equal(again[:n], out[:n])
    for s in states:
        assert torch.equal(state[s], state_out[s])


def test_conv_long_rows_use_long_runs_and_chunks_join():
    """A batch large enough for the long runs, and the same rows as two calls that hand the state on."""
    lens, c, w = [20000, 333], 2048, 4
    x, weight = _randn(1, sum(lens), c), _randn(2, c, w)
    off = _offsets(lens)
    whole, st = torch.empty_like(x), torch.empty(2, w - 1, c, dtype=BF16, device="cuda")
    conv = dsa.ConvShape(c, w)
    dsa.dsa_short_conv(conv, dsa.ragged(off, off, lens, lens), x, weight, whole, state_out=st)
    ref, mag, states = _conv_ref(x, lens, weight, None, True, None, None, 2)
    _near(whole, ref, U * ref.abs() + 2.0 ** -20 * 1.1 * mag, "out")
    cut = [1002, 17]
    parts = [torch.cat([x[:cut[0]], x[lens[0]:lens[0] + cut[1]]]), torch.cat([x[cut[0]:lens[0]], x[lens[0] + cut[1]:]])]
    state, got = torch.zeros_like(st), []
    for p, ln in zip(parts, (cut, [a - b for a, b in zip(lens, cut)])):
        o, y = _offsets(ln), torch.empty_like(p)
        dsa.dsa_short_conv(conv, dsa.ragged(o, o, ln, ln), p, weight, y, state_in=state, state_out=state)
        got.append(y)
    joined = torch.cat([got[0][:cut[0]], got[1][:lens[0] - cut[0]], got[0][cut[0]:], got[1][lens[0] - cut[0]:]])
    assert torch.equal(joined, whole) and torch.equal(state, st)


# ---------------------------------------------------------------- gated delta rule

class _Delta:
    def __init__(self, lens, hk=2, hv=4, norm=True, seed=0, rate=0.2, extra_rows=0, slots=None, g=None, beta=None, kscale=1.0):
        self.lens, self.hk, self.hv, self.norm = lens, hk, hv, norm
        self.n = sum(lens)
        t = self.n + extra_rows
        fused = _randn(seed, t, (2 * hk + hv) * 128)
        self.q, self.k = fused[:, :hk * 128].view(t, hk, 128), fused[:, hk * 128:2 * hk * 128].view(t, hk, 128)
        self.v = fused[:, 2 * hk * 128:].view(t, hv, 128)
        if not norm:
            self.k.copy_(self.k.float() / self.k.float().norm(dim=-1, keepdim=True) * kscale)
        self.g = -rate * torch.nn.functional.softplus(_randn(seed + 1, t, hv, dtype=torch.float32)) if g is None else g.cuda()
        self.beta = torch.sigmoid(_randn(seed + 2, t, hv, dtype=torch.float32)) if beta is None else beta.cuda()
        self.slots = len(lens) + 2 if slots is None else slots
        self.state = _randn(seed + 3, self.slots, hv, 128, 128, dtype=torch.float32)
        self.index = torch.randperm(self.slots, generator=torch.Generator().manual_seed(seed))[:len(lens)].to(torch.int32).cuda()
        off = _offsets(lens)
        self.keep = off
        self.rg = dsa.ragged(off, off, lens, lens)
        self.rg.total_q = t
        self.shape = dsa.DeltaShape(hk, hv, qk_norm=norm, norm_eps=1e-6)

    def call(self, state_in="own", state_out=None, ws_bytes=None, decode=False, ragged=None, index="own"):
        out = torch.full((self.q.shape[0], self.hv, 128), 7.0, dtype=BF16, device="cuda")
        st = torch.full_like(self.state, 7.0) if state_out is None else state_out
        kw = dict(state_in=self.state if isinstance(state_in, str) else state_in, state_out=st,
                  state_index=self.index if isinstance(index, str) else index)
        rg = ragged or self.rg
        args = (self.shape, rg, self.q, self.k, self.v, self.g, self.beta, out)
        if decode:
            dsa.dsa_gated_delta_decode(*args, **kw)
        else:
            size = dsa.dsa_gated_delta_workspace_size(self.shape, rg)[1] if ws_bytes is None else ws_bytes
            dsa.dsa_gated_delta_prefill(*args, workspace=torch.empty(size, dtype=torch.uint8, device="cuda") if size else None, **kw)
        torch.cuda.synchronize()
        return out, st

    def ref(self, zero=False):
        """(out, tolerance, {slot: state}), token after token in 64 bits."""
        q, k, v = (x[:self.n].double().cpu() for x in (self.q, self.k, self.v))
        if self.norm:
            q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
        rep = self.hv // self.hk
        q, k = q.repeat_interleave(rep, 1) / math.sqrt(128), k.repeat_interleave(rep, 1)
        g, beta = self.g.double().cpu(), self.beta.double().cpu()
        out, tol, states, at = torch.zeros_like(v), torch.zeros_like(v), {}, 0
        for b, n in enumerate(self.lens):
            s = int(self.index[b])
            kept = 0 <= s < self.slots
            S = self.state[s].double().cpu() if kept and not zero else torch.zeros(self.hv, 128, 128, dtype=torch.float64)
            us, first = [], 0
            for t in range(at, at + n):
                i = t - at
                if i % 64 == 0:
                    us, first = [], t
                a = torch.exp(g[t])
                S = S * a[:, None, None]
                u = beta[t][:, None] * (v[t] - (S @ k[t][..., None])[..., 0])
                S = S + u[..., None] * k[t][:, None, :]
                out[t] = (S @ q[t][..., None])[..., 0]
                us.append(u.abs())
                mag = (S.abs() @ q[t].abs()[..., None])[..., 0]
                tol[t] = U * out[t].abs() + 2.0 ** -18 * mag
                if n > 24:
                    G = torch.flip(torch.cumsum(torch.flip(torch.cat([g[first + 1:t + 1], torch.zeros(1, self.hv, dtype=torch.float64)]), [0]), 0), [0])
                    P = (torch.exp(G) * (k[first:t + 1] * q[t]).sum(-1)).abs()
                    tol[t] += U * (P[..., None] * torch.stack(us)).sum(0)
            if kept:
                states[s] = S
            at += n
        return out, tol, states

    def check(self, out, st, zero=False):
        ref, tol, states = self.ref(zero)
        _near(out[:self.n], ref, tol, "out")
        assert (out[self.n:] == 7.0).all()
        for s in range(self.slots):
            if s in states:
                norm = states[s].norm()
                off = (st[s].double().cpu() - states[s]).norm()
                assert off <= 1e-5 * norm, (s, float(off / norm) if norm else float(off))
            else:
                assert (st[s] == 7.0).all(), s


@pytest.mark.parametrize("lens", [[1, 1, 1], [0, 1, 2, 24], [5]])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("heads", [(1, 1), (2, 6)])
def test_delta_recurrent(lens, norm, heads):
    d = _Delta(lens, *heads, norm=norm)
    d.check(*d.call())


@pytest.mark.parametrize("lens", [[25], [63, 64, 65], [128, 1, 129, 0, 24, 200], [700]])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("heads", [(1, 1), (2, 6), (20, 40)])  # 40: a CTA takes a whole head
def test_delta_chunked(lens, norm, heads):
    d = _Delta(lens, *heads, norm=norm)
    d.check(*d.call())


@pytest.mark.parametrize("hv", [2, 40])
@pytest.mark.parametrize("rate", [0.0, 1e-4, 3.0, 40.0])
def test_delta_decays(rate, hv):
    d = _Delta([300, 9], 1, hv, rate=rate)
    d.check(*d.call())


@pytest.mark.parametrize("hv", [2, 40])
@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_delta_write_strengths(beta, hv):
    n = 150
    d = _Delta([n], 1, hv, beta=torch.full((n, hv), beta))
    d.check(*d.call())


@pytest.mark.parametrize("hv", [2, 40])
def test_delta_decay_to_nothing(hv):
    """g = -inf forgets the state; tokens behind it are as if it were the first."""
    n = 200
    g = torch.full((n, hv), -0.05)
    for t in (0, 1, 40, 63, 64, 130):
        g[t, 0] = -math.inf
    g[100:, 1] = -1e30
    d = _Delta([n], 1, hv, g=g)
    d.check(*d.call())
    d = _Delta([7, 3], 1, hv, g=g[:10])
    d.check(*d.call())


@pytest.mark.parametrize("hv", [1, 40])
def test_delta_equal_keys(hv):
    """All keys of a chunk the same: the inverse's entries stay bounded by beta."""
    d = _Delta([130], 1, hv, rate=0.01)
    d.k.copy_(d.k[:1].expand_as(d.k).clone())
    d.check(*d.call())


@pytest.mark.parametrize("lens,hk,hv", [([70, 25, 129, 90], 4, 24), ([70, 25, 129, 90], 4, 8), ([200], 8, 32)])
def test_delta_many_heads_take_wide_parts(lens, hk, hv):
    """Sequences times heads beyond the narrow parts' range, uneven lengths, and whole heads."""
    d = _Delta(lens, hk, hv)
    out, st = d.call()
    d.check(out, st)
    # a head at a time, where there are parts the narrow ones are taken: the same bits
    o, s = d.call(ws_bytes=dsa.dsa_gated_delta_workspace_size(d.shape, d.rg)[0])
    assert torch.equal(o, out) and torch.equal(s, st)


@pytest.mark.parametrize("hv", [2, 40])
@pytest.mark.parametrize("lens", [[70, 65], [65, 3, 70]])
def test_delta_sequences_do_not_touch_one_another(lens, hv):
    """NaN and infinities in one sequence leave the others, whose last chunks end beside it, alone."""
    d = _Delta(lens, 1, hv)
    want = d.call()
    a, b = lens[0], lens[0] + lens[1]
    for x, bad in ((d.q, math.nan), (d.k, math.inf), (d.v, math.nan), (d.g, math.nan), (d.beta, math.inf)):
        x[a:b] = bad
    out, st = d.call()
    keep = torch.ones(sum(lens), dtype=torch.bool)
    keep[a:b] = False
    assert torch.equal(out[keep.cuda()], want[0][keep.cuda()])
    for i, slot in enumerate(d.index.tolist()):
        if i != 1:
            assert torch.equal(st[slot], want[1][slot])


def test_delta_scale_and_few_heads_of_many():
    """An explicit scale; sequences times heads on both sides of the narrow parts' limit."""
    for lens, hv in (([200, 90], 2), ([200, 90, 70, 100, 65], 6)):
        d = _Delta(lens, 1, hv)
        d.shape = dsa.DeltaShape(1, hv, scale=1 / math.sqrt(128))
        out, st = d.call()
        d.check(out, st)
        d.shape = dsa.DeltaShape(1, hv)
        again, st2 = d.call()
        assert torch.equal(again, out) and torch.equal(st2, st)


@pytest.mark.parametrize("hv", [4, 40])
def test_delta_no_state_no_index_and_padding(hv):
    d = _Delta([90, 1, 20], hv=hv, extra_rows=70)
    out, st = d.call(state_in=None)
    d.check(out, st, zero=True)
    d.index = torch.arange(3, dtype=torch.int32, device="cuda")
    out, st = d.call(index=None)
    d.check(out, st)


@pytest.mark.parametrize("hv", [4, 40])
def test_delta_slots_outside_are_not_kept(hv):
    d = _Delta([70, 1, 80, 2], hv=hv)
    d.index[0], d.index[1] = -1, d.slots
    d.check(*d.call())


@pytest.mark.parametrize("hv", [4, 40])
def test_delta_state_in_place(hv):
    d = _Delta([100, 3, 0, 64], hv=hv)
    out, st = d.call()
    state = d.state.clone()
    out2, _ = d.call(state_in=state, state_out=state)
    assert torch.equal(out2, out)
    for s in d.index.tolist():
        assert torch.equal(state[s], st[s])
    # without a state to keep, the outputs are the same
    only = torch.empty_like(out)
    dsa.dsa_gated_delta_prefill(d.shape, d.rg, d.q, d.k, d.v, d.g, d.beta, only, state_in=d.state, state_index=d.index,
                                workspace=torch.empty(dsa.dsa_gated_delta_workspace_size(d.shape, d.rg)[1], dtype=torch.uint8, device="cuda"))
    assert torch.equal(only, out)


def test_delta_results_do_not_depend_on_the_workspace_or_the_batch():
    d = _Delta([100, 64, 300], 2, 6)
    out, st = d.call()
    mn, rec = dsa.dsa_gated_delta_workspace_size(d.shape, d.rg)
    for size in (mn, 2 * mn + 128, 4 * mn):  # 1, 2 and 4 heads a pass
        o, s = d.call(ws_bytes=size)
        assert torch.equal(o, out) and torch.equal(s, st)
    # without the host's offsets
    rg = dsa.ragged(d.keep, d.keep, d.lens, d.lens)
    rg.q_offsets_host = None
    o, s = d.call(ragged=rg)
    assert torch.equal(o, out) and torch.equal(s, st)
    # the middle sequence alone
    a, b = 100, 164
    one = torch.empty(64, 6, 128, dtype=BF16, device="cuda")
    off = _offsets([64])
    rg1 = dsa.ragged(off, off, [64], [64])
    stx = torch.empty_like(d.state)
    dsa.dsa_gated_delta_prefill(d.shape, rg1, d.q[a:b], d.k[a:b], d.v[a:b], d.g[a:b].contiguous(), d.beta[a:b].contiguous(), one,
                                state_in=d.state, state_out=stx, state_index=d.index[1:2].contiguous(),
                                workspace=torch.empty(rec, dtype=torch.uint8, device="cuda"))
    assert torch.equal(one, out[a:b])
    assert torch.equal(stx[int(d.index[1])], st[int(d.index[1])])


@pytest.mark.parametrize("hv", [4, 40])
def test_delta_prefill_then_decode_is_the_whole_sequence(hv):
    n, steps = 150, 5
    d = _Delta([n + steps], 2, hv, slots=3)
    ref, tol, states = d.ref()
    off = _offsets([n])
    rg = dsa.ragged(off, off, [n], [n])
    state = d.state.clone()
    cut = lambda x, a, b: x[a:b].contiguous()  # noqa: E731
    outs = []
    for a, b in [(0, n)] + [(n + i, n + i + 1) for i in range(steps)]:
        out = torch.empty(b - a, hv, 128, dtype=BF16, device="cuda")
        args = [cut(x, a, b) for x in (d.q, d.k, d.v, d.g, d.beta)] + [out]
        kw = dict(state_in=state, state_out=state, state_index=d.index)
        if b - a > 1:
            dsa.dsa_gated_delta_prefill(d.shape, rg, *args, workspace=torch.empty(
                dsa.dsa_gated_delta_workspace_size(d.shape, rg)[1], dtype=torch.uint8, device="cuda"), **kw)
        else:
            o1 = _offsets([1])
            dsa.dsa_gated_delta_decode(d.shape, dsa.ragged(o1, o1, [1], [1]), *args, **kw)
        outs.append(out)
    _near(torch.cat(outs), ref, tol, "out")
    s = int(d.index[0])
    assert (state[s].double().cpu() - states[s]).norm() <= 1e-5 * states[s].norm()


@pytest.mark.parametrize("hv", [4, 40])
def test_delta_captured_replays_on_another_stream(hv):
    """A captured call replayed with new inputs, and two calls at once on two streams."""
    d, e = _Delta([130, 1, 40], 2, hv, seed=1), _Delta([130, 1, 40], 2, hv, seed=9)
    want_d, want_e = d.call(), e.call()
    size = dsa.dsa_gated_delta_workspace_size(d.shape, d.rg)[1]
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out, st = torch.full_like(want_d[0], 7.0), torch.full_like(want_d[1], 7.0)
    t = _Delta([130, 1, 40], 2, hv, seed=1)
    run = lambda: dsa.dsa_gated_delta_prefill(t.shape, t.rg, t.q, t.k, t.v, t.g, t.beta, out, state_in=t.state,  # noqa: E731
                                              state_out=st, state_index=t.index, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for src, want in ((d, want_d), (e, want_e)):
        for name in ("q", "k", "v", "g", "beta", "state", "index"):
            getattr(t, name).copy_(getattr(src, name))
        out.fill_(7.0), st.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(st, want[1])
    # two streams at once, a workspace each
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for s, x in zip(streams, (d, e)):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            w = torch.empty(size, dtype=torch.uint8, device="cuda")
            o, so = torch.full_like(out, 7.0), torch.full_like(st, 7.0)
            dsa.dsa_gated_delta_prefill(x.shape, x.rg, x.q, x.k, x.v, x.g, x.beta, o, state_in=x.state, state_out=so,
                                        state_index=x.index, workspace=w)
            got.append((o, so, w))
    torch.cuda.synchronize()
    for (o, so, _), want in zip(got, (want_d, want_e)):
        assert torch.equal(o, want[0]) and torch.equal(so, want[1])


@pytest.mark.parametrize("rows", [1, 3])
def test_delta_whole_heads_alone_and_together(rows):
    """More heads and sequences than SMs, so that CTAs follow one another: each sequence's results
    are those of a batch with fewer, and a second call's the first's."""
    lens = [130, 70, 64, 90, 33, 200][:2 * rows]
    d = _Delta(lens, 4, 96)
    out, st = d.call()
    again, st2 = d.call()
    assert torch.equal(out, again) and torch.equal(st, st2)
    few = _Delta(lens, 4, 96)  # one head's share of the heads apart: 24 of 96, the same kernel
    for h in (0, 24):
        sel = lambda x: x[:, h:h + 48].contiguous()  # noqa: E731
        hk = slice(h // 24, h // 24 + 2)
        o = torch.empty(out.shape[0], 48, 128, dtype=BF16, device="cuda")
        so = torch.full((d.slots, 48, 128, 128), 7.0, device="cuda")
        shape = dsa.DeltaShape(2, 48, qk_norm=True, norm_eps=1e-6)
        ws = torch.empty(dsa.dsa_gated_delta_workspace_size(shape, d.rg)[1], dtype=torch.uint8, device="cuda")
        dsa.dsa_gated_delta_prefill(shape, d.rg, few.q[:, hk], few.k[:, hk], sel(few.v), sel(few.g), sel(few.beta), o,
                                    state_in=sel(few.state), state_out=so, state_index=d.index, workspace=ws)
        assert torch.equal(o, out[:, h:h + 48]) and torch.equal(so, st[:, h:h + 48])


def test_delta_decode_large_slots():
    """States past 2^31 elements: the last slot of a pool of 8.6 GB."""
    hv, slots = 8, 2 ** 31 // (8 * 128 * 128) + 3
    state = torch.empty(slots, hv, 128, 128, device="cuda")
    d = _Delta([1, 1], 2, hv, slots=4)
    d.index = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    out, st = d.call(decode=True)
    state[slots - 1] = d.state[3]
    state[1] = d.state[0]
    o = torch.empty_like(out)
    dsa.dsa_gated_delta_decode(d.shape, d.rg, d.q, d.k, d.v, d.g, d.beta, o, state_in=state, state_out=state,
                               state_index=torch.tensor([slots - 1, 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(o, out)
    assert torch.equal(state[slots - 1], st[3]) and torch.equal(state[1], st[0])


def test_binding_refuses_what_the_library_cannot_see():
    d = _Delta([20])
    ws = torch.empty(dsa.dsa_gated_delta_workspace_size(d.shape, d.rg)[1], dtype=torch.uint8, device="cuda")
    out = torch.empty(20, 4, 128, dtype=BF16, device="cuda")
    good = dict(q=d.q, k=d.k, v=d.v, g=d.g, beta=d.beta, out=out, state_in=d.state, state_index=d.index, workspace=ws)
    bad = dict(q=d.q.float(), k=d.k[:, :1], v=d.v[:10], g=d.g.to(BF16), beta=d.beta.t().contiguous().t(), out=out[:, :, :64],
               state_in=d.state.half(), state_index=d.index.long(), workspace=ws.cpu())
    for name, t in bad.items():
        with pytest.raises(dsa.DsaError):
            dsa.dsa_gated_delta_prefill(d.shape, d.rg, **dict(good, **{name: t}))
    with pytest.raises(dsa.DsaError):  # rows that are not dense
        dsa.dsa_gated_delta_prefill(d.shape, d.rg, **dict(good, q=_randn(0, 20, 2, 256)[..., ::2]))


# ---------------------------------------------------------------- many sequences

def test_batches_of_thousands_of_sequences():
    """More sequences than a block-wide search reads at once, empty ones among them."""
    rng = np.random.default_rng(3)
    lens = [int(n) for n in rng.integers(0, 4, 1500)]
    lens[700], lens[1499] = 70, 26
    rope = dsa.RopeShape()
    t = _Rope(lens, [int(h) for h in rng.integers(0, 9, 1500)], heads=(2, 1, 1))
    t.call(rope)
    t.check(rope)
    n, c, w = sum(lens), 64, 4
    x, weight = _randn(1, n, c), _randn(2, c, w)
    out, st = torch.empty_like(x), torch.empty(len(lens), w - 1, c, dtype=BF16, device="cuda")
    off = _offsets(lens)
    dsa.dsa_short_conv(dsa.ConvShape(c, w), dsa.ragged(off, off, lens, lens), x, weight, out, state_out=st)
    ref, mag, states = _conv_ref(x, lens, weight, None, True, None, None, len(lens))
    _near(out, ref, U * ref.abs() + 2.0 ** -20 * 1.1 * mag, "out")
    assert torch.equal(st.double().cpu(), torch.stack([states[s] for s in range(len(lens))]))
    d = _Delta(lens, 1, 1)
    d.check(*d.call())


# ---------------------------------------------------------------- a run of them together

def test_hybrid_layer_end_to_end():
    """Projections of new tokens over a paged cache: rotary append, then the layer's selection and
    attention mixed with the linear branch (short convolution, gated delta rule), against a 64-bit
    computation fed with the intermediate tensors the library stored (each is checked by itself
    above)."""
    q_lens, hists, hq, hkv, hi, page, K = [90, 1, 40], [0, 200, 77], 8, 2, 4, 128, 48
    t = _Rope(q_lens, hists, heads=(hq, hkv, hi), page=page)
    n = t.n
    rope = dsa.RopeShape(theta=1e6)
    for i, name in enumerate(("k_cache", "v_cache", "k_idx_cache")):  # histories
        t.out[name].copy_(_randn(20 + i, *t.out[name].shape))
    t.call(rope)
    shape = dsa.LayerShape(n_idx_heads=hi, n_q_heads=hq, n_kv_heads=hkv, top_k=K)
    w = torch.tensor([0.25, 0.5, 1.0, 0.5], device="cuda")
    _, rec = dsa.dsa_index_topk_workspace_size(shape, t.rg, n)
    idx = torch.empty(n, K, dtype=torch.int32, device="cuda")
    dsa.dsa_index_topk(shape, t.rg, t.out["q_idx_out"], t.out["k_idx_cache"], w, 0, n, idx, K,
                       workspace=torch.empty(rec, dtype=torch.uint8, device="cuda"))
    # linear branch: 4 key heads, 8 value heads
    hk = 4
    c = (2 * hk + hq) * 128
    x, weight = _randn(11, n, c), _randn(12, c, 4, scale=0.5)
    mixed = torch.empty_like(x)
    dsa.dsa_short_conv(dsa.ConvShape(c, 4), t.rg, x, weight, mixed)
    d = _Delta(q_lens, hk, hq)
    d.q, d.k, d.v = (mixed[:, a * 128:b * 128].view(n, -1, 128) for a, b in ((0, hk), (hk, 2 * hk), (2 * hk, 2 * hk + hq)))
    other, st = d.call()
    d.check(other, st)
    gate = _randn(13, n, hq, 128)
    out, err = torch.empty_like(gate), torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_sparse_attn_gated_mix(shape, t.rg, t.out["q_out"], t.out["k_cache"], t.out["v_cache"], idx, K, 0, n, gate,
                                  other, out, err_count=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    k, v, q = (t.out[m].double().cpu() for m in ("k_cache", "v_cache", "q_out"))
    o, mag = torch.zeros(n, hq, 128, dtype=torch.float64), torch.zeros(n, hq, 128, dtype=torch.float64)
    at = 0
    for b, m in enumerate(q_lens):
        for i in range(m):
            sel = idx[at].long().cpu()
            sel = sel[sel >= 0]
            assert len(sel) == min(K, hists[b] + i + 1)
            rows = t.table[b].long()[sel // page] * page + sel % page
            for h in range(hq):
                p = torch.softmax(k[rows, h // (hq // hkv)] @ q[at, h] / math.sqrt(128), 0)
                o[at, h] = p @ v[rows, h // (hq // hkv)]
                mag[at, h] = p @ v[rows, h // (hq // hkv)].abs()
            at += 1
    g = torch.sigmoid(gate.double().cpu())
    ref = g * o + (1 - g) * other.double().cpu()
    # the weights enter P V rounded to bf16 (u of each), the result is rounded once; exponentials
    # and the gate's sigmoid are fp32 approximations
    _near(out, ref, U * (ref.abs() + g * mag) + 2.0 ** -14 * (mag + other.double().cpu().abs()), "mixed")
