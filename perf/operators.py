"""Cases of the operators around the sparse-attention layer: rotary positions with the append to
the caches, the short convolution, and the gated delta rule (the linear branch that the layer's
gate mixes in).  Each case is computed in plain torch operations, or (own = True) by the library."""
import math

import torch

own = False

HEAD_DIM = 128
IDX_DIM = 64
NORM_EPS = 1e-6
CHUNK = 64


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token for each of 64 sequences of 131072 cached positions: latency
        dict(name="rope_decode_b64", op="rope", batch=64, q_len=1, ragged=False, hist=131071, page=128,
             q_heads=32, kv_heads=4, idx_heads=4, layout="half", rot=128, idx_rot=64, offset=0,
             scaling="none", theta=1e6, factor=1.0, fp8=False),
        # the 32768-token prefill, q/k/v being slices of one fused projection's output
        dict(name="rope_prefill_t32768", op="rope", batch=1, q_len=32768, ragged=False, hist=0, page=0,
             q_heads=32, kv_heads=4, idx_heads=4, layout="half", rot=128, idx_rot=64, offset=0,
             scaling="none", theta=1e6, factor=1.0, fp8=False),
        # chunks of a serving batch far into long contexts: half of each head turns, in adjacent pairs,
        # frequencies scaled by parts, indexer rows kept in e4m3
        dict(name="rope_ragged_parts_fp8", op="rope", batch=9, q_len=2500, ragged=True, hist=262144, page=256,
             q_heads=64, kv_heads=8, idx_heads=4, layout="interleaved", rot=64, idx_rot=32, offset=64,
             scaling="by_parts", theta=1e4, factor=8.0, fp8=True),
        # one token for each of 256 sequences
        dict(name="conv_decode_b256", op="conv", batch=256, q_len=1, ragged=False, channels=8192, width=4,
             silu=True, bias=False, strided=False),
        # q, k and v channels of 16 + 16 + 32 heads over the long prefill
        dict(name="conv_prefill_t32768", op="conv", batch=1, q_len=32768, ragged=False, channels=8192, width=4,
             silu=True, bias=False, strided=False),
        # uneven chunks, some empty, a channel count that is no power of two, input rows inside wider ones
        dict(name="conv_ragged_w3", op="conv", batch=17, q_len=1500, ragged=True, channels=5128, width=3,
             silu=False, bias=True, strided=True),
        # one token for each of 64 sequences, 32 heads sharing 16 key heads
        dict(name="delta_decode_b64", op="delta", batch=64, q_len=1, ragged=False, tail=0, k_heads=16, v_heads=32,
             norm=True, state=True),
        # a full decode batch, 64 heads
        dict(name="delta_decode_b256", op="delta", batch=256, q_len=1, ragged=False, tail=0, k_heads=16,
             v_heads=64, norm=True, state=True),
        # a short prompt of one request
        dict(name="delta_prefill_t4096", op="delta", batch=1, q_len=4096, ragged=False, tail=0, k_heads=8,
             v_heads=8, norm=True, state=False),
        # the 32768-token prefill
        dict(name="delta_prefill_t32768", op="delta", batch=1, q_len=32768, ragged=False, tail=0, k_heads=32,
             v_heads=32, norm=True, state=False),
        # a serving batch: 8 chunks of up to 8192 tokens and 64 single tokens, all with states
        dict(name="delta_serving", op="delta", batch=8, q_len=8192, ragged=True, tail=64, k_heads=16, v_heads=64,
             norm=True, state=True),
        # few tokens for each of many sequences, keys that are unit vectors already
        dict(name="delta_short_q5", op="delta", batch=48, q_len=5, ragged=True, tail=0, k_heads=4, v_heads=12,
             norm=False, state=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "conv", "delta", "delta"])
    if op == "rope":
        batch = _log_int(rng, 1, 64)
        kv = rng.choice([1, 2, 4, 8])
        rot = 16 * rng.randint(1, 8)
        scaling = rng.choice(["none", "linear", "ntk", "by_parts"])
        return dict(op="rope", batch=batch, q_len=_log_int(rng, 1, max(1, 32768 // batch)), ragged=rng.random() < 0.6,
                    hist=_log_int(rng, 1, 1000000), page=rng.choice([128, 256, 1024]),
                    q_heads=kv * rng.randint(1, 8), kv_heads=kv, idx_heads=rng.randint(1, 4),
                    layout=rng.choice(["half", "interleaved"]), rot=rot, idx_rot=16 * rng.randint(1, 4),
                    offset=rng.choice([0, 128 - rot]), scaling=scaling, theta=rng.choice([1e4, 5e5, 1e6]),
                    factor=1.0 if scaling == "none" else rng.uniform(1.5, 40.0), fp8=rng.random() < 0.3)
    if op == "conv":
        batch = _log_int(rng, 1, 256)
        return dict(op="conv", batch=batch, q_len=_log_int(rng, 1, max(1, 32768 // batch)), ragged=rng.random() < 0.6,
                    channels=8 * _log_int(rng, 16, 1024), width=rng.randint(2, 4), silu=rng.random() < 0.7,
                    bias=rng.random() < 0.5, strided=rng.random() < 0.5)
    k_heads = rng.choice([1, 2, 3, 4, 8, 16])
    v_heads = k_heads * rng.randint(1, 4)
    if rng.random() < 0.4:
        batch, q_len, tail = _log_int(rng, 1, 256), rng.choice([1, 1, 2, 7]), 0
    else:
        batch = _log_int(rng, 1, 12)
        tail = rng.choice([0, 0, rng.randint(1, 40)])
        q_len = _log_int(rng, 20, max(21, 300000 // (batch * v_heads)))
    return dict(op="delta", batch=batch, q_len=q_len, ragged=rng.random() < 0.6, tail=tail, k_heads=k_heads,
                v_heads=v_heads, norm=rng.random() < 0.7, state=rng.random() < 0.6)


# ---------------------------------------------------------------- inputs

def _lens(case, seed):
    """Query rows of each sequence: q_len, or uneven ones up to it (an empty one among four or more)."""
    n, top = case["batch"], case["q_len"]
    if not case["ragged"]:
        got = [top] * n
    else:
        got = [max(1, top * (3 + (i * 7 + 5) % 13) // 15) for i in range(n)]
        got[(n - 1) // 2] = top
        if n >= 4 and top > 1:
            got[1] = 0
    return got + [1] * case.get("tail", 0)


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(torch.bfloat16)


def _gen(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return gen


def _rope_inputs(case, seed):
    gen = _gen(seed)
    lens = _lens(case, seed)
    hists = [case["hist"] * (b + 1) // len(lens) for b in range(len(lens))]
    kv_lens = [h + n for h, n in zip(hists, lens)]
    total = sum(lens)
    hq, hkv, hi = case["q_heads"], case["kv_heads"], case["idx_heads"]
    fused = _normal(gen, total, (hq + 2 * hkv) * HEAD_DIM)
    fused_idx = _normal(gen, total, 2 * hi * IDX_DIM)
    s = dict(case=case, q_lens=lens, kv_lens=kv_lens, q_offsets=_offsets(lens), kv_offsets=_offsets(kv_lens),
             q=fused[:, :hq * HEAD_DIM].view(total, hq, HEAD_DIM),
             k=fused[:, hq * HEAD_DIM:(hq + hkv) * HEAD_DIM].view(total, hkv, HEAD_DIM),
             v=fused[:, (hq + hkv) * HEAD_DIM:].view(total, hkv, HEAD_DIM),
             q_idx=fused_idx[:, :hi * IDX_DIM].view(total, hi, IDX_DIM),
             k_idx=fused_idx[:, hi * IDX_DIM:].view(total, hi, IDX_DIM))
    page = case["page"]
    if page:
        # a page is its sequence's own where new rows go; earlier pages, which the append does not touch,
        # all stand on page 0
        first = [h // page for h in hists]
        count = [(n + page - 1) // page - f if n > h else 0 for h, n, f in zip(hists, kv_lens, first)]
        n_pages = 1 + sum(count)
        order = (torch.randperm(n_pages - 1, device="cuda", generator=gen) + 1).tolist()
        width = max((n + page - 1) // page for n in kv_lens)
        table = torch.zeros(len(lens), width, dtype=torch.int32)
        at = 0
        for b, (f, c) in enumerate(zip(first, count)):
            table[b, f:f + c] = torch.tensor(order[at:at + c], dtype=torch.int32)
            at += c
        s["block_table"] = table.cuda()
        rows = n_pages * page
    else:
        rows = sum(kv_lens)
    idx_type = torch.float8_e4m3fn if case["fp8"] else torch.bfloat16
    s["cache_rows"] = rows
    s["k_cache"] = torch.zeros(rows, hkv, HEAD_DIM, dtype=torch.bfloat16, device="cuda")
    s["v_cache"] = torch.zeros(rows, hkv, HEAD_DIM, dtype=torch.bfloat16, device="cuda")
    s["k_idx_cache"] = torch.zeros(rows, hi, IDX_DIM, device="cuda").to(idx_type)
    s["q_out"] = torch.empty(total, hq, HEAD_DIM, dtype=torch.bfloat16, device="cuda")
    s["q_idx_out"] = torch.empty(total, hi, IDX_DIM, dtype=idx_type, device="cuda")
    return s


def _conv_inputs(case, seed):
    gen = _gen(seed)
    lens = _lens(case, seed)
    total, c, w = sum(lens), case["channels"], case["width"]
    wide = c + (64 if case["strided"] else 0)
    slots = len(lens) + 3
    return dict(case=case, q_lens=lens, q_offsets=_offsets(lens), x=_normal(gen, total, wide)[:, :c],
                weight=_normal(gen, c, w, scale=0.5), bias=_normal(gen, c, scale=0.1) if case["bias"] else None,
                state_in=_normal(gen, slots, w - 1, c), state_out=torch.zeros(slots, w - 1, c, dtype=torch.bfloat16, device="cuda"),
                state_index=torch.randperm(slots, device="cuda", generator=gen)[:len(lens)].to(torch.int32),
                out=torch.empty(total, c, dtype=torch.bfloat16, device="cuda"))


def _delta_inputs(case, seed):
    gen = _gen(seed)
    lens = _lens(case, seed)
    total, hk, hv, d = sum(lens), case["k_heads"], case["v_heads"], HEAD_DIM
    fused = _normal(gen, total, (2 * hk + hv) * d)  # what a short convolution over q, k and v leaves
    q = fused[:, :hk * d].view(total, hk, d)
    k = fused[:, hk * d:2 * hk * d].view(total, hk, d)
    v = fused[:, 2 * hk * d:].view(total, hv, d)
    if not case["norm"]:
        k.copy_(k.float() / k.float().norm(dim=-1, keepdim=True))
        q.copy_(q.float() / q.float().norm(dim=-1, keepdim=True))
    # decays from nearly none to a few e-folds a token, one rate to a head
    rate = torch.exp(torch.rand(hv, device="cuda", generator=gen) * 5 - 4)
    g = -rate * torch.nn.functional.softplus(torch.randn(total, hv, device="cuda", generator=gen))
    beta = torch.sigmoid(torch.randn(total, hv, device="cuda", generator=gen))
    slots = len(lens) + 2
    s = dict(case=case, q_lens=lens, q_offsets=_offsets(lens), q=q, k=k, v=v, g=g, beta=beta, state_in=None,
             state_out=torch.zeros(slots, hv, d, d, device="cuda"),
             state_index=torch.randperm(slots, device="cuda", generator=gen)[:len(lens)].to(torch.int32),
             out=torch.empty(total, hv, d, dtype=torch.bfloat16, device="cuda"))
    if case["state"]:
        s["state_in"] = torch.randn(slots, hv, d, d, device="cuda", generator=gen) * 0.3
    return s


def prepare(case, seed):
    return {"rope": _rope_inputs, "conv": _conv_inputs, "delta": _delta_inputs}[case["op"]](case, seed)


# ---------------------------------------------------------------- the framework's calls

def _handle(s):
    """The descriptors that a serving program keeps for a batch: its ragged layout and the operator's shape."""
    import indexer_top_gated_b200 as dsa
    if "handle" not in s:
        c = s["case"]
        if c["op"] == "rope":
            rg = dsa.ragged(s["q_offsets"], s["kv_offsets"], s["q_lens"], s["kv_lens"],
                            block_table=s.get("block_table"), page_size=c["page"], cache_rows=s["cache_rows"])
            shape = dsa.LayerShape(n_idx_heads=c["idx_heads"], idx_dim=IDX_DIM, n_q_heads=c["q_heads"],
                                   n_kv_heads=c["kv_heads"], head_dim=HEAD_DIM,
                                   idx_dtype=dsa.DSA_FP8_E4M3 if c["fp8"] else dsa.DSA_BF16)
            rope = dsa.RopeShape(layout=dict(half=dsa.DSA_ROPE_HALF, interleaved=dsa.DSA_ROPE_INTERLEAVED)[c["layout"]],
                                 rot_dim=c["rot"], idx_rot_dim=c["idx_rot"], rot_offset=c["offset"],
                                 scaling=dict(none=dsa.DSA_ROPE_SCALE_NONE, linear=dsa.DSA_ROPE_SCALE_LINEAR,
                                              ntk=dsa.DSA_ROPE_SCALE_NTK, by_parts=dsa.DSA_ROPE_SCALE_BY_PARTS)[c["scaling"]],
                                 theta=c["theta"], factor=c["factor"], orig_len=4096.0)
            s["handle"] = (dsa, shape, rg, rope)
        elif c["op"] == "conv":
            rg = dsa.ragged(s["q_offsets"], s["q_offsets"], s["q_lens"], s["q_lens"])
            s["handle"] = (dsa, dsa.ConvShape(c["channels"], c["width"], silu=c["silu"]), rg)
        else:
            rg = dsa.ragged(s["q_offsets"], s["q_offsets"], s["q_lens"], s["q_lens"])
            shape = dsa.DeltaShape(c["k_heads"], c["v_heads"], HEAD_DIM, qk_norm=c["norm"], norm_eps=NORM_EPS)
            ws = None
            if max(s["q_lens"]) > 1:
                _, size = dsa.dsa_gated_delta_workspace_size(shape, rg)
                ws = torch.empty(size, dtype=torch.uint8, device="cuda")
            s["handle"] = (dsa, shape, rg, ws)
    return s["handle"]


def _own(s):
    c = s["case"]
    if c["op"] == "rope":
        dsa, shape, rg, rope = _handle(s)
        dsa.dsa_rope_append(shape, rg, rope, q=s["q"], k=s["k"], v=s["v"], q_idx=s["q_idx"], k_idx=s["k_idx"],
                            q_out=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                            q_idx_out=s["q_idx_out"], k_idx_cache=s["k_idx_cache"])
        return {n: s[n] for n in ("q_out", "k_cache", "v_cache", "q_idx_out", "k_idx_cache")}
    if c["op"] == "conv":
        dsa, shape, rg = _handle(s)
        dsa.dsa_short_conv(shape, rg, s["x"], s["weight"], s["out"], bias=s["bias"], state_in=s["state_in"],
                           state_out=s["state_out"], state_index=s["state_index"])
    else:
        dsa, shape, rg, ws = _handle(s)
        if ws is None:
            dsa.dsa_gated_delta_decode(shape, rg, s["q"], s["k"], s["v"], s["g"], s["beta"], s["out"],
                                       state_in=s["state_in"], state_out=s["state_out"], state_index=s["state_index"])
        else:
            dsa.dsa_gated_delta_prefill(shape, rg, s["q"], s["k"], s["v"], s["g"], s["beta"], s["out"],
                                        state_in=s["state_in"], state_out=s["state_out"],
                                        state_index=s["state_index"], workspace=ws)
    return {"out": s["out"], "state": s["state_out"]}


# ---------------------------------------------------------------- plain forms

def _rows(s):
    """Sequence and place in it of each query row."""
    lens = torch.tensor(s["q_lens"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(s["q_lens"]), device="cuda"), lens)
    return seq, torch.arange(int(s["q_offsets"].numel() and sum(s["q_lens"])), device="cuda") - s["q_offsets"].long()[seq]


def _freqs(c, dim):
    """Angle per position of each pair, in 64 bits."""
    i = torch.arange(dim // 2, dtype=torch.float64, device="cuda")
    theta = c["theta"]
    if c["scaling"] == "ntk" and dim > 2:
        theta = theta * c["factor"] ** (dim / (dim - 2))
    f = theta ** (-2 * i / dim)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "by_parts":
        turns = 4096.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * (keep + (1 - keep) / c["factor"])
    return f


def _turned(x, p, c, dim, offset):
    """x with dims offset .. offset+dim-1 of each head turned by the position's angles, in 32 bits."""
    a = p.double()[:, None] * _freqs(c, dim)
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    y = x.float().clone()
    part = y[..., offset:offset + dim]
    if c["layout"] == "half":
        u, w = part[..., :dim // 2].clone(), part[..., dim // 2:].clone()
        part[..., :dim // 2] = u * cos - w * sin
        part[..., dim // 2:] = u * sin + w * cos
    else:
        u, w = part[..., 0::2].clone(), part[..., 1::2].clone()
        part[..., 0::2] = u * cos - w * sin
        part[..., 1::2] = u * sin + w * cos
    return y


def _to_idx(x, fp8):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else x.to(torch.bfloat16)


def _plain_rope(s):
    c = s["case"]
    seq, place = _rows(s)
    q_off, kv_off = s["q_offsets"].long(), s["kv_offsets"].long()
    p = (kv_off[1:] - kv_off[:-1] - (q_off[1:] - q_off[:-1]))[seq] + place
    if c["page"]:
        row = s["block_table"].long()[seq, p // c["page"]] * c["page"] + p % c["page"]
    else:
        row = kv_off[seq] + p
    s["k_cache"][row] = _turned(s["k"], p, c, c["rot"], c["offset"]).to(torch.bfloat16)
    s["v_cache"][row] = s["v"]
    k_idx = _to_idx(_turned(s["k_idx"], p, c, c["idx_rot"], 0), c["fp8"])
    if c["fp8"]:
        s["k_idx_cache"].view(torch.uint8)[row] = k_idx.view(torch.uint8)
    else:
        s["k_idx_cache"][row] = k_idx
    return dict(q_out=_turned(s["q"], p, c, c["rot"], c["offset"]).to(torch.bfloat16), k_cache=s["k_cache"],
                v_cache=s["v_cache"], q_idx_out=_to_idx(_turned(s["q_idx"], p, c, c["idx_rot"], 0), c["fp8"]),
                k_idx_cache=s["k_idx_cache"])


def _plain_conv(s):
    c = s["case"]
    w = c["width"]
    seq, place = _rows(s)
    x, old = s["x"].float(), s["state_in"].float()[s["state_index"].long()]
    at = torch.arange(len(x), device="cuda")
    y = torch.zeros_like(x) if s["bias"] is None else s["bias"].float().expand_as(x).clone()
    for j in range(w):  # tap j reads the row w-1-j back, from the state before the sequence's first row
        back = w - 1 - j
        past = (place < back)[:, None]
        row = torch.where(past, old[seq, (place - back + w - 1).clamp(0, w - 2)], x[(at - back).clamp(min=0)])
        y += s["weight"].float()[:, j] * row
    if c["silu"]:
        y = y / (1 + torch.exp(-y))
    n = torch.tensor(s["q_lens"], device="cuda")[:, None]
    want = n - (w - 1) + torch.arange(w - 1, device="cuda")  # places of the rows that the new state holds
    first = s["q_offsets"].long()[:-1, None]
    from_x = s["x"][(first + want).clamp(0, max(0, len(x) - 1))]
    from_old = s["state_in"][s["state_index"].long()[:, None], (want + w - 1).clamp(0, w - 2)]
    s["state_out"][s["state_index"].long()] = torch.where((want < 0)[..., None], from_old, from_x)
    return {"out": y.to(torch.bfloat16), "state": s["state_out"]}


def _plain_delta_steps(s, q, k, v, state, out):
    """Token after token, for the few tokens of decode."""
    lens = torch.tensor(s["q_lens"], device="cuda")
    first = s["q_offsets"].long()[:-1]
    for t in range(max(s["q_lens"])):
        b = torch.nonzero(lens > t)[:, 0] if len(set(s["q_lens"])) > 1 else slice(None)
        r = (first + t)[b]
        S = state[b] * torch.exp(s["g"][r])[..., None, None]
        u = s["beta"][r][..., None] * (v[r] - (S * k[r][..., None, :]).sum(-1))
        S = S + u[..., None] * k[r][..., None, :]
        out[r] = (S * q[r][..., None, :]).sum(-1)
        state[b] = S
    return out, state


def _plain_delta_chunks(s, q, k, v, state, out):
    """Chunks of 64 tokens: what a chunk's tokens do to one another at once, the state from chunk to chunk."""
    lens, C = s["q_lens"], CHUNK
    counts = [(n + C - 1) // C for n in lens]
    first, begin = [], 0
    for n in counts:
        first.append(begin)
        begin += n
    nc = begin
    offs = s["q_offsets"].tolist()
    start = torch.tensor([offs[b] + C * i for b, n in enumerate(counts) for i in range(n)], device="cuda")
    stop = torch.tensor([offs[b + 1] for b, n in enumerate(counts) for i in range(n)], device="cuda")
    row = start[:, None] + torch.arange(C, device="cuda")
    real = row < stop[:, None]
    row = row.clamp(max=len(q) - 1)

    def chunks(x):  # [rows, heads, ...] -> [chunks, heads, 64, ...], zeros behind a sequence's end
        y = x[row].transpose(1, 2)
        return y * real[:, None, :].reshape(nc, 1, C, *([1] * (y.dim() - 3))).to(y.dtype)

    Q, K, V, beta = chunks(q), chunks(k), chunks(v), chunks(s["beta"])
    G = torch.cumsum(chunks(s["g"]).double(), -1)
    tri = torch.tril(torch.ones(C, C, dtype=torch.bool, device="cuda"))
    D = torch.where(tri, torch.exp(torch.where(tri, G[..., :, None] - G[..., None, :], 0.0)), 0.0).float()
    A = torch.tril(beta[..., None] * D * (K @ K.transpose(-1, -2)), -1)
    T = torch.eye(C, device="cuda").expand_as(A).clone()
    for i in range(1, C):  # row i of (I + A)^-1 from the rows above it
        T[..., i, :i] = -(A[..., i:i + 1, :i] @ T[..., :i, :i])[..., 0, :]
    P = D * (Q @ K.transpose(-1, -2))
    del A, D
    eg = torch.exp(G).float()[..., None]
    tail = torch.exp(G[..., -1:] - G).float()[..., None]
    for i in range(max(counts)):
        b = [j for j, n in enumerate(counts) if n > i]
        c = torch.tensor([first[j] + i for j in b], device="cuda")
        S = state[b] if len(b) < len(counts) else state
        St = S.transpose(-1, -2)
        U = T[c] @ (beta[c][..., None] * (V[c] - eg[c] * (K[c] @ St)))
        O = (eg[c] * (Q[c] @ St) + P[c] @ U).transpose(1, 2)
        keep = real[c]
        out[row[c][keep]] = O[keep]
        S = eg[c][..., -1:, :] * S + U.transpose(-1, -2) @ (tail[c] * K[c])
        if len(b) < len(counts):
            state[b] = S
        else:
            state = S
    return out, state


def _plain_delta(s):
    c = s["case"]
    group = c["v_heads"] // c["k_heads"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if c["norm"]:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + NORM_EPS)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + NORM_EPS)
    q = (q / math.sqrt(HEAD_DIM)).repeat_interleave(group, 1)
    k = k.repeat_interleave(group, 1)
    slot = s["state_index"].long()
    if s["state_in"] is None:
        state = torch.zeros(len(s["q_lens"]), c["v_heads"], HEAD_DIM, HEAD_DIM, device="cuda")
    else:
        state = s["state_in"][slot]
    form = _plain_delta_steps if max(s["q_lens"]) <= 16 else _plain_delta_chunks
    out, state = form(s, q, k, v, state, torch.zeros_like(v))
    s["state_out"][slot] = state
    return {"out": out.to(torch.bfloat16), "state": s["state_out"]}


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "conv": _plain_conv, "delta": _plain_delta}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_rope(s):
    """Pairs as complex numbers times exp(i p f), row by row of each sequence."""
    c = s["case"]
    fine = dict(q_out=s["q"].double().clone(), q_idx_out=s["q_idx"].double().clone())
    k, k_idx = s["k"].double().clone(), s["k_idx"].double().clone()
    k_cache, v_cache, k_idx_cache = (s[n].double() for n in ("k_cache", "v_cache", "k_idx_cache"))

    def turn(x, p, r, off):
        j = torch.arange(r // 2, dtype=torch.float64, device="cuda")
        base = c["theta"]
        if c["scaling"] == "ntk" and r > 2:
            base *= c["factor"] ** (r / (r - 2))
        f = torch.exp(-math.log(base) * 2 * j / r)
        if c["scaling"] == "linear":
            f /= c["factor"]
        elif c["scaling"] == "by_parts":
            y = ((4096.0 / (2 * math.pi / f) - 1.0) / 31.0).clamp(0, 1)
            f = (1 - y) * f / c["factor"] + y * f
        z = torch.polar(torch.ones_like(p[:, None] * f), p[:, None] * f)[:, None]
        h = x[..., off:off + r]
        a, b = (slice(0, r // 2), slice(r // 2, r)) if c["layout"] == "half" else (slice(0, r, 2), slice(1, r, 2))
        z = torch.complex(h[..., a].contiguous(), h[..., b].contiguous()) * z
        h[..., a], h[..., b] = z.real, z.imag

    at = 0
    for b, n in enumerate(s["q_lens"]):
        if not n:
            continue
        p = torch.arange(s["kv_lens"][b] - n, s["kv_lens"][b], device="cuda")
        rows = slice(at, at + n)
        for x, r, off in ((fine["q_out"], c["rot"], c["offset"]), (k, c["rot"], c["offset"]),
                          (fine["q_idx_out"], c["idx_rot"], 0), (k_idx, c["idx_rot"], 0)):
            turn(x[rows], p.double(), r, off)
        if c["page"]:
            to = s["block_table"][b].long()[torch.div(p, c["page"], rounding_mode="floor")] * c["page"] + p % c["page"]
        else:
            to = int(s["kv_offsets"][b]) + p
        k_cache[to], v_cache[to], k_idx_cache[to] = k[rows], s["v"][rows].double(), k_idx[rows]
        at += n
    return dict(q_out=fine["q_out"], k_cache=k_cache, v_cache=v_cache, q_idx_out=fine["q_idx_out"], k_idx_cache=k_idx_cache)


def _exact_conv(s):
    """Each sequence with its history in front, as one sum over windows."""
    c = s["case"]
    w = c["width"]
    out, state, at = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda"), s["state_out"].double(), 0
    for b, n in enumerate(s["q_lens"]):
        slot = int(s["state_index"][b])
        rows = torch.cat([s["state_in"][slot].double(), s["x"][at:at + n].double()])
        if n:
            y = (rows.unfold(0, w, 1) * s["weight"].double()).sum(-1)
            y = y + s["bias"].double() if s["bias"] is not None else y
            out[at:at + n] = y * torch.sigmoid(y) if c["silu"] else y
        state[slot] = rows[n:]
        at += n
    return {"out": out, "state": state}


def _exact_delta(s):
    """The recurrence itself, token after token."""
    c = s["case"]
    group = c["v_heads"] // c["k_heads"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if c["norm"]:
        q, k = (x * (x.square().sum(-1, keepdim=True) + NORM_EPS).rsqrt() for x in (q, k))
    q, k = (q * HEAD_DIM ** -0.5).repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    decay, beta = torch.exp(s["g"].double()), s["beta"].double()
    out = torch.zeros_like(v)
    order = sorted(range(len(s["q_lens"])), key=lambda b: -s["q_lens"][b])
    slots = s["state_index"].long()[order]
    S = s["state_in"].double()[slots] if s["state_in"] is not None else torch.zeros(
        len(order), c["v_heads"], HEAD_DIM, HEAD_DIM, dtype=torch.float64, device="cuda")
    first = s["q_offsets"].long()[:-1][order]
    lens = [s["q_lens"][b] for b in order]
    live = len(order)
    for t in range(lens[0]):
        while lens[live - 1] <= t:
            live -= 1
        r = first[:live] + t
        kt = k[r]
        now = S[:live]
        now *= decay[r][..., None, None]
        u = beta[r][..., None] * (v[r] - torch.matmul(now, kt[..., None])[..., 0])
        now += u[..., None] * kt[..., None, :]
        out[r] = torch.matmul(now, q[r][..., None])[..., 0]
    state = s["state_out"].double()
    state[slots] = S
    return {"out": out, "state": state}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "conv": _exact_conv, "delta": _exact_delta}[case["op"]](s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    lens = _lens(c, 0)
    n = sum(lens)
    if c["op"] == "rope":
        idx = n * 2 * c["idx_heads"] * IDX_DIM
        att = n * (c["q_heads"] + 2 * c["kv_heads"]) * HEAD_DIM
        turned = n * ((c["q_heads"] + c["kv_heads"]) * c["rot"] + 2 * c["idx_heads"] * c["idx_rot"])
        return {"bytes": att * 4 + idx * (3 if c["fp8"] else 4), "flops": 3 * turned}
    if c["op"] == "conv":
        ch, w = c["channels"], c["width"]
        return {"bytes": 4 * n * ch + 2 * ch * w + 4 * len(lens) * (w - 1) * ch + (2 * ch if c["bias"] else 0),
                "flops": 2 * n * ch * w}
    d, hk, hv = HEAD_DIM, c["k_heads"], c["v_heads"]
    states = len(lens) * hv * d * d * 4 * (2 if c["state"] else 1)
    # the recurrence: two products of the state with a vector and one outer product a token
    return {"bytes": n * (2 * hk + 2 * hv) * d * 2 + n * hv * 8 + states, "flops": n * hv * 6 * d * d}
