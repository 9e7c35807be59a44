"""What is measured of the linear-attention block's operators: linear attention with a decay for each
head (whole sequences, with its backward pass, and single tokens) and the layer norm (with its backward
pass).

Every operator is here twice: in its plain form (elementary torch operations in 32 bits, rounded
once at the end; ``own`` false) and as the framework's calls (``own`` true).

Linear attention, per sequence and head (q and k of the head's group; g its log decay, one for each head
or one for each token and head):
    S_t = exp(g_t) S_{t-1} + k_t^T v_t  (dk x dv), from h0;  y_t = scale q_t S_t
Layer norm, per row (residual optional):
    s = x + residual,  n = (s - mean s) / sqrt(mean (s - mean s)^2 + eps) weight + bias
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5
CHUNK = 64    # tokens of a chunk of the plain form
DEV = "cuda:0"

# ------------------------------------------------------------------------------------------
# Cases


def listed():
    return [
        # one token of one stream: the smallest call of a serving loop
        dict(name="step_b1_h12_64x64_bf16", op="step", batch=1, heads=12, groups=12, dk=64, dv=64, io="bf16", decay="head",
             slots=False),
        # one token of every stream of a serving batch, states in a pool of slots: the states' traffic
        dict(name="step_b256_h24_64x64_bf16", op="step", batch=256, heads=24, groups=24, dk=64, dv=64, io="bf16",
             decay="token", slots=True),
        # two 8x8-patch images at a toy width: a small call over whole sequences
        dict(name="attn_2x65_h2_16x16_f32", op="attn", nseq=2, length=65, heads=2, groups=2, dk=16, dv=16, io="f32",
             decay="head", packed=False, reverse=False, fused=False, state=False, train=False),
        # 512x512 images (1025 tokens), inference with states carried in and out, the inputs being slices of
        # one projection's output, a decay for each token
        dict(name="attn_8x1025_h12_64x64_bf16", op="attn", nseq=8, length=1025, heads=12, groups=12, dk=64, dv=64,
             io="bf16", decay="token", packed=False, reverse=False, fused=True, state=True, train=False),
        # one long prompt, fixed decays: the long axis
        dict(name="attn_1x65537_h24_64x64_bf16", op="attn", nseq=1, length=65537, heads=24, groups=24, dk=64, dv=64,
             io="bf16", decay="head", packed=False, reverse=False, fused=False, state=False, train=False),
        # packed prompts of different lengths (0 to 1025 tokens), q and k shared by all heads (the causal
        # state-space dual form), wide states
        dict(name="attn_packed64_1025_h24g1_128x64_bf16", op="attn", nseq=64, length=1025, heads=24, groups=1, dk=128,
             dv=64, io="bf16", decay="token", packed=True, reverse=False, fused=False, state=True, train=False),
        # a training step's forward and backward at the Vim-S shape
        dict(name="attn_train_128x197_h12_64x64_bf16", op="attn", nseq=128, length=197, heads=12, groups=12, dk=64,
             dv=64, io="bf16", decay="token", packed=False, reverse=False, fused=False, state=False, train=True),
        # packed sequences walked from their ends in training, odd head sizes, pairs of heads that share q and k, fp32
        dict(name="attn_train_packed32_513_h6g3_40x56_f32", op="attn", nseq=32, length=513, heads=6, groups=3, dk=40,
             dv=56, io="f32", decay="token", packed=True, reverse=True, fused=False, state=True, train=True),
        # one token's norm
        dict(name="ln_1x768_bf16", op="ln", rows=1, d=768, io="bf16", res="f32", affine=True, train=False),
        # residual add and norm between two blocks at the Vim-S shape
        dict(name="ln_25216x768_bf16", op="ln", rows=25216, d=768, io="bf16", res="f32", affine=True, train=False),
        # the same in training, forward and backward
        dict(name="ln_train_25216x768_bf16", op="ln", rows=25216, d=768, io="bf16", res="f32", affine=True, train=True),
        # a norm alone in training, an odd width (no wide loads), fp32
        dict(name="ln_train_13056x1531_f32", op="ln", rows=13056, d=1531, io="f32", res="none", affine=True, train=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _head_dim(rng):
    """Two thirds common sizes, the rest anything."""
    return rng.choice([16, 32, 64, 64, 128, 128]) if rng.random() < 0.67 else rng.randint(4, 128)


def draw(rng):
    op = rng.choice(["step", "attn", "attn", "attn", "ln", "ln"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "ln":
        train = rng.random() < 0.5
        d = _log_int(rng, 16, 8192)
        q = rng.choice([64, 32, 1])
        d = max(q, d // q * q)
        rows = _log_int(rng, 1, min(100000, 15000000 // d))
        return dict(op=op, rows=rows, d=d, io=io, res=rng.choice(["f32", "io", "none"]), affine=rng.random() < 0.8,
                    train=train)
    dk, dv = _head_dim(rng), _head_dim(rng)
    heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 32])
    groups = rng.choice([g for g in (1, heads, heads, heads // 2 or 1) if heads % g == 0])
    decay = rng.choice(["head", "token"])
    if op == "step":
        batch = _log_int(rng, 1, max(1, min(512, 25000000 // (heads * dk * dv))))
        return dict(op=op, batch=batch, heads=heads, groups=groups, dk=dk, dv=dv, io=io, decay=decay,
                    slots=rng.random() < 0.5)
    train = rng.random() < 0.5
    rows = (30000000 if train else 100000000) // (heads * (dk + dv)) // (1 if io == "bf16" else 2)    # tokens
    length = _log_int(rng, 1, min(8192 if train else 65537, rows))
    nseq = _log_int(rng, 1, max(1, min(256, rows // length, 20000000 // (heads * dk * dv))))
    return dict(op=op, nseq=nseq, length=length, heads=heads, groups=groups, dk=dk, dv=dv, io=io, decay=decay,
                packed=nseq > 1 and rng.random() < 0.4, reverse=rng.random() < 0.4, fused=rng.random() < 0.3,
                state=rng.random() < 0.5, train=train)


def _lengths(case):
    """Sequence lengths: equal, or spread over 0..length with an empty sequence and a single token among them."""
    n, length = case["nseq"], case["length"]
    if not case["packed"]:
        return [length] * n
    out = [1 + (7919 * k * k + 104729 * k + 31) % length for k in range(n)]
    out[0] = length
    out[n // 2] = 0
    if n > 2:
        out[n - 1] = 1
    return out


def _io(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


# ------------------------------------------------------------------------------------------
# Inputs


def _log_decays(case, gen, *lead):
    """One for each head: horizons of 32 to some thousand tokens. One for each token and head: -rate softplus(.)."""
    heads = case["heads"]
    if case["decay"] == "head":
        return torch.log1p(-torch.exp2(-5 - 7 * torch.arange(heads, device=DEV, dtype=torch.float32) / heads))
    rate = torch.rand(heads, generator=gen, device=DEV) * 1.5 + 0.1
    return -rate * torch.nn.functional.softplus(torch.randn((*lead, heads), generator=gen, device=DEV) - 2)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = _io(case)

    def normal(*shape, std=1.0, dtype=dt, mean=0.0):
        return (torch.randn(shape, generator=gen, device=DEV) * std + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "ln":
        n, d = case["rows"], case["d"]
        rdt = {"f32": torch.float32, "io": dt, "none": None}[case["res"]]
        s["x"] = normal(n, d, mean=0.2)
        s["residual"] = normal(n, d, std=3.0, mean=-0.5, dtype=rdt) if rdt else None
        s["weight"] = normal(d, std=0.1, mean=1.0, dtype=torch.float32) if case["affine"] else None
        s["bias"] = normal(d, std=0.1, dtype=torch.float32) if case["affine"] else None
        if case["train"]:
            s["dn"] = normal(n, d)
            s["dsum"] = normal(n, d, dtype=rdt) if rdt else None
        if own:
            from bidirectional_selective_scan_amd import binding
            args = (s["x"], s["residual"], s["weight"], s["bias"])
            s["call"] = binding.PreparedLayerNorm(*args, eps=EPS, with_sum=rdt is not None)
            if case["train"]:
                s["grad"] = binding.PreparedLayerNormGrad(*args, dsum=s["dsum"], dn=s["dn"], eps=EPS)
        return s
    heads, groups, dk, dv = (case[k] for k in ("heads", "groups", "dk", "dv"))
    s["scale"] = dk ** -0.5
    if case["op"] == "step":
        n = case["batch"]
        s.update(q=normal(n, groups, dk), k=normal(n, groups, dk), v=normal(n, heads, dv),
                 log_decay=_log_decays(case, gen, n))
        # slots: every stream reads its state at one place of the pool and writes it at another
        s["pool"] = normal(2 * n, heads, dk, dv, dtype=torch.float32)
        if case["slots"]:
            perm = torch.randperm(2 * n, generator=gen, device=DEV).to(torch.int32)
            s["src"], s["dst"] = perm[:n].contiguous(), perm[n:].contiguous()
        else:
            s["src"] = torch.arange(n, device=DEV, dtype=torch.int32)
            s["dst"] = s["src"] + n
        if own:
            from bidirectional_selective_scan_amd import binding
            s["call"] = binding.PreparedLinAttnStep(s["q"], s["k"], s["v"], s["log_decay"], s["pool"], scale=s["scale"],
                                                    slots_in=s["src"], slots_out=s["dst"])
        return s
    lens = _lengths(case)
    shape = (1, sum(lens)) if case["packed"] else (case["nseq"], case["length"])
    if case["fused"]:
        wide = [groups * dk, groups * dk, heads * dv]
        parts = normal(*shape, sum(wide)).split(wide, -1)
        s["q"], s["k"], s["v"] = (p.unflatten(-1, (h, -1)) for p, h in zip(parts, (groups, groups, heads)))
    else:
        s.update(q=normal(*shape, groups, dk), k=normal(*shape, groups, dk), v=normal(*shape, heads, dv))
    s["log_decay"] = _log_decays(case, gen, *shape)
    s["h0"] = normal(len(lens), heads, dk, dv, dtype=torch.float32) if case["state"] else None
    if case["train"]:
        s["dy"] = normal(*shape, heads, dv)
        s["dh_last"] = normal(len(lens), heads, dk, dv, dtype=torch.float32) if case["state"] else None
    starts = [0]
    for v in lens:
        starts.append(starts[-1] + v)
    s["offsets"] = torch.tensor(starts, dtype=torch.int32).to(DEV)
    if own:
        from bidirectional_selective_scan_amd import binding
        s["call"] = binding.PreparedLinAttn(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], h0=s["h0"],
                                            offsets=s["offsets"] if case["packed"] else None, reverse=case["reverse"])
        if case["train"]:
            s["grad"] = binding.PreparedLinAttnGrad(s["call"], dy=s["dy"], dh_last=s["dh_last"])
    else:
        # the chunks of the plain form: tokens in walking order (-1: none), the sequence of each, where it starts and ends
        rows, seq, first, last = [], [], [], []
        for k, v in enumerate(lens):
            pos = torch.arange(starts[k], starts[k] + v)
            pos = pos.flip(0) if case["reverse"] else pos
            m = -(-v // CHUNK)
            full = torch.full((m * CHUNK,), -1, dtype=torch.long)
            full[:v] = pos
            rows.append(full.view(m, CHUNK))
            seq += [k] * m
            first += [j == 0 for j in range(m)]
            last += [j == m - 1 for j in range(m)]
        s["index"] = torch.cat(rows).to(DEV)
        s["seq"] = torch.tensor(seq, dtype=torch.long, device=DEV)
        s["first"] = torch.tensor(first, dtype=torch.bool, device=DEV)
        s["last"] = torch.tensor(last, dtype=torch.bool, device=DEV)
        s["steps"] = max(-(-v // CHUNK) for v in lens)
    return s


# ------------------------------------------------------------------------------------------
# Plain forms, 32 bits


def _doubling(a, b, steps):
    """S_n = a_n S_{n-1} + b_n along dim 0 by doubling (a 0 where a sequence starts)."""
    step = 1
    while step < steps:
        nb, na = b.clone(), a.clone()
        nb[step:] += a[step:] * b[:-step]
        na[step:] *= a[:-step]
        a, b, step = na, nb, 2 * step
    return b


def _chunks(t, index, live, heads):
    """Rows (tokens, h, d) as chunks (n, heads, CHUNK, d) in 32 bits, zeros where there is no token."""
    c = t[index.clamp(min=0)].float() * live[..., None, None]
    c = c.transpose(1, 2)
    return c.repeat_interleave(heads // c.shape[1], 1).contiguous()


def _turned(t):
    return t.transpose(-1, -2).contiguous()


def _attn_plain(s):
    case = s["case"]
    heads, groups, dk, dv = (case[k] for k in ("heads", "groups", "dk", "dv"))
    dt, index, scale = s["q"].dtype, s["index"], s["scale"]
    lead = s["q"].shape[:2]
    live = index >= 0
    q = _chunks(s["q"].reshape(-1, groups, dk), index, live, heads)
    k = _chunks(s["k"].reshape(-1, groups, dk), index, live, heads)
    v = _chunks(s["v"].reshape(-1, heads, dv), index, live, heads)
    ld = s["log_decay"]
    ld = ld.expand(lead[0] * lead[1], heads) if ld.dim() == 1 else ld.reshape(-1, heads)
    G = (ld[index.clamp(min=0)] * live[..., None]).transpose(1, 2).double().cumsum(-1)       # (n, heads, CHUNK)
    end = G[..., -1:]
    tri = torch.ones(CHUNK, CHUNK, device=G.device).tril().bool()
    M = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~tri, -math.inf).float())
    into = torch.exp(G.float())[..., None]                  # from the chunk's start to a token
    out = torch.exp((end - G).float())[..., None]           # from a token to the chunk's end
    a = torch.exp(end.float())[..., None]
    first, last, seq, steps = s["first"], s["last"], s["seq"], s["steps"]
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(case["nseq"], heads, dk, dv, device=q.device)
    part = _turned(k * out) @ v
    part[first] += a[first] * h0[seq[first]]
    cut = a.clone()
    cut[first] = 0
    after = _doubling(cut, part, steps)
    before = torch.zeros_like(after)
    before[1:] = after[:-1]
    before[first] = h0[seq[first]]
    A = q @ _turned(k) * M
    y = scale * (A @ v + (q * into) @ before)
    h_last = h0.clone()
    h_last[seq[last]] = after[last]

    def rows(t, groups_):
        """Chunks back as rows of tokens, summed over the heads of a group."""
        t = t.view(t.shape[0], groups_, heads // groups_, CHUNK, -1).sum(2).transpose(1, 2)
        o = torch.zeros(lead[0] * lead[1], groups_, t.shape[-1], device=t.device)
        o[index[live]] = t[live]
        return o.view(*lead, groups_, -1)

    outs = [rows(y, heads).to(dt), h_last]
    if not case["train"]:
        return outs
    dy = _chunks(s["dy"].reshape(-1, heads, dv), index, live, heads) * scale
    dh = s["dh_last"] if s["dh_last"] is not None else torch.zeros_like(h0)
    # gradient of the state that leaves a chunk, from the last chunk to the first
    own_part = _turned(q * into) @ dy
    own_part[last] += a[last] * dh[seq[last]]
    cut = a.clone()
    cut[last] = 0
    enter = _doubling(cut.flip(0), own_part.flip(0), steps).flip(0)
    leave = torch.zeros_like(enter)
    leave[:-1] = enter[1:]
    leave[last] = dh[seq[last]]
    P = dy @ _turned(v) * M
    dq = P @ k + into * (dy @ _turned(before))
    dk_ = _turned(P) @ q + out * (v @ _turned(leave))
    dv_ = _turned(A) @ dy + out * (k @ leave)
    w = ((q * dq).sum(-1) - (k * dk_).sum(-1)).double()
    w[..., -1] += (after.double() * leave).sum((-1, -2))
    dg = rows(w.flip(-1).cumsum(-1).flip(-1).float()[..., None], heads)[..., 0]
    if s["log_decay"].dim() == 1:
        dg = dg.double().sum((0, 1)).float()
    outs += [rows(dq, groups).to(dt), rows(dk_, groups).to(dt), rows(dv_, heads).to(dt), dg]
    if s["h0"] is not None:
        dh0 = dh.clone()
        dh0[seq[first]] = enter[first]
        outs.append(dh0)
    return outs


def _step_plain(s):
    case = s["case"]
    rep = case["heads"] // case["groups"]
    src, dst = s["src"].long(), s["dst"].long()
    q, k = (s[n].float().repeat_interleave(rep, 1) for n in ("q", "k"))
    a = torch.exp(s["log_decay"]).expand(case["batch"], case["heads"])
    h = a[..., None, None] * s["pool"][src] + k[..., None] * s["v"].float()[..., None, :]
    s["pool"][dst] = h
    return [(s["scale"] * (q[..., None] * h).sum(-2)).to(s["q"].dtype), s["pool"]]


def _ln_plain(s):
    x, dt = s["x"].float(), s["x"].dtype
    res = s["residual"]
    tot = x + res.float() if res is not None else x
    off = tot - tot.mean(-1, keepdim=True)
    rho = torch.rsqrt((off * off).mean(-1, keepdim=True) + EPS)
    xh = off * rho
    n = xh * s["weight"] + s["bias"] if s["weight"] is not None else xh
    outs = ([tot.to(res.dtype)] if res is not None else []) + [n.to(dt)]
    if not s["case"]["train"]:
        return outs
    dn = s["dn"].float()
    g = dn * s["weight"] if s["weight"] is not None else dn
    ds = rho * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    if res is not None:
        ds = ds + s["dsum"].float()
    outs.append(ds.to(dt))
    if res is not None:
        outs.append(ds.to(res.dtype))
    if s["weight"] is not None:
        outs += [(dn * xh).sum(0), dn.sum(0)]
    return outs


def run(state):
    case = state["case"]
    if not own:
        return {"step": _step_plain, "attn": _attn_plain, "ln": _ln_plain}[case["op"]](state)
    call = state["call"]
    call()
    if case["op"] == "step":
        return [call.y, state["pool"]]
    if case["op"] == "attn":
        outs = [call.y, call.h_last]
        if case["train"]:
            g = state["grad"]
            g()
            outs += [g.dq, g.dk, g.dv, g.dlog_decay] + ([g.dh0] if case["state"] else [])
        return outs
    outs = [t for t in (call.sum, call.n) if t is not None]
    if case["train"]:
        g = state["grad"]
        g()
        outs += [t for t in (g.dx, g.dresidual, g.dweight, g.dbias) if t is not None]
    return outs


# ------------------------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    e = 2 if case["io"] == "bf16" else 4
    if case["op"] == "ln":
        size, d = case["rows"] * case["d"], case["d"]
        re = {"f32": 4, "io": e, "none": 0}[case["res"]]
        nw = 8 * d if case["affine"] else 0
        b, f = size * (2 * e + 2 * re) + nw, 10 * size
        if case["train"]:
            b += size * (3 * e + 3 * re) + 2 * nw    # x and the residual again, dn and dsum; dx and dresidual
            f += 18 * size
        return {"bytes": b, "flops": f}
    heads, groups, dk, dv = (case[k] for k in ("heads", "groups", "dk", "dv"))
    if case["op"] == "step":
        n = case["batch"]
        gb = 4 * heads * (n if case["decay"] == "token" else 1)
        return {"bytes": n * (heads * dk * dv * 8 + e * (2 * groups * dk + 2 * heads * dv) + 8) + gb,
                "flops": n * heads * dk * dv * 5}
    lens = _lengths(case)
    n = sum(lens)
    state = len(lens) * heads * dk * dv * 4
    gb = 4 * heads * (n if case["decay"] == "token" else 1)
    b = n * e * (2 * groups * dk + 2 * heads * dv) + gb + state * (2 if case["state"] else 1)
    b += 4 * len(lens) + 4 if case["packed"] else 0
    f = n * heads * 4 * dk * dv
    if case["train"]:
        b += n * e * (4 * groups * dk + 3 * heads * dv) + 2 * gb + (3 * state if case["state"] else 0)
        f += n * heads * 10 * dk * dv
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------------------------
# The definitions in 64 bits, token by token


def _exact_attn(case, s):
    lens = _lengths(case)
    heads, groups, dk, dv = (case[k] for k in ("heads", "groups", "dk", "dv"))
    n, nseq, longest, rep = sum(lens), len(lens), max(lens), heads // groups
    wide = dict(dtype=torch.float64, device=DEV)
    # a token's place in walking order: (longest, nseq); tokens past an end go to a row of their own (n)
    pos = torch.full((longest, nseq), n, dtype=torch.long)
    at = 0
    for j, v in enumerate(lens):
        p = torch.arange(at, at + v)
        pos[:v, j] = p.flip(0) if case["reverse"] else p
        at += v
    live = (pos < n).double().to(DEV)[..., None, None, None]
    whole = all(v == longest for v in lens)
    pos = pos.to(DEV)

    def padded(t, h, d):
        return torch.cat([t.reshape(n, h, d).double(), torch.zeros(1, h, d, **wide)]).repeat_interleave(heads // h, 1)

    q, k, v = padded(s["q"], groups, dk), padded(s["k"], groups, dk), padded(s["v"], heads, dv)
    ld = s["log_decay"]
    ld = ld.expand(n, heads) if ld.dim() == 1 else ld
    dec = torch.exp(padded(ld, heads, 1))[..., None]          # 1 in the row past the end
    h0 = s["h0"].double() if s["h0"] is not None else torch.zeros(nseq, heads, dk, dv, **wide)
    S = h0.clone()
    y = torch.zeros(n + 1, heads, dv, **wide)
    train = case["train"]
    if train:
        dy = padded(s["dy"], heads, dv) * s["scale"]
        store = torch.empty(longest, nseq, heads, dk, dv, **wide)    # the state before a token
        dq = torch.zeros(n + 1, heads, dk, **wide)
        dk_, dv_, dg = torch.zeros_like(dq), torch.zeros_like(y), torch.zeros(n + 1, heads, **wide)
    for t in range(longest):
        i = pos[t]
        if train:
            store[t] = S
        S = dec[i] * S
        S += k[i].unsqueeze(-1) * v[i].unsqueeze(-2)
        y[i] = torch.matmul(q[i].unsqueeze(-2), S).squeeze(-2)
        if train:
            dq[i] = (S * dy[i].unsqueeze(-2)).sum(-1)
    outs = [(y[:n] * s["scale"]).view(s["v"].shape), S]
    if not train:
        return outs
    E = s["dh_last"].double() if s["dh_last"] is not None else torch.zeros_like(h0)
    for t in range(longest - 1, -1, -1):
        i = pos[t]
        D = E + q[i].unsqueeze(-1) * dy[i].unsqueeze(-2)
        dk_[i] = (D * v[i].unsqueeze(-2)).sum(-1)
        dv_[i] = (D * k[i].unsqueeze(-1)).sum(-2)
        B = dec[i] * D
        dg[i] = (B * store[t]).sum((-1, -2))
        E = B if whole else torch.where(live[t] > 0, B, E)

    def shared(t):
        return t[:n].view(n, groups, rep, dk).sum(2).view(s["q"].shape)

    dg = dg[:n]
    outs += [shared(dq), shared(dk_), dv_[:n].view(s["v"].shape),
             dg.sum(0) if s["log_decay"].dim() == 1 else dg.view(s["log_decay"].shape)]
    if s["h0"] is not None:
        outs.append(E)
    return outs


def _exact_ln(case, s):
    """Chunks of rows through torch's own differentiation of the definition in 64 bits."""
    names = ("x", "residual", "weight", "bias")
    wgrad = {k: 0 for k in ("weight", "bias")}
    parts = []
    per = max(1, (1 << 24) // case["d"])
    for lo in range(0, case["rows"], per):
        v = {}
        for k in names:
            t = s[k]
            if t is not None:
                t = (t if k in wgrad else t[lo:lo + per]).double().detach().requires_grad_(case["train"])
            v[k] = t
        tot = v["x"] + v["residual"] if v["residual"] is not None else v["x"]
        var = tot.pow(2).mean(1, keepdim=True) - tot.mean(1, keepdim=True).pow(2)
        nn = (tot - tot.mean(1, keepdim=True)) / torch.sqrt(var + EPS)
        if v["weight"] is not None:
            nn = nn * v["weight"] + v["bias"]
        part = ([tot.detach()] if v["residual"] is not None else []) + [nn.detach()]
        if case["train"]:
            obj = (nn * s["dn"][lo:lo + per].double()).sum()
            if v["residual"] is not None:
                obj = obj + (tot * s["dsum"][lo:lo + per].double()).sum()
            have = [k for k in names if v[k] is not None]
            for k, g in zip(have, torch.autograd.grad(obj, [v[k] for k in have])):
                if k in wgrad:
                    wgrad[k] = wgrad[k] + g
                else:
                    part.append(g)
        parts.append(part)
    outs = [torch.cat([p[j] for p in parts]) for j in range(len(parts[0]))]
    if case["train"]:
        outs += [wgrad[k] for k in ("weight", "bias") if s[k] is not None]
    return outs


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    if case["op"] == "attn":
        return _exact_attn(case, s)
    if case["op"] == "ln":
        return _exact_ln(case, s)
    rep = case["heads"] // case["groups"]
    q, k = (s[n].double().repeat_interleave(rep, 1) for n in ("q", "k"))
    pool = s["pool"].double()
    h = pool[s["src"].long()] * torch.exp(s["log_decay"].double()).expand(case["batch"], case["heads"])[..., None, None]
    h = h + torch.matmul(k.unsqueeze(-1), s["v"].double().unsqueeze(-2))
    pool[s["dst"].long()] = h
    return [torch.matmul(q.unsqueeze(-2), h).squeeze(-2) * s["scale"], pool]
