"""Cases of the selective state space block's operators: the short causal convolution, the
selective scan, and the norms, gate and residual around a block.

`run` computes them either with elementary torch operations in 32 bits (own = False) or through
the library's entry points (own = True).  `exact` computes the same outputs in 64 bits, token by
token, from the definitions.

    convolution   pre[t] = bias + sum_j w[:, j] x[t - K + 1 + j],   y = silu(pre)
    scan          d = softplus(dt + dt_bias),  h[t] = exp(d A) h[t-1] + d x B,
                  y = (sum_n C h + D x) silu(z)
    block norm    n = w_post norm(o) silu(gate),  r' = r + scale n,  v = w_pre norm(r')

Sizes follow the repository's workloads (one prompt of 8192 tokens, 65536 tokens, a training
batch of 8 x 2048, 64 sequences decoded together, 32 heads x 128 = 4096 channels) and generic odd
ones.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------- the cases


def listed():
    return [
        # one long prompt through the convolution in front of the scan; the tail is kept for decoding
        dict(name="conv_prompt", op="conv", mode="prompt", dtype="bf16", B=1, L=8192, C=4096, K=4, lens=""),
        # a training step's convolution, forward and gradients
        dict(name="conv_train", op="conv", mode="train", dtype="bf16", B=8, L=2048, C=4096, K=4, lens=""),
        # one token for each of 64 sequences whose states sit in a cache of slots, some rows idle
        dict(name="conv_step", op="conv", mode="step", dtype="bf16", B=64, L=1, C=4096, K=4, lens=""),
        # one long prompt through the scan, final state kept for decoding
        dict(name="scan_prompt", op="scan", mode="prompt", dtype="bf16", B=1, L=8192, C=4096, N=16, G=1, lens=""),
        # a packed batch of ragged prompts (one empty, one of a single token) continuing earlier states, fp32
        dict(name="scan_packed", op="scan", mode="prompt", dtype="f32", B=1, L=8362, C=1000, N=16, G=2,
             lens="1,2047,0,333,64,5000,17,900"),
        # a very long context with few channels: only the time axis is long
        dict(name="scan_long", op="scan", mode="prompt", dtype="bf16", B=1, L=65536, C=1024, N=16, G=8, lens=""),
        # a training step's scan, forward and all gradients
        dict(name="scan_train", op="scan", mode="train", dtype="bf16", B=8, L=2048, C=4096, N=16, G=1, lens=""),
        # training on odd sizes in fp32, as in a numerics check of a small model
        dict(name="scan_train_odd", op="scan", mode="train", dtype="f32", B=3, L=777, C=520, N=24, G=4, lens=""),
        # one token for each of 64 sequences, states in a cache of slots, some rows idle
        dict(name="scan_step", op="scan", mode="step", dtype="bf16", B=64, L=1, C=4096, N=16, G=1, lens=""),
        # a training step's norms around a block, everything on, forward and all gradients
        dict(name="norm_train", op="norm", mode="train", dtype="bf16", T=16384, D=4096, groups=1, gate=True, gate_first=False,
             residual="bf16", pre=True),
        # the gated norm over 32 heads between a prompt's scan and its output projection
        dict(name="norm_heads", op="norm", mode="prompt", dtype="bf16", T=8192, D=4096, groups=32, gate=True, gate_first=True,
             residual="", pre=False),
        # one token for each of 64 sequences, residual stream in fp32
        dict(name="norm_token", op="norm", mode="prompt", dtype="bf16", T=64, D=4096, groups=1, gate=False, gate_first=False,
             residual="f32", pre=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        T, D = _log(rng, 1, 16384), _log(rng, 8, 8192)
        T = min(T, 16384 * 4096 // (D * SIZE[dtype] // 2))
        groups = rng.choice([g for g in (1, 1, 2, 4, 8, 16, 32) if D % g == 0])
        residual = rng.choice(["", dtype, "f32"])
        return dict(op=op, mode=rng.choice(["prompt", "train"]), dtype=dtype, T=T, D=D, groups=groups, gate=rng.random() < 0.7,
                    gate_first=rng.random() < 0.5, residual=residual, pre=residual != "" and rng.random() < 0.8)
    mode = rng.choice(["prompt", "train", "step"])
    if mode == "step":
        c = dict(op=op, mode=mode, dtype=dtype, B=_log(rng, 1, 256), L=1, C=_log(rng, 8, 6144), lens="")
    else:
        B, C = rng.choice([1, 1, 2, 3, 8]), _log(rng, 8, 6144)
        top = 16384 * 4096 // (2 * C * B) if mode == "train" else 8192 * 4096 // (C * B)
        L = _log(rng, 1, max(1, min(65536, top)))
        lens = ""
        if mode == "prompt" and B > 1:  # the same tokens as one packed batch with ragged lengths
            T = B * L
            cuts = sorted(rng.randrange(T + 1) for _ in range(B - 1))
            lens = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [T]))
            B, L = 1, T
        c = dict(op=op, mode=mode, dtype=dtype, B=B, L=L, C=C, lens=lens)
    if op == "conv":
        return dict(c, K=rng.choice([2, 3, 4, 4, 5, 8]))
    N = rng.choice([1, 4, 8, 16, 16, 16, 24, 32, 64])
    if N > 16:  # no more elements than with 16 states
        c["C"] = max(8, c["C"] * 16 // N)
    return dict(c, N=N, G=rng.choice([g for g in (1, 1, 2, 4, 8) if c["C"] % g == 0]))


# ------------------------------------------------------------------------------- the inputs


def prepare(case, seed):
    gen = torch.Generator(DEVICE)
    gen.manual_seed(seed)
    tp = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=None):
        t = torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)
        return (t * std + mean).to(tp if dtype is None else dtype)

    f32 = torch.float32
    s = dict(case=case)
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        s.update(o=normal(T, D), w_post=normal(D, std=0.1, mean=1.0, dtype=f32))
        s["gate"] = normal(T, D) if case["gate"] else None
        rtp = TYPES[case["residual"]] if case["residual"] else tp
        s["r"] = normal(T, D, dtype=rtp) if case["residual"] else None
        s["scale"] = normal(D, std=0.1, mean=0.5, dtype=f32) if case["residual"] else None
        s["w_pre"] = normal(D, std=0.1, mean=1.0, dtype=f32) if case["pre"] else None
        if case["mode"] == "train":
            s["dr_out"] = normal(T, D, dtype=rtp)
            s["dn_out"] = normal(T, D) if case["pre"] else None
        return s
    B, L, C = case["B"], case["L"], case["C"]
    step, train = case["mode"] == "step", case["mode"] == "train"
    lens = [int(v) for v in case["lens"].split(",")] if case["lens"] else []
    s["cu_seqlens"] = None
    if lens:
        ends = torch.tensor(lens, dtype=torch.int64).cumsum(0)
        s["cu_seqlens"] = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(DEVICE)
    nstate = len(lens) if lens else B
    slots = None
    if step:  # each sequence's state sits in a slot of its own; a slot of -1 is an idle row
        nstate = B + B // 2 + 1
        order = torch.randperm(nstate, generator=gen, device=DEVICE)[:B]
        idle = torch.rand(B, generator=gen, device=DEVICE) < 0.05
        slots = torch.where(idle, torch.full_like(order, -1), order)
    s["slots"] = slots
    shape = (B,) if step else (B, L)
    if case["op"] == "conv":
        K = case["K"]
        s.update(x=normal(*shape, C), w=normal(C, K, std=K ** -0.5, dtype=f32), bias=normal(C, std=0.1, dtype=f32))
        s["state"] = normal(nstate, K - 1, C) if step or lens else None
        s["state_out"] = None if step or train else torch.empty(nstate, K - 1, C, dtype=tp, device=DEVICE)
        if train:
            s["dy"] = normal(*shape, C)
        return s
    N, G = case["N"], case["G"]
    # step sizes of 0.001 to 0.1 through the bias, decay rates 1 .. N with some spread
    size = torch.exp(torch.rand(C, generator=gen, device=DEVICE) * math.log(100.0) + math.log(1e-3))
    s.update(x=normal(*shape, C), dt=normal(*shape, C, std=0.5), dt_bias=torch.log(torch.expm1(size)),
             Bm=normal(*shape, G, N), Cm=normal(*shape, G, N), D=normal(C, std=0.1, mean=1.0, dtype=f32),
             z=normal(*shape, C))
    s["A"] = -torch.arange(1, N + 1, device=DEVICE, dtype=f32) * torch.exp(normal(C, N, std=0.1, dtype=f32))
    s["state"] = normal(nstate, C, N, dtype=f32) if step or lens else None
    s["h_out"] = None if step or train else torch.empty(nstate, C, N, dtype=f32, device=DEVICE)
    if train:
        s["dy"] = normal(*shape, C)
    return s


# ------------------------------------------------------------------- the operators, plain form


def _dsilu(v, sg):
    return sg * (1 + v * (1 - sg))


def _places(s, rows):
    """For each token row of a batch: its sequence and its place in it."""
    case = s["case"]
    at = torch.arange(rows, device=DEVICE)
    if s["cu_seqlens"] is None:
        return at // case["L"], at % case["L"]
    seq = torch.searchsorted(s["cu_seqlens"], at, right=True) - 1
    return seq, at - s["cu_seqlens"][seq]


def _ends(s):
    """Offsets of the sequences, one more than there are."""
    case = s["case"]
    if s["cu_seqlens"] is not None:
        return s["cu_seqlens"]
    return torch.arange(case["B"] + 1, device=DEVICE) * case["L"]


def _conv(s):
    case, x = s["case"], s["x"]
    C, K = case["C"], case["K"]
    if case["mode"] == "step":
        live = (s["slots"] >= 0)[:, None]
        slot = s["slots"].clamp(min=0)
        seen = torch.cat([s["state"][slot], x[:, None]], 1)  # [B, K, C]
        pre = s["bias"] + (seen.float() * s["w"].t()).sum(1)
        y = torch.where(live, pre * torch.sigmoid(pre), 0.0).to(x.dtype)
        # rows that are idle write to a slot that is thrown away
        spare = torch.cat([s["state"], s["state"][:1]])
        spare[torch.where(live[:, 0], slot, len(s["state"]))] = seen[:, 1:]
        s["state"].copy_(spare[:-1])
        return dict(y=y, state=s["state"])
    rows = x.shape[0] * x.shape[1]
    seq, place = _places(s, rows)
    ends = _ends(s)
    nseq = len(ends) - 1
    before = torch.zeros(nseq, K - 1, C, device=DEVICE) if s["state"] is None else s["state"].float()
    known = torch.cat([before.reshape(-1, C), x.reshape(rows, C).float()])
    base = nseq * (K - 1)
    tap = torch.arange(K, device=DEVICE)
    back = place[:, None] - (K - 1) + tap  # place of each tap's input in its sequence
    index = torch.where(back >= 0, base + torch.arange(rows, device=DEVICE)[:, None] - (K - 1) + tap,
                        (seq * (K - 1) + place)[:, None] + tap)
    seen = known[index]  # [rows, K, C]
    pre = s["bias"] + (seen * s["w"].t()).sum(1)
    sg = torch.sigmoid(pre)
    y = (pre * sg).to(x.dtype).reshape(x.shape)
    if case["mode"] == "prompt":
        tail = torch.arange(K - 1, device=DEVICE) - (K - 1)
        length = (ends[1:] - ends[:-1])[:, None]
        last = torch.where(length + tail >= 0, base + ends[1:, None] + tail,
                           torch.arange(nseq, device=DEVICE)[:, None] * (K - 1) + length + tail + (K - 1))
        s["state_out"].copy_(known[last])
        return dict(y=y, state=s["state_out"])
    dp = s["dy"].reshape(rows, C).float() * _dsilu(pre, sg)
    dknown = torch.zeros_like(known).index_add_(0, index.reshape(-1), (dp[:, None] * s["w"].t()).reshape(-1, C))
    return dict(y=y, dx=dknown[base:].to(x.dtype).reshape(x.shape),
                dw=(dp[:, None].double() * seen).sum(0).t().float(), dbias=dp.sum(0, dtype=torch.float64).float())


def _recur(a, b):
    """h[t] = a[t] h[t-1] + b[t] over axis 1, by halving: pairs of steps make one step."""
    n = a.shape[1]
    if n == 1:
        return b
    even, odd = slice(0, n - n % 2, 2), slice(1, n, 2)
    half = _recur(a[:, odd] * a[:, even], torch.addcmul(b[:, odd], a[:, odd], b[:, even]))
    h = torch.empty_like(b)
    h[:, odd] = half
    h[:, 0] = b[:, 0]
    h[:, 2::2] = torch.addcmul(b[:, 2::2], a[:, 2::2], half[:, : (n + 1) // 2 - 1])
    return h


def _scan(s):
    case, x = s["case"], s["x"]
    C, N, G = case["C"], case["N"], case["G"]
    step = case["mode"] == "step"
    B, L = (case["B"], 1) if step else (case["B"], case["L"])
    xf, z = x.float().reshape(B, L, C, 1), s["z"].float().reshape(B, L, C)
    raw = s["dt"].float().reshape(B, L, C) + s["dt_bias"]
    d = torch.logaddexp(raw, torch.zeros_like(raw))[..., None]
    Bm = s["Bm"].float().reshape(B, L, G, 1, N)
    Cm = s["Cm"].float().reshape(B, L, G, 1, N)
    a = torch.exp(d * s["A"])  # [B, L, C, N]
    b = ((d * xf).reshape(B, L, G, C // G, 1) * Bm).reshape(B, L, C, N)
    sz = torch.sigmoid(z)
    if step:
        live = s["slots"] >= 0
        slot = s["slots"].clamp(min=0)
        h = torch.addcmul(b, a, s["state"][slot][:, None])
        y = ((h.reshape(B, L, G, C // G, N) * Cm).sum(-1).reshape(B, L, C) + s["D"] * xf[..., 0]) * (z * sz)
        spare = torch.cat([s["state"], s["state"][:1]])
        spare[torch.where(live, slot, len(s["state"]))] = h[:, 0]
        s["state"].copy_(spare[:-1])
        return dict(y=torch.where(live[:, None], y[:, 0], 0.0).to(x.dtype), state=s["state"])
    ends = _ends(s)
    if s["state"] is not None:  # a sequence's first token takes the state it begins with, and nothing else
        seq, place = _places(s, L)
        begin = (place == 0)[None, :, None, None]
        b = b + torch.where(begin, a * s["state"][seq], 0.0)
        a = torch.where(begin, 0.0, a)
    h = _recur(a, b)
    ch = (h.reshape(B, L, G, C // G, N) * Cm).sum(-1).reshape(B, L, C) + s["D"] * xf[..., 0]
    y = (ch * (z * sz)).to(x.dtype)
    if case["mode"] == "prompt":
        # an empty sequence keeps the state it begins with
        last = h.reshape(B * L, C, N)[(ends[1:] - 1).clamp(min=0)]
        if s["state"] is not None:
            last = torch.where((ends[1:] > ends[:-1])[:, None, None], last, s["state"])
        s["h_out"].copy_(last)
        return dict(y=y, h=s["h_out"])
    dy = s["dy"].float()
    e = (dy * (z * sz))[..., None]
    ec = (e.reshape(B, L, G, C // G, 1) * Cm).reshape(B, L, C, N)
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)  # the decay of the step after
    g = _recur(after.flip(1), ec.flip(1)).flip(1)
    del ec, after
    gb = (g.reshape(B, L, G, C // G, N) * Bm).sum(-1).reshape(B, L, C)
    dBm = (g * (d * xf)).reshape(B, L, G, C // G, N).sum(3)
    dCm = (h * e).reshape(B, L, G, C // G, N).sum(3)
    q = g * a
    q[:, 1:] *= h[:, :-1]
    q[:, 0] = 0
    dd = xf[..., 0] * gb + (q * s["A"]).sum(-1)
    ddt = dd * torch.sigmoid(raw)
    return dict(y=y, dx=(d[..., 0] * gb + s["D"] * e[..., 0]).to(x.dtype), ddt=ddt.to(x.dtype),
                dz=(dy * ch * _dsilu(z, sz)).to(x.dtype), dBm=dBm.to(x.dtype), dCm=dCm.to(x.dtype),
                dA=(q * d).sum(1, dtype=torch.float64).sum(0).float(),
                dD=(e * xf)[..., 0].sum((0, 1), dtype=torch.float64).float(),
                ddt_bias=ddt.sum((0, 1), dtype=torch.float64).float())


def _norm(s):
    case, o = s["case"], s["o"]
    T, D, groups = case["T"], case["D"], case["groups"]
    u = o.float()
    if case["gate"]:
        gate = s["gate"].float()
        sg = torch.sigmoid(gate)
        act = gate * sg
    if case["gate"] and case["gate_first"]:
        u = u * act
    ug = u.reshape(T, groups, D // groups)
    rs = torch.rsqrt(ug.square().mean(-1, keepdim=True) + EPS)
    unit = (ug * rs).reshape(T, D)
    n = unit * s["w_post"]
    if case["gate"] and not case["gate_first"]:
        n = n * act
    rr = n if s["r"] is None else s["r"].float() + s["scale"] * n
    out = dict(r_out=rr.to(s["r"].dtype if s["r"] is not None else o.dtype))
    if case["pre"]:
        rp = torch.rsqrt(rr.square().mean(-1, keepdim=True) + EPS)
        out["n_out"] = (rr * rp * s["w_pre"]).to(o.dtype)
    if case["mode"] == "prompt":
        return out
    dr = s["dr_out"].float()
    if case["pre"]:
        dn = s["dn_out"].float()
        dv = dn * s["w_pre"]
        dr = dr + rp * (dv - rr * rp.square() * (dv * rr).mean(-1, keepdim=True))
        out["dw_pre"] = (dn * rr * rp).sum(0, dtype=torch.float64).float()
    dm = dr
    if s["r"] is not None:
        out["dr"] = dr.to(s["r"].dtype)
        out["dscale"] = (dr * n).sum(0, dtype=torch.float64).float()
        dm = dr * s["scale"]
    if case["gate"] and not case["gate_first"]:
        out["dgate"] = (dm * unit * s["w_post"] * _dsilu(gate, sg)).to(o.dtype)
        dm = dm * act
    out["dw_post"] = (dm * unit).sum(0, dtype=torch.float64).float()
    du = (dm * s["w_post"]).reshape(T, groups, D // groups)
    uu = unit.reshape(T, groups, D // groups)
    du = (rs * (du - uu * (du * uu).mean(-1, keepdim=True))).reshape(T, D)
    if case["gate"] and case["gate_first"]:
        out["dgate"] = (du * o.float() * _dsilu(gate, sg)).to(o.dtype)
        du = du * act
    out["do"] = du.to(o.dtype)
    return out


# ---------------------------------------------------------- the same through the library's calls


def _own_conv(s):
    from gated_linear_sliding_gb300 import lizard as lz

    if s["case"]["mode"] == "step":
        y = lz.lizard_conv_step(s["x"], s["w"], s["bias"], s["state"], slots=s["slots"], act=lz.LIZARD_ACT_SILU)
        return dict(y=y, state=s["state"])
    y = lz.lizard_conv_fwd(s["x"], s["w"], s["bias"], act=lz.LIZARD_ACT_SILU, state_in=s["state"], state_out=s["state_out"],
                           cu_seqlens=s["cu_seqlens"])
    if s["case"]["mode"] == "prompt":
        return dict(y=y, state=s["state_out"])
    g = lz.lizard_conv_bwd(s["x"], s["w"], s["bias"], s["dy"], act=lz.LIZARD_ACT_SILU)
    return dict(y=y, dx=g["dx"], dw=g["dw"], dbias=g["dbias"])


def _own_scan(s):
    from gated_linear_sliding_gb300 import lizard as lz

    args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
    more = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], softplus=True)
    if s["case"]["mode"] == "step":
        y = lz.lizard_scan_step(*args, s["state"], slots=s["slots"], **more)
        return dict(y=y, state=s["state"])
    if s["case"]["mode"] == "prompt":
        y = lz.lizard_scan_fwd(*args, h0=s["state"], h_out=s["h_out"], cu_seqlens=s["cu_seqlens"], **more)
        return dict(y=y, h=s["h_out"])
    y, states = lz.lizard_scan_fwd(*args, save_states=True, **more)
    g = lz.lizard_scan_bwd(*args, s["dy"], states, **more)
    return dict(y=y, **{k: g[k] for k in ("dx", "ddt", "dz", "dBm", "dCm", "dA", "dD", "ddt_bias")})


def _own_norm(s):
    from gated_linear_sliding_gb300 import lizard as lz

    case = s["case"]
    how = dict(gate=s["gate"], r=s["r"], w_post=s["w_post"], scale=s["scale"], w_pre=s["w_pre"], groups=case["groups"],
               act=lz.LIZARD_ACT_SILU, gate_first=case["gate_first"], eps=EPS)
    r_out, n_out = lz.lizard_block_norm_fwd(s["o"], **how)
    out = dict(r_out=r_out)
    if case["pre"]:
        out["n_out"] = n_out
    if case["mode"] == "train":
        g = lz.lizard_block_norm_bwd(s["o"], dr_out=s["dr_out"], dn_out=s["dn_out"], **how)
        out.update({k: g[k] for k in ("do", "dgate", "dr", "dw_post", "dscale", "dw_pre") if g[k] is not None})
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm}[op](state)
    return {"conv": _conv, "scan": _scan, "norm": _norm}[op](state)


# --------------------------------------------------------------------------------- the bounds


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        er = SIZE[case["residual"]] if case["residual"] else e
        res = 1 if case["residual"] else 0
        fwd = T * D * (e * (1 + case["gate"]) + er * res + er + e * case["pre"])
        nbytes, flops = fwd, 12 * T * D
        if case["mode"] == "train":
            # o, gate, r, dr_out, dn_out in; do, dgate, dr out
            nbytes += T * D * (e * (2 + 2 * case["gate"]) + er * (1 + 2 * res) + e * case["pre"])
            flops += 30 * T * D
        return {"bytes": nbytes, "flops": flops}
    rows = case["B"] * case["L"]
    C = case["C"]
    nstate = len(case["lens"].split(",")) if case["lens"] else case["B"]
    begin = 2 if case["lens"] or case["mode"] == "step" else 1  # states read and written, or written
    if case["op"] == "conv":
        K = case["K"]
        nbytes, flops = 2 * rows * C * e, rows * C * (2 * K + 6)
        if case["mode"] == "train":
            nbytes += 3 * rows * C * e + 2 * C * (K + 1) * 4
            flops += rows * C * (6 * K + 12)
        else:
            nbytes += begin * nstate * (K - 1) * C * e
        return {"bytes": nbytes, "flops": flops}
    N, G = case["N"], case["G"]
    nbytes = rows * (4 * C + 2 * G * N) * e + C * (N + 2) * 4
    flops = rows * C * (7 * N + 12)
    if case["mode"] == "train":
        nbytes += rows * (7 * C + 4 * G * N) * e + 2 * C * (N + 2) * 4
        flops += rows * C * (20 * N + 30)
    else:
        nbytes += begin * nstate * C * N * 4
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------- the definitions, in 64 bits


def _sequences(s):
    """(row of the batch, first token, end) of each sequence."""
    case = s["case"]
    if s["cu_seqlens"] is None:
        return [(b, 0, case["L"]) for b in range(case["B"])]
    cu = s["cu_seqlens"].tolist()
    return [(0, a, b) for a, b in zip(cu, cu[1:])]


def _exact_conv(s):
    case, K = s["case"], s["case"]["K"]
    x, w, bias = s["x"].double(), s["w"].double(), s["bias"].double()
    if case["mode"] == "step":
        y, state = torch.zeros_like(x), s["state"].double()
        for b, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            pre = bias + w[:, K - 1] * x[b]
            for j in range(K - 1):
                pre = pre + w[:, j] * state[slot, j]
            y[b] = pre / (1 + torch.exp(-pre))
            state[slot] = torch.cat([state[slot, 1:], x[b][None]])
        return dict(y=y, state=state)
    y, tails = torch.zeros_like(x), []
    dx, dw, dbias = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(bias)
    for i, (row, lo, hi) in enumerate(_sequences(s)):
        past = torch.zeros(K - 1, x.shape[-1], dtype=torch.float64, device=DEVICE)
        if s["state"] is not None:
            past = s["state"][i].double()
        line = torch.cat([past, x[row, lo:hi]])
        n = hi - lo
        tails.append(line[len(line) - (K - 1):])
        pre = bias.expand(n, -1).clone()
        for j in range(K):
            pre += w[:, j] * line[j:j + n]
        y[row, lo:hi] = pre / (1 + torch.exp(-pre))
        if case["mode"] == "train":
            sg = 1 / (1 + torch.exp(-pre))
            dp = s["dy"][row, lo:hi].double() * (sg + pre * sg * (1 - sg))
            dline = torch.zeros_like(line)
            for j in range(K):
                dline[j:j + n] += w[:, j] * dp
                dw[:, j] += (dp * line[j:j + n]).sum(0)
            dx[row, lo:hi] = dline[K - 1:]
            dbias += dp.sum(0)
    if case["mode"] == "prompt":
        return dict(y=y, state=torch.stack(tails))
    return dict(y=y, dx=dx, dw=dw, dbias=dbias)


def _exact_scan(s):
    case = s["case"]
    C, G = case["C"], case["G"]
    A, D = s["A"].double(), s["D"].double()

    def spread(t):  # a group's B or C for each of its channels
        return t.double().repeat_interleave(C // G, dim=-2)

    def token(pick):
        """The step size, its inner value, input, gate of the tokens that `pick` picks."""
        raw = pick(s["dt"]).double() + s["dt_bias"].double()
        return torch.logaddexp(raw, torch.zeros_like(raw)), raw, pick(s["x"]).double(), pick(s["z"]).double()

    if case["mode"] == "step":
        live = s["slots"] >= 0
        slot = s["slots"][live]
        d, _, x, z = token(lambda t: t[live])
        state = s["state"].double()
        h = torch.exp(d[..., None] * A) * state[slot] + (d * x)[..., None] * spread(s["Bm"][live])
        y = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEVICE)
        y[live] = ((h * spread(s["Cm"][live])).sum(-1) + D * x) * z / (1 + torch.exp(-z))
        state[slot] = h
        return dict(y=y, state=state)
    if case["mode"] == "prompt":
        y, out = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEVICE), []
        for i, (row, lo, hi) in enumerate(_sequences(s)):
            h = torch.zeros_like(A) if s["state"] is None else s["state"][i].double()
            for t0 in range(lo, hi, 256):
                t1 = min(hi, t0 + 256)
                d, _, x, z = token(lambda t: t[row, t0:t1])
                a = torch.exp(d[..., None] * A)
                b = (d * x)[..., None] * spread(s["Bm"][row, t0:t1])
                for k in range(t1 - t0):
                    h = torch.addcmul(b[k], a[k], h)
                    b[k] = h
                y[row, t0:t1] = ((b * spread(s["Cm"][row, t0:t1])).sum(-1) + D * x) * z / (1 + torch.exp(-z))
            out.append(h)
        return dict(y=y, h=torch.stack(out))
    d, raw, x, z = token(lambda t: t)
    B, L = x.shape[:2]
    past = [torch.zeros(B, *A.shape, dtype=torch.float64, device=DEVICE)]
    for t in range(L):
        past.append(torch.addcmul((d[:, t] * x[:, t])[..., None] * spread(s["Bm"][:, t]), torch.exp(d[:, t, :, None] * A), past[-1]))
    sg = 1 / (1 + torch.exp(-z))
    dy = s["dy"].double()
    e = dy * z * sg
    y, gb, qa = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    dBm, dCm = (torch.zeros(B, L, G, A.shape[1], dtype=torch.float64, device=DEVICE) for _ in range(2))
    dA, g = torch.zeros_like(A), torch.zeros_like(past[0])
    for t in range(L - 1, -1, -1):
        Ct, a = spread(s["Cm"][:, t]), torch.exp(d[:, t, :, None] * A)
        h = past.pop()
        y[:, t] = (h * Ct).sum(-1) + D * x[:, t]
        g = g + Ct * e[:, t, :, None]
        gb[:, t] = (g * spread(s["Bm"][:, t])).sum(-1)
        dBm[:, t] = (g * (d[:, t] * x[:, t])[..., None]).reshape(B, G, C // G, -1).sum(2)
        dCm[:, t] = (h * e[:, t, :, None]).reshape(B, G, C // G, -1).sum(2)
        g = g * a
        q = g * past[-1]
        qa[:, t] = (q * A).sum(-1)
        dA += (q * d[:, t, :, None]).sum(0)
    ddt = (x * gb + qa) / (1 + torch.exp(-raw))
    return dict(y=y * z * sg, dx=d * gb + D * e, ddt=ddt, dz=dy * y * (sg + z * sg * (1 - sg)), dBm=dBm, dCm=dCm, dA=dA,
                dD=(e * x).sum((0, 1)), ddt_bias=ddt.sum((0, 1)))


def _exact_norm(s):
    """The forward from its definition; the gradients by the chain rule, one row's norm at a time."""
    case = s["case"]
    T, D, groups = case["T"], case["D"], case["groups"]

    def unit(v, k):
        v = v.reshape(T, k, D // k)
        root = torch.sqrt((v * v).sum(-1, keepdim=True) * k / D + EPS)
        return (v / root).reshape(T, D), root

    def dunit(dv, v, root, k):  # the gradient of v / root
        dv, v = dv.reshape(T, k, D // k), v.reshape(T, k, D // k)
        return (dv / root - v * ((dv * v).sum(-1, keepdim=True) * k / D) / root ** 3).reshape(T, D)

    o, wp = s["o"].double(), s["w_post"].double()
    gate = s["gate"].double() if case["gate"] else None
    sg = 1 / (1 + torch.exp(-gate)) if case["gate"] else None
    first, last = case["gate"] and case["gate_first"], case["gate"] and not case["gate_first"]
    u = o * gate * sg if first else o
    un, root = unit(u, groups)
    m = un * wp * gate * sg if last else un * wp
    rr = m if s["r"] is None else s["r"].double() + s["scale"].double() * m
    out = dict(r_out=rr)
    if case["pre"]:
        rn, rroot = unit(rr, 1)
        out["n_out"] = rn * s["w_pre"].double()
    if case["mode"] == "prompt":
        return out
    drr = s["dr_out"].double()
    if case["pre"]:
        dn = s["dn_out"].double()
        out["dw_pre"] = (dn * rn).sum(0)
        drr = drr + dunit(dn * s["w_pre"].double(), rr, rroot, 1)
    dm = drr
    if s["r"] is not None:
        out["dr"], out["dscale"] = drr, (drr * m).sum(0)
        dm = drr * s["scale"].double()
    if last:
        out["dgate"] = dm * un * wp * (sg + gate * sg * (1 - sg))
        dm = dm * gate * sg
    out["dw_post"] = (dm * un).sum(0)
    du = dunit(dm * wp, u, root, groups)
    if first:
        out["dgate"] = du * o * (sg + gate * sg * (1 - sg))
        du = du * gate * sg
    out["do"] = du
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](s)
