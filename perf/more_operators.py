"""Cases of two operators around a constant-memory mixer: the norms of queries and keys for each head
with the position rotation, and linear attention with a decay for each head.

`run` computes them either with elementary torch operations in 32 bits (own = False) or through the
library's entry points (own = True).  `exact` computes the same outputs in 64 bits, token by token
where there is a recurrence, from the definitions.

    rope    n = w x / sqrt(mean(x^2) + eps) per head,   a[i] = position[axis(i)] freqs[i]
            (y1, y2) = (n1 cos a - n2 sin a, n2 cos a + n1 sin a) for the pairs of the first `rot` values
    decay   S[t] = exp(log_decay) S[t-1] + k[t] v[t]^T,   o[t] = scale q[t] S[t]
            with query head h on the state of head h / (Hq / Hkv)

Sizes follow the repository's workloads (one prompt of 8192 tokens, 65536 tokens, a training batch of
8 x 2048, 64 sequences decoded together, 32 query heads on 8 of keys and values, 128 values a head) and
generic odd ones.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
BASE = 500000.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------- the cases


def _rope(name, mode, dtype, B, L, Hq, Hkv, d, rot, axes="", norm=True, weight=True, pairs="half", far=0):
    return dict(name=name, op="rope", mode=mode, dtype=dtype, B=B, L=L, Hq=Hq, Hkv=Hkv, d=d, rot=rot, axes=axes, norm=norm,
                weight=weight, pairs=pairs, far=far)


def _decay(name, mode, dtype, B, L, Hq, Hkv, dk, dv, lens="", carry=False):
    return dict(name=name, op="decay", mode=mode, dtype=dtype, B=B, L=L, Hq=Hq, Hkv=Hkv, dk=dk, dv=dv, lens=lens, carry=carry)


def listed():
    return [
        # one long prompt between the projections and the mixer
        _rope("rope_prompt", "prompt", "bf16", 1, 8192, 32, 8, 128, 128),
        # a training step, forward and gradients
        _rope("rope_train", "train", "bf16", 8, 2048, 32, 8, 128, 128),
        # one token for each of 64 sequences, far into their contexts
        _rope("rope_token", "prompt", "bf16", 64, 1, 32, 8, 128, 128, far=32768),
        # the patches of a clip, positions in time, height and width, part of a head rotated, no weights
        _rope("rope_clip", "prompt", "bf16", 2, 4097, 16, 16, 80, 64, axes="8,12,12", weight=False, pairs="neighbours"),
        # a numerics check of a small model: odd sizes, two axes, gradients
        _rope("rope_odd", "train", "f32", 3, 333, 6, 2, 72, 40, axes="7,13"),
        # one long prompt, the last state kept for decoding
        _decay("decay_prompt", "prompt", "bf16", 1, 8192, 32, 8, 128, 128),
        # a very long context: only the time axis grows
        _decay("decay_long", "prompt", "bf16", 1, 65536, 32, 8, 128, 128),
        # ragged prompts in one row (one empty, one of a single token) continuing earlier states
        _decay("decay_packed", "prompt", "bf16", 1, 8362, 32, 8, 128, 128, lens="1,2047,0,333,64,5000,17,900", carry=True),
        # a training step, forward and gradients, four query heads on each state
        _decay("decay_train", "train", "bf16", 8, 2048, 32, 8, 128, 128),
        # a training step with a state for every head, narrower keys than values
        _decay("decay_train_heads", "train", "bf16", 4, 4096, 16, 16, 64, 128),
        # a numerics check in fp32 on odd sizes, states and their gradients carried across the cut of a long text
        _decay("decay_odd", "train", "f32", 3, 777, 6, 2, 40, 72, carry=True),
        # one token for each of 64 sequences whose states sit in a cache of slots, some rows idle
        _decay("decay_step", "step", "bf16", 64, 1, 32, 8, 128, 128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, dtype = rng.choice(["rope", "decay", "decay"]), rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
    Hq = Hkv * rng.choice([g for g in (1, 1, 2, 3, 4, 4, 8) if g * Hkv <= 48])
    room = 16384 * 32 * 128 * 2 // SIZE[dtype]  # values of all query heads
    if op == "rope":
        d = rng.choice([32, 64, 72, 80, 96, 128, 128, 128, 256])
        rot = rng.choice([d, d, d, d // 2, 2 * rng.randint(1, d // 2)])
        n = min(rng.choice([1, 1, 1, 2, 3, 4]), rot // 2)
        cuts = sorted(rng.sample(range(1, rot // 2), n - 1))
        axes = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [rot // 2])) if n > 1 else ""
        B = rng.choice([1, 1, 2, 3, 8, 64])
        L = _log(rng, 1, max(1, min(65536, room // (B * Hq * d))))
        norm = rng.random() < 0.8
        c = _rope("", rng.choice(["prompt", "train"]), dtype, B, L, Hq, Hkv, d, rot, axes, norm, norm and rng.random() < 0.7,
                  rng.choice(["half", "half", "neighbours"]), rng.choice([0, 0, 4096, 1 << 20]))
    else:
        mode = rng.choice(["prompt", "prompt", "train", "train", "step"])
        dk, dv = rng.choice([32, 40, 64, 64, 80, 128, 128, 128, 33, 160]), rng.choice([32, 64, 72, 96, 128, 128, 128, 128, 57, 192])
        lens = ""
        if mode == "step":
            B, L = _log(rng, 1, 256), 1
        else:
            B = rng.choice([1, 1, 2, 3, 8])
            L = _log(rng, 1, max(1, min(65536, room // 2 // (B * Hq * max(dk, dv)))))
            if B > 1 and mode == "prompt":  # the same tokens as one packed batch with ragged lengths
                T = B * L
                cuts = sorted(rng.randrange(T + 1) for _ in range(B - 1))
                lens = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [T]))
                B, L = 1, T
        c = _decay("", mode, dtype, B, L, Hq, Hkv, dk, dv, lens, mode != "step" and rng.random() < 0.4)
    del c["name"]
    return c


# ------------------------------------------------------------------------------- the inputs


def _lens(case):
    return [int(v) for v in case["lens"].split(",")] if case["lens"] else []


def prepare(case, seed):
    gen = torch.Generator(DEVICE)
    gen.manual_seed(seed)
    tp, f32 = TYPES[case["dtype"]], torch.float32

    def normal(*shape, std=1.0, mean=0.0, dtype=None):
        t = torch.randn(shape, generator=gen, device=DEVICE, dtype=f32)
        return (t * std + mean).to(tp if dtype is None else dtype)

    B, L, Hq, Hkv = case["B"], case["L"], case["Hq"], case["Hkv"]
    s = dict(case=case)
    if case["op"] == "rope":
        d, half = case["d"], case["rot"] // 2
        s.update(q=normal(B, L, Hq, d), k=normal(B, L, Hkv, d))
        s["w_q"] = normal(d, std=0.1, mean=1.0, dtype=f32) if case["weight"] else None
        s["w_k"] = normal(d, std=0.1, mean=1.0, dtype=f32) if case["weight"] else None
        s["sections"] = [int(v) for v in case["axes"].split(",")] if case["axes"] else None
        place = torch.arange(half, device=DEVICE, dtype=torch.float64)
        s["freqs"] = (BASE ** (-place / half)).to(f32)
        s["positions"] = None  # the places 0 .. L - 1 of each row
        if case["axes"]:  # a grid's coordinates, one more axis each
            n, side = len(s["sections"]), max(1, int(round(L ** 0.5)))
            t = torch.arange(L, device=DEVICE)
            grid = torch.stack([t // side, t % side, t // (side * 4), t % 7], -1)[:, :n]
            s["positions"] = (grid[None] + case["far"]).expand(B, L, n).contiguous()
        elif case["far"]:
            first = torch.randint(case["far"] // 2, case["far"], (B, 1), generator=gen, device=DEVICE)
            s["positions"] = first + torch.arange(L, device=DEVICE)
        if case["mode"] == "train":
            s.update(dq_out=normal(B, L, Hq, d), dk_out=normal(B, L, Hkv, d))
        return s
    dk, dv = case["dk"], case["dv"]
    step = case["mode"] == "step"
    shape = (B,) if step else (B, L)
    lens = _lens(case)
    n = len(lens) or B
    s.update(q=normal(*shape, Hq, dk), k=normal(*shape, Hkv, dk), v=normal(*shape, Hkv, dv), scale=dk ** -0.5)
    # decays from 0.5 a token to 2^-12 less than one
    u = torch.rand(Hkv, generator=gen, device=DEVICE)
    s["log_decay"] = -torch.exp(u * math.log(0.7 * 4096) - math.log(4096.0))
    s["cu_seqlens"], s["slots"], s["s0"], s["s_out"] = None, None, None, None
    if lens:
        ends = torch.tensor(lens, dtype=torch.int64).cumsum(0)
        s["cu_seqlens"] = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(DEVICE)
    if step:  # each sequence's state sits in a slot of its own; a slot of -1 is an idle row
        nslots = B + B // 2 + 1
        order = torch.randperm(nslots, generator=gen, device=DEVICE)[:B]
        idle = torch.rand(B, generator=gen, device=DEVICE) < 0.05
        s["slots"] = torch.where(idle, torch.full_like(order, -1), order)
        s["state"] = normal(nslots, Hkv, dk, dv, dtype=f32)
        return s
    if case["carry"]:
        s["s0"] = normal(n, Hkv, dk, dv, dtype=f32)
    if case["mode"] == "prompt" or case["carry"]:
        s["s_out"] = torch.empty(n, Hkv, dk, dv, dtype=f32, device=DEVICE)
    if case["mode"] == "train":
        s["do"] = normal(*shape, Hq, dv)
        s["ds_out"] = normal(n, Hkv, dk, dv, dtype=f32) if case["carry"] else None
        s["ds0"] = torch.empty(n, Hkv, dk, dv, dtype=f32, device=DEVICE) if case["carry"] else None
    return s


# ------------------------------------------------------------------- the operators, plain form


def _angles(s):
    """Cosine and sine of each token's angles [B, L, 1, rot / 2]: products of far positions need 64 bits."""
    case, half = s["case"], s["case"]["rot"] // 2
    at = s["positions"]
    if at is None:
        at = torch.arange(case["L"], device=DEVICE).expand(case["B"], case["L"])
    if s["sections"] is None:
        at = at[..., None].expand(*at.shape, half)
    else:
        axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=DEVICE),
                                       torch.tensor(s["sections"], device=DEVICE), output_size=half)
        at = at[..., axis]
    a = (at.double() * s["freqs"].double())[:, :, None]
    return torch.cos(a).float(), torch.sin(a).float()


def _turn(n, cos, sin, case):
    """The first `rot` values of each head turned in pairs."""
    half = case["rot"] // 2
    if case["pairs"] == "half":
        n1, n2 = n[..., :half], n[..., half:2 * half]
        return torch.cat([n1 * cos - n2 * sin, n2 * cos + n1 * sin, n[..., 2 * half:]], -1)
    pair = n[..., :2 * half].unflatten(-1, (half, 2))
    n1, n2 = pair[..., 0], pair[..., 1]
    turned = torch.stack([n1 * cos - n2 * sin, n2 * cos + n1 * sin], -1).flatten(-2)
    return torch.cat([turned, n[..., 2 * half:]], -1)


def _rope_one(x, w, dy, cos, sin, case):
    xf = x.float()
    if not case["norm"]:
        y = _turn(xf, cos, sin, case)
        return y.to(x.dtype), None if dy is None else _turn(dy.float(), cos, -sin, case).to(x.dtype), None
    rs = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
    unit = xf * rs
    y = _turn(unit if w is None else unit * w, cos, sin, case).to(x.dtype)
    if dy is None:
        return y, None, None
    dn = _turn(dy.float(), cos, -sin, case)
    dw = None if w is None else (dn * unit).sum((0, 1, 2), dtype=torch.float64).float()
    du = dn if w is None else dn * w
    return y, (rs * (du - unit * (du * unit).mean(-1, keepdim=True))).to(x.dtype), dw


def _run_rope(s):
    case = s["case"]
    cos, sin = _angles(s)
    q, dq, dwq = _rope_one(s["q"], s["w_q"], s.get("dq_out"), cos, sin, case)
    k, dk, dwk = _rope_one(s["k"], s["w_k"], s.get("dk_out"), cos, sin, case)
    out = dict(q=q, k=k)
    if case["mode"] == "train":
        out.update(dq=dq, dk=dk)
        if case["weight"]:
            out.update(dw_q=dwq, dw_k=dwk)
    return out


def _recurrent(q, k, v, decay, first):
    """o[t] = q[t] S[t], S[t] = e^decay S[t-1] + k[t] v[t]^T in chunks: q, k [n, L, H, dk], v [n, L, H, dv],
    decay [H] in 64 bits, first [n, H, dk, dv] (e^decay times the state before the first token) or None.
    Returns o and the states behind chunks of C tokens, decayed up to the chunk's end."""
    n, L, H, _ = q.shape
    C = 128
    pad = -L % C
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, 0, 0, pad)).unflatten(1, (-1, C)).transpose(2, 3) for t in (q, k, v))
    N = (L + pad) // C  # [n, N, H, C, d]
    place = torch.arange(C, device=DEVICE)
    apart = (place[:, None] - place).clamp(min=0)
    mask = torch.where(place[:, None] >= place, torch.exp(decay[:, None, None] * apart), 0.0).float()
    o = (q @ k.transpose(-1, -2) * mask) @ v
    to_end = torch.exp(decay[:, None] * (C - 1 - place)).float()[..., None]
    own_part = (k * to_end).transpose(-1, -2) @ v  # [n, N, H, dk, dv]
    number = torch.arange(N, device=DEVICE)
    behind = number[:, None] - 1 - number
    carry = torch.where(behind >= 0, torch.exp(decay[:, None, None] * (C * behind.clamp(min=0))), 0.0).float()  # [H, N, N]
    before = torch.einsum("hab,nbhij->nahij", carry, own_part)  # S after the chunks before
    seen = torch.exp(decay[:, None] * (place + 1)).float()[..., None]
    o = o + (q * seen) @ before
    if first is not None:
        far = torch.exp(decay[None, :, None] * (number[:, None, None] * C + place)).float()  # [N, H, C]
        o = o + (q * far[..., None]) @ first[:, None]
    return o.transpose(2, 3).flatten(1, 2)[:, :L]


def _last_state(k, v, decay, lens, shift):
    """sum over t < len of e^(decay (len - 1 - t + shift)) k[t] v[t]^T for each sequence."""
    L = k.shape[1]
    left = lens[:, None] - 1 - torch.arange(L, device=DEVICE)
    w = torch.where(left[..., None] >= 0, torch.exp(decay * (left.clamp(min=0)[..., None] + shift)), 0.0).float()
    kw = k * w[..., None]
    return torch.einsum("nlhi,nlhj->nhij", kw, v)


def _run_decay(s):
    case, scale = s["case"], s["scale"]
    Hkv, G = case["Hkv"], case["Hq"] // case["Hkv"]
    decay = s["log_decay"].double()
    if case["mode"] == "step":
        live = (s["slots"] >= 0)[:, None, None, None]
        slot = s["slots"].clamp(min=0)
        S = s["state"][slot] * torch.exp(s["log_decay"])[:, None, None] + s["k"].float()[..., None] * s["v"].float()[..., None, :]
        q = s["q"].float().unflatten(1, (Hkv, G)) * scale
        o = torch.where(live, q @ S, 0.0).flatten(1, 2)
        spare = torch.cat([s["state"], s["state"][:1]])  # rows that are idle write to a slot that is thrown away
        spare[torch.where(live[:, 0, 0, 0], slot, len(s["state"]))] = S
        s["state"].copy_(spare[:-1])
        return dict(o=o.to(s["q"].dtype), state=s["state"])
    tp = s["q"].dtype
    q, k, v = s["q"].float() * scale, s["k"].float(), s["v"].float()
    B, L = q.shape[:2]
    lens = torch.full((B,), L, device=DEVICE)
    rows = None
    if s["cu_seqlens"] is not None:  # one row of sequences as a padded batch
        lens = s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]
        at = torch.arange(max(1, max(_lens(case))), device=DEVICE)
        valid = at < lens[:, None]
        rows = torch.where(valid, s["cu_seqlens"][:-1, None] + at, L).clamp(max=L)
        q, k, v = (torch.cat([t[0], torch.zeros_like(t[0, :1])])[rows] for t in (q, k, v))
    kk, vv = (t.repeat_interleave(G, 2) for t in (k, v))
    dd = decay.repeat_interleave(G)
    first = None if s["s0"] is None else s["s0"] * torch.exp(decay).float()[:, None, None]
    o = _recurrent(q, kk, vv, dd, None if first is None else first.repeat_interleave(G, 1))
    if rows is None:
        out = dict(o=o.to(tp))
    else:
        whole = torch.empty(1, L + 1, *o.shape[2:], device=DEVICE)
        whole[0, rows] = o
        out = dict(o=whole[:, :L].to(tp))
    if s["s_out"] is not None:
        last = _last_state(k, v, decay, lens, 0)
        if s["s0"] is not None:
            last = last + s["s0"] * torch.exp(decay * lens[:, None]).float()[..., None, None]
        s["s_out"].copy_(last)
        out["s_out"] = s["s_out"]
    if case["mode"] == "train":
        do = s["do"].float()
        # the gradients are the operator itself, backwards in time for keys and values
        s0t = None if first is None else first.repeat_interleave(G, 1).transpose(-1, -2)
        out["dq"] = (_recurrent(do, vv, kk, dd, s0t) * scale).to(tp)
        back = None if s["ds_out"] is None else s["ds_out"].repeat_interleave(G, 1) / G
        qf, kf, vf, df = (t.flip(1) for t in (q, kk, vv, do))
        dv = _recurrent(kf, qf, df, dd, back).flip(1)
        dk = _recurrent(vf, df, qf, dd, None if back is None else back.transpose(-1, -2)).flip(1)
        out["dk"] = dk.unflatten(2, (Hkv, G)).sum(3).to(tp)
        out["dv"] = dv.unflatten(2, (Hkv, G)).sum(3).to(tp)
        if s["ds0"] is not None:
            ds = _last_state(qf, df, dd, lens, 1).unflatten(1, (Hkv, G)).sum(2)
            s["ds0"].copy_(ds + s["ds_out"] * torch.exp(decay * lens[:, None]).float()[..., None, None])
            out["ds0"] = s["ds0"]
    return out


# ---------------------------------------------------------- the same through the library's calls


def _own_rope(s):
    from gated_linear_sliding_gb300 import lizard as lz

    case = s["case"]
    how = dict(positions=s["positions"], sections=s["sections"], w_q=s["w_q"], w_k=s["w_k"], norm=case["norm"], eps=EPS,
               neighbours=case["pairs"] == "neighbours")
    q, k = lz.lizard_qk_rope_fwd(s["q"], s["k"], s["freqs"], **how)
    out = dict(q=q, k=k)
    if case["mode"] == "train":
        g = lz.lizard_qk_rope_bwd(s["q"], s["k"], s["freqs"], s["dq_out"], s["dk_out"], **how)
        out.update(dq=g["dq"], dk=g["dk"])
        if case["weight"]:
            out.update(dw_q=g["dw_q"], dw_k=g["dw_k"])
    return out


def _own_decay(s):
    from gated_linear_sliding_gb300 import lizard as lz

    case = s["case"]
    args = (s["q"], s["k"], s["v"], s["log_decay"])
    if case["mode"] == "step":
        o = lz.lizard_decay_attn_step(*args, s["state"], slots=s["slots"], scale=s["scale"])
        return dict(o=o, state=s["state"])
    o = lz.lizard_decay_attn_fwd(*args, scale=s["scale"], s0=s["s0"], s_out=s["s_out"], cu_seqlens=s["cu_seqlens"])
    out = dict(o=o)
    if s["s_out"] is not None:
        out["s_out"] = s["s_out"]
    if case["mode"] == "train":
        g = lz.lizard_decay_attn_bwd(*args, s["do"], scale=s["scale"], s0=s["s0"], ds_out=s["ds_out"], ds0=s["ds0"])
        out.update(dq=g["dq"], dk=g["dk"], dv=g["dv"])
        if s["ds0"] is not None:
            out["ds0"] = s["ds0"]
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "decay": _own_decay}[op](state)
    return {"rope": _run_rope, "decay": _run_decay}[op](state)


# --------------------------------------------------------------------------------- the bounds


def work(case):
    e = SIZE[case["dtype"]]
    rows, Hq, Hkv = case["B"] * case["L"], case["Hq"], case["Hkv"]
    train = case["mode"] == "train"
    if case["op"] == "rope":
        values = rows * (Hq + Hkv) * case["d"]
        axes = len(case["axes"].split(",")) if case["axes"] else 1
        at = 8 * rows * axes if case["axes"] or case["far"] else 0
        return {"bytes": values * e * (5 if train else 2) + at, "flops": values * (22 if train else 8)}
    dk, dv = case["dk"], case["dv"]
    lens = _lens(case)
    states = (len(lens) or case["B"]) * Hkv * dk * dv * 4
    # the recurrence in chunks of 64 tokens: the pairs in a chunk, then the state's part and its update
    flops = rows * (Hq * (2 * dk * dv + 64 * (dk + dv)) + Hkv * 2 * dk * dv)
    nbytes = rows * (Hq + Hkv) * (dk + dv) * e
    if case["mode"] == "step":
        live = 2 * states
        return {"bytes": nbytes + live, "flops": rows * (Hq * 2 * dk * dv + Hkv * 3 * dk * dv)}
    nbytes += states * ((1 if case["carry"] else 0) + (1 if not train or case["carry"] else 0))
    if train:
        nbytes += rows * (Hq * (2 * dk + dv) + 2 * Hkv * (dk + dv)) * e + (3 * states if case["carry"] else 0)
        flops += rows * (Hq * (4 * dk * dv + 64 * 3 * (dk + dv)) + Hkv * 6 * dk * dv)
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------- the definitions, in 64 bits


def _exact_rope(s):
    """Each pair as one complex number, turned by multiplication; the gradient by the chain rule."""
    case, rot = s["case"], s["case"]["rot"]
    B, L = case["B"], case["L"]
    at = s["positions"] if s["positions"] is not None else torch.arange(L, device=DEVICE).repeat(B, 1)
    at = at.double().reshape(B, L, -1)
    sizes = s["sections"] or [rot // 2]
    freqs = s["freqs"].double().split(sizes)
    a = torch.cat([at[..., i:i + 1] * f for i, f in enumerate(freqs)], -1)[:, :, None]
    z = torch.polar(torch.ones_like(a), a)

    def turn(n, z):
        if case["pairs"] == "half":
            c = torch.complex(n[..., :rot // 2], n[..., rot // 2:rot]) * z
            return torch.cat([c.real, c.imag, n[..., rot:]], -1)
        c = torch.view_as_complex(n[..., :rot].reshape(*n.shape[:-1], rot // 2, 2).contiguous()) * z
        return torch.cat([torch.view_as_real(c).reshape(*n.shape[:-1], rot), n[..., rot:]], -1)

    out, grads, sums = {}, {}, {}
    for name in ("q", "k"):
        x, w = s[name].double(), s["w_" + name]
        w = 1.0 if w is None else w.double()
        d = x.shape[-1]
        root = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) if case["norm"] else torch.ones_like(x[..., :1])
        out[name] = turn(x / root * w, z)
        if case["mode"] == "train":
            dn = turn(s["d" + name + "_out"].double(), z.conj())
            dx = dn * w / root
            if case["norm"]:
                dx = dx - x * ((dn * w * x).sum(-1, keepdim=True) / d) / root ** 3
            grads["d" + name] = dx
            if case["weight"]:
                sums["dw_" + name] = (dn * x / root).sum((0, 1, 2))
    return {**out, **grads, **sums}


def _exact_decay(s):
    case, scale = s["case"], s["scale"]
    Hkv, G, dk, dv = case["Hkv"], case["Hq"] // case["Hkv"], case["dk"], case["dv"]
    keep = torch.exp(s["log_decay"].double())[:, None, None]

    def heads(t):  # [..., Hq, d] as [..., Hkv, G, d]
        return t.unflatten(-2, (Hkv, G))

    if case["mode"] == "step":
        state = s["state"].double()
        o = torch.zeros(*s["q"].shape[:2], dv, dtype=torch.float64, device=DEVICE)
        for b, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                S = keep * state[slot] + s["k"][b].double()[..., None] * s["v"][b].double()[:, None]
                o[b] = (scale * heads(s["q"][b].double()) @ S).flatten(0, 1)
                state[slot] = S
        return dict(o=o, state=state)
    train = case["mode"] == "train"
    B, L = s["q"].shape[:2]
    o = torch.zeros(B, L, case["Hq"], dv, dtype=torch.float64, device=DEVICE)
    zero = torch.zeros(B, Hkv, dk, dv, dtype=torch.float64, device=DEVICE)
    cu = s["cu_seqlens"].tolist() if s["cu_seqlens"] is not None else [0, L]
    packed = s["cu_seqlens"] is not None
    ends, starts = [], []
    dq, dkey, dval = (torch.zeros(t.shape, dtype=torch.float64, device=DEVICE) for t in (s["q"], s["k"], s["v"]))
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        pick = slice(i, i + 1) if packed else slice(None)
        S = zero if s["s0"] is None else s["s0"][pick].double()
        for a in range(lo, hi, 512):  # a block of tokens in 64 bits at a time
            b = min(hi, a + 512)
            q, k, v = heads(s["q"][:, a:b].double()), s["k"][:, a:b].double(), s["v"][:, a:b].double()
            do = heads(s["do"][:, a:b].double()) if train else None
            for t in range(b - a):
                S = keep * S + k[:, t, :, :, None] * v[:, t, :, None]
                o[:, a + t] = (scale * q[:, t] @ S).flatten(1, 2)
                if train:
                    dq[:, a + t] = (scale * do[:, t] @ S.transpose(-1, -2)).flatten(1, 2)
        ends.append(S)
        if not train:
            continue
        D = zero if s["ds_out"] is None else s["ds_out"][pick].double()
        for b in range(hi, lo, -512):
            a = max(lo, b - 512)
            q, k, v = heads(s["q"][:, a:b].double()), s["k"][:, a:b].double(), s["v"][:, a:b].double()
            do = heads(s["do"][:, a:b].double())
            for t in range(b - a - 1, -1, -1):
                D = D + scale * q[:, t].transpose(-1, -2) @ do[:, t]
                dkey[:, a + t] = (D @ v[:, t, :, :, None])[..., 0]
                dval[:, a + t] = (k[:, t, :, None] @ D)[:, :, 0]
                D = keep * D
        starts.append(D)
    out = dict(o=o)
    if s["s_out"] is not None:
        out["s_out"] = torch.cat(ends)
    if train:
        out.update(dq=dq, dk=dkey, dv=dval)
        if s["ds0"] is not None:
            out["ds0"] = torch.cat(starts)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "decay": _exact_decay}[case["op"]](s)
