"""The selective state space block on the GPU against its float64 definitions.

Tolerances.  Every output is an fp32 sum rounded once to its type: its error is at most half a
step of the type (eps / 2 relative to the value) plus n roundings of fp32 (2^-24 each) relative to
the sum of its terms' magnitudes, which the definitions give with absolute=True.  n counts the
roundings a term can pass: at most 16 a token of the recurrence (step size, exponent, exponential
of two ulps, product and sum), two for each term of a sum over channels or tokens, and 64 for the
rest (softplus, sigmoid, gate).
"""
import numpy as np
import pytest

from oracle import selective as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def lz():
    from gated_linear_sliding_gb300 import lizard

    lizard.load()
    return lizard


def tdt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


class Draw:
    """Seeded inputs: the device tensor and the same (rounded) values in float64."""

    def __init__(self, seed, dtype):
        self.rng, self.dtype = np.random.default_rng(seed), tdt(dtype)

    def __call__(self, *shape, dtype=None, scale=1.0, shift=0.0, stride=0, at=0):
        a = (self.rng.normal(size=shape) * scale + shift).astype(np.float32)
        return self.dev(a, dtype or self.dtype, stride, at)

    def dev(self, a, dtype=torch.float32, stride=0, at=0):
        t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda", dtype)
        v = t.double().cpu().numpy()
        if stride:  # columns [at, at + width) of rows of `stride` elements
            wide = torch.full(t.shape[:2] + (stride,), 77.0, dtype=dtype, device="cuda")
            flat = wide[..., at:at + int(np.prod(t.shape[2:]))]
            flat.copy_(t.reshape(flat.shape))
            t = flat.unflatten(-1, t.shape[2:]) if t.dim() > 3 else flat
        return t, v


def check(got, ref, mag, n, what):
    got_t = got
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: not finite"
    half = torch.finfo(got_t.dtype).eps / 2
    arith = n * U32 * mag
    tol = half * (np.abs(ref) + arith) + arith + 1e-37
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (what, int(bad.sum()), got.size, float((np.abs(got - ref) / tol).max()))


def seqs(L, B, lens):
    """(row, first token, end) of each sequence."""
    if lens is None:
        return [(b, 0, L) for b in range(B)]
    ends = np.cumsum(lens)
    return [(0, int(e - n), int(e)) for n, e in zip(lens, ends)]


def offsets(lens):
    return None if lens is None else torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64, device="cuda")


# ------------------------------------------------------------------------------ convolution

CONV = [  # B, L, C, K, lens, column stride (0: dense)
    (1, 1, 8, 4, None, 0),
    (2, 2, 16, 4, None, 0),
    (3, 37, 40, 3, None, 0),
    (1, 100, 37, 4, None, 0),
    (2, 70, 24, 4, None, 64),
    (1, 65, 13, 2, None, 29),
    (1, 33, 8, 8, None, 0),
    (2, 9, 8, 1, None, 0),
    (1, 150, 64, 4, [0, 1, 2, 0, 64, 3, 80, 0], 0),
    (1, 40, 19, 8, [5, 1, 6, 28], 0),
    (1, 0, 16, 4, [0, 0], 0),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("case", range(len(CONV)))
@pytest.mark.parametrize("state", [False, True])
def test_conv(lz, dtype, act, case, state):
    B, L, C, K, lens, stride = CONV[case]
    d = Draw(case, dtype)
    x, xv = d(B, L, C, stride=stride, at=8 if stride % 8 == 0 else 0)
    w, wv = d(C, K, dtype=torch.float32)
    b, bv = d(C, dtype=torch.float32) if act else (None, np.zeros(C))
    n = B if lens is None else len(lens)
    st, sv = d(n, K - 1, C) if state else (None, np.zeros((n, K - 1, C)))
    dy, dyv = d(B, L, C, stride=stride)
    ds, dsv = d(n, K - 1, C) if state else (None, np.zeros((n, K - 1, C)))
    cu = offsets(lens)
    out = torch.full((n, K - 1, C), 9.0, dtype=x.dtype, device="cuda")
    y = lz.lizard_conv_fwd(x, w, b, act=act, state_in=st, state_out=out, cu_seqlens=cu)
    din = torch.full((n, K - 1, C), 9.0, dtype=x.dtype, device="cuda") if state else None
    g = lz.lizard_conv_bwd(x, w, b, dy, act=act, state_in=st, dstate_out=ds, dstate_in=din, cu_seqlens=cu)
    torch.cuda.synchronize()
    dw, dwm, db, dbm = (np.zeros(s) for s in ((C, K), (C, K), C, C))
    N = 64 + 2 * K
    for i, (row, lo, hi) in enumerate(seqs(L, B, lens)):
        a = (xv[row, lo:hi], wv, bv, sv[i], bool(act))
        ry, rs, _ = S.conv_fwd(*a)
        my, _, mp = S.conv_fwd(*a, absolute=True)
        check(y[row, lo:hi], ry, my, N, f"y {i}")
        assert np.array_equal(out[i].double().cpu().numpy(), rs), f"state {i}"
        r = S.conv_bwd(*a, dyv[row, lo:hi], dsv[i])
        m = S.conv_bwd(*a, dyv[row, lo:hi], dsv[i], absolute=True)
        # act' is a function of the pre-activation, whose own error counts by |act''| < 1
        soft = (np.abs(dyv[row, lo:hi]) * (1 + mp)).max(initial=0) if act else 0
        wide = m[0] + soft * np.abs(wv).sum(1)
        check(g["dx"][row, lo:hi], r[0], wide, N, f"dx {i}")
        if state:
            check(g["dstate_in"][i], r[3], m[3] + soft * np.abs(wv).sum(1), N, f"dstate_in {i}")
        dw, dwm = dw + r[1], dwm + m[1] + soft * np.abs(xv).max(initial=0) * (hi - lo + 1)
        db, dbm = db + r[2], dbm + m[2] + soft * (hi - lo + 1)
    check(g["dw"], dw, dwm + 1e-30, N + 2 * B * L, "dw")
    if b is not None:
        check(g["dbias"], db, dbm + 1e-30, N + 2 * B * L, "dbias")


def test_conv_state_in_place_and_steps(lz):
    """A prompt in two calls and single tokens, the state passed on in place, give the one call's
    outputs bit for bit."""
    d = Draw(3, "bf16")
    B, L, C, K = 3, 21, 40, 4
    x, _ = d(B, L, C)
    w, _ = d(C, K, dtype=torch.float32)
    b, _ = d(C, dtype=torch.float32)
    whole = lz.lizard_conv_fwd(x, w, b, act=1)
    st = torch.zeros(B, K - 1, C, dtype=x.dtype, device="cuda")
    parts = []
    for lo, hi in ((0, 2), (2, 15)):
        parts.append(lz.lizard_conv_fwd(x[:, lo:hi].contiguous(), w, b, act=1, state_in=st, state_out=st))
    cache = torch.full((7, K - 1, C), 5.0, dtype=x.dtype, device="cuda")
    slots = torch.tensor([4, 0, 6], dtype=torch.int64, device="cuda")
    cache[slots] = st
    keep = cache.clone()
    for t in range(15, L):
        parts.append(lz.lizard_conv_step(x[:, t], w, b, cache, slots=slots, act=1)[:, None])
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(parts, 1), whole)
    assert torch.equal(cache[slots], x[:, L - K + 1:])
    others = [1, 2, 3, 5]
    assert torch.equal(cache[others], keep[others])


# ------------------------------------------------------------------------------------- scan

SCAN = [  # B, L, C, N, G, lens, softplus, gate, strided
    (1, 1, 8, 16, 1, None, True, True, False),
    (2, 5, 8, 4, 1, None, True, False, False),
    (2, 33, 40, 16, 1, None, True, True, True),
    (1, 64, 37, 16, 1, None, True, True, False),
    (1, 70, 24, 24, 4, None, True, True, False),
    (1, 50, 6, 64, 3, None, False, True, False),
    (1, 47, 130, 1, 2, None, True, True, False),
    (2, 40, 72, 3, 1, None, True, False, False),
    (1, 55, 16, 8, 2, None, True, True, True),
    (1, 50, 20, 7, 1, None, True, True, True),
    (1, 300, 16, 16, 1, None, True, True, False),
    (2, 323, 9, 5, 3, None, False, False, False),
    (1, 403, 16, 16, 1, [0, 1, 15, 48, 2, 0, 64, 200, 73, 0], True, True, False),
    (1, 90, 10, 16, 2, [3, 1, 1, 20, 7, 58], True, True, False),
    (1, 600, 8, 4, 1, [64, 64, 128, 1, 343], True, False, False),
    (1, 0, 16, 16, 1, [0, 0, 0], True, True, False),
]


def scan_inputs(case, dtype, seed=0):
    B, L, C, N, G, lens, sp, gate, strided = SCAN[case]
    d = Draw(case + 100 * seed, dtype)
    s = dict(stride=2 * C + 24) if strided else {}
    sb = dict(stride=2 * G * N + 8) if strided else {}
    n = B if lens is None else len(lens)
    v = dict(x=d(B, L, C, **s), dt=d(B, L, C, scale=0.7 if sp else 0.1, shift=-1.0 if sp else 0.4, **s),
             A=d.dev(-np.exp(d.rng.normal(size=(C, N)))), Bm=d(B, L, G, N, **sb), Cm=d(B, L, G, N, **sb),
             D=d(C, dtype=torch.float32), z=d(B, L, C, **s) if gate else (None, None),
             dt_bias=d(C, dtype=torch.float32, scale=0.3 if sp else 0.02),
             h0=d(n, C, N, dtype=torch.float32), dy=d(B, L, C, **s), dh=d(n, C, N, dtype=torch.float32))
    return v, n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("case", range(len(SCAN)))
def test_scan(lz, dtype, state, case):
    B, L, C, N, G, lens, sp, gate, _ = SCAN[case]
    v, n = scan_inputs(case, dtype)
    t = {k: a[0] for k, a in v.items()}
    r64 = {k: a[1] for k, a in v.items()}
    if not state:
        t["h0"] = t["dh"] = None
        r64["h0"], r64["dh"] = np.zeros((n, C, N)), np.zeros((n, C, N))
    cu = offsets(lens)
    args = (t["x"], t["dt"], t["A"], t["Bm"], t["Cm"])
    how = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], softplus=sp, h0=t["h0"], cu_seqlens=cu)
    h_out = torch.full((n, C, N), 9.0, device="cuda")
    y, states = lz.lizard_scan_fwd(*args, **how, h_out=h_out, save_states=True)
    dh0 = torch.full((n, C, N), 9.0, device="cuda") if state else None
    g = lz.lizard_scan_bwd(*args, t["dy"], states, **how, dh_out=t["dh"], dh0=dh0)
    plain = lz.lizard_scan_fwd(*args, **how)
    torch.cuda.synchronize()
    assert torch.equal(plain, y)
    tot = {k: 0.0 for k in ("dA", "dD", "ddt_bias")}
    mag = dict(tot)
    for i, (row, lo, hi) in enumerate(seqs(L, B, lens)):
        cut = lambda k: None if r64[k] is None else r64[k][row, lo:hi]  # noqa: E731
        a = (cut("x"), cut("dt"), r64["A"], cut("Bm"), cut("Cm"), r64["D"], cut("z"), r64["dt_bias"], r64["h0"][i])
        cnt = 16 * (hi - lo) + 64 + N
        ry, rh = S.scan_fwd(*a, use_softplus=sp)
        my, mh = S.scan_fwd(*a, use_softplus=sp, absolute=True)
        check(y[row, lo:hi], ry, my, cnt, f"y {i}")
        check(h_out[i], rh[-1], mh[-1], cnt, f"h {i}")
        r = S.scan_bwd(*a, cut("dy"), r64["dh"][i], use_softplus=sp)
        m = S.scan_bwd(*a, cut("dy"), r64["dh"][i], use_softplus=sp, absolute=True)
        cnt = 32 * (hi - lo) + 128 + N + 2 * C
        for k, gk in (("dx", "dx"), ("ddt", "ddt"), ("dz", "dz"), ("dB", "dBm"), ("dC", "dCm")):
            if r[k] is not None:
                check(g[gk][row, lo:hi], r[k], m[k], cnt, f"{gk} {i}")
        if state:
            check(dh0[i], r["dh0"], m["dh0"], cnt, f"dh0 {i}")
        for k in tot:
            tot[k], mag[k] = tot[k] + r[k], mag[k] + m[k]
    cnt = 32 * L + 128 + N + 2 * B * L
    for k in tot:
        check(g[k], tot[k], mag[k] + 1e-30, cnt, k)
    if not gate:
        assert g["dz"] is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [0, 2, 4, 5, 6, 8, 9])
def test_scan_step(lz, dtype, case):
    """A prompt's state, then single tokens through slots, equal the whole sequence's definition;
    idle rows give zeros and touch nothing, whatever their inputs hold."""
    B, L, C, N, G, _, sp, gate, _ = SCAN[case]
    v, _ = scan_inputs(case, dtype, seed=1)
    t = {k: a[0] for k, a in v.items()}
    r64 = {k: a[1] for k, a in v.items()}
    cut = max(0, L - 4)
    nslots = B + 3
    slots = torch.tensor([(2 * b + 1) % nslots for b in range(B)] + [-1], dtype=torch.int64, device="cuda")
    cache = torch.full((nslots, C, N), float("nan"), device="cuda")
    state = t["h0"].clone()
    if cut:
        pre = {k: (a[:, :cut] if k in ("x", "dt", "Bm", "Cm", "z") and a is not None else a) for k, a in t.items()}
        pre = {k: (a.contiguous() if a is not None else None) for k, a in pre.items()}
        lz.lizard_scan_fwd(pre["x"], pre["dt"], t["A"], pre["Bm"], pre["Cm"], D=t["D"], z=pre["z"], dt_bias=t["dt_bias"],
                           softplus=sp, h0=state, h_out=state)
    cache[slots[:B]] = state
    ys = []
    for k in range(cut, L):
        row = {}
        for name in ("x", "dt", "Bm", "Cm", "z"):
            if t[name] is not None:
                a = t[name][:, k]
                row[name] = torch.cat([a, torch.full_like(a[:1], float("nan"))])  # an idle row of NaN
            else:
                row[name] = None
        y = lz.lizard_scan_step(row["x"], row["dt"], t["A"], row["Bm"], row["Cm"], cache, D=t["D"], z=row["z"],
                                dt_bias=t["dt_bias"], softplus=sp, slots=slots)
        ys.append(y)
    torch.cuda.synchronize()
    got = torch.stack(ys, 1)
    assert (got[B] == 0).all()
    used = set(slots[:B].tolist())
    for s in range(nslots):
        if s not in used:
            assert torch.isnan(cache[s]).all()
    for b in range(B):
        a = (r64["x"][b], r64["dt"][b], r64["A"], r64["Bm"][b], r64["Cm"][b], r64["D"],
             None if r64["z"] is None else r64["z"][b], r64["dt_bias"], r64["h0"][b])
        ry, rh = S.scan_fwd(*a, use_softplus=sp)
        my, mh = S.scan_fwd(*a, use_softplus=sp, absolute=True)
        cnt = 16 * L + 64 + N
        check(got[b], ry[cut:], my[cut:], cnt, f"y {b}")
        check(cache[slots[b]], rh[-1], mh[-1], cnt, f"state {b}")


def test_scan_extremes(lz):
    """Decays that underflow, rates of zero, step sizes far out on both sides of softplus."""
    B, L, C, N = 1, 40, 16, 16
    d = Draw(5, "f32")
    x, xv = d(B, L, C)
    dt, dtv = d(B, L, C, scale=40.0)  # softplus from e^-100 to 100
    a = -np.exp(d.rng.normal(size=(C, N)) * 3)
    a[:, 0] = 0.0
    a[:, 1] = -1e4
    A, Av = d.dev(a)
    Bm, Bv = d(B, L, 1, N)
    Cm, Cv = d(B, L, 1, N)
    dy, dyv = d(B, L, C)
    y, st = lz.lizard_scan_fwd(x, dt, A, Bm, Cm, save_states=True)
    g = lz.lizard_scan_bwd(x, dt, A, Bm, Cm, dy, st)
    torch.cuda.synchronize()
    zero = np.zeros(C)
    args = (xv[0], dtv[0], Av, Bv[0], Cv[0], zero, None, zero, np.zeros((C, N)))
    ry, _ = S.scan_fwd(*args)
    my, _ = S.scan_fwd(*args, absolute=True)
    cnt = 16 * L + 64 + N
    check(y[0], ry, my, cnt, "y")
    r = S.scan_bwd(*args, dyv[0], np.zeros((C, N)))
    m = S.scan_bwd(*args, dyv[0], np.zeros((C, N)), absolute=True)
    # an exponent of size E is rounded by E 2^-24: the decay e^-E is off by E e^-E <= 0.37
    cnt = 32 * L + 128 + N + 2 * C
    for k, gk in (("dx", "dx"), ("dB", "dBm"), ("dC", "dCm")):
        check(g[gk][0], r[k], m[k], cnt, gk)
    check(g["ddt"][0], r["ddt"], m["ddt"], cnt, "ddt")
    check(g["dA"], r["dA"], m["dA"] + 1e-30, cnt + 2 * L, "dA")


@pytest.mark.parametrize("lens", [[40, 60], [300, 64, 200]])
def test_scan_sequences_do_not_leak(lz, lens):
    """A sequence of NaN in a packed batch leaves the others' results as they are alone."""
    L, C, N = sum(lens), 16, 16
    d = Draw(8, "bf16")
    t = {k: d(1, L, *s)[0] for k, s in (("x", (C,)), ("dt", (C,)), ("Bm", (1, N)), ("Cm", (1, N)), ("z", (C,)), ("dy", (C,)))}
    A = d.dev(-np.exp(d.rng.normal(size=(C, N))))[0]
    clean = {k: a.clone() for k, a in t.items()}
    bad = 0
    lo, hi = sum(lens[:bad]), sum(lens[:bad + 1])
    for k in t:
        t[k][:, lo:hi] = float("nan")
    cu = offsets(lens)

    def both(v):
        y, st = lz.lizard_scan_fwd(v["x"], v["dt"], A, v["Bm"], v["Cm"], z=v["z"], cu_seqlens=cu, save_states=True)
        g = lz.lizard_scan_bwd(v["x"], v["dt"], A, v["Bm"], v["Cm"], v["dy"], st, z=v["z"], cu_seqlens=cu)
        return dict(y=y, **{k: g[k] for k in ("dx", "ddt", "dz", "dBm", "dCm")})

    got, ref = both(t), both(clean)
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(got[k][:, hi:], ref[k][:, hi:]), k
        assert torch.isnan(got[k][:, lo:hi]).any(), k


def test_scan_in_place_state_over_segments(lz):
    """h_out may be h0 although the time axis is walked by several CTAs at once."""
    v, n = scan_inputs(12, "f32")
    t = {k: a[0] for k, a in v.items()}
    lens = SCAN[12][5]
    cu = offsets(lens)
    how = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], cu_seqlens=cu)
    h = torch.empty_like(t["h0"])
    y = lz.lizard_scan_fwd(t["x"], t["dt"], t["A"], t["Bm"], t["Cm"], h0=t["h0"], h_out=h, **how)
    st = t["h0"].clone()
    y2 = lz.lizard_scan_fwd(t["x"], t["dt"], t["A"], t["Bm"], t["Cm"], h0=st, h_out=st, **how)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, st)


def test_bad_offsets_and_slots_are_reported(lz):
    """Inconsistent device offsets and a slot past the cache record INVALID_ARG; nothing outside
    the buffers is touched and the other rows are computed."""
    d = Draw(9, "f32")
    L, C, N = 80, 8, 4
    x, dt, z = (d(1, L, C)[0] for _ in range(3))
    Bm, Cm = (d(1, L, 1, N)[0] for _ in range(2))
    A = -torch.ones(C, N, device="cuda")
    w = torch.ones(C, 4, device="cuda")
    for offs in ([0, 50, 40, 80], [0, -5, 20, 80], [0, 30, 999, 80], [7, 30, 50, 80], [0, 10, 20, 60]):
        cu = torch.tensor(offs, dtype=torch.int64, device="cuda")
        h = torch.zeros(5, C, N, device="cuda")
        ws = lz.new_workspace(1 << 20, "cuda")
        y = torch.zeros(1, L + 8, C, device="cuda")
        lz.lizard_scan_fwd(x, dt, A, Bm, Cm, cu_seqlens=cu, y=y[:, :L], h_out=h[:3], workspace=ws)
        assert lz.lizard_read_device_status(ws) == lz.LIZARD_ERR_INVALID_ARG, offs
        assert (y[:, L:] == 0).all() and (h[3:] == 0).all()
        ws = lz.new_workspace(256, "cuda")
        lz.lizard_conv_fwd(x, w, None, cu_seqlens=cu, y=y[:, :L], workspace=ws)
        assert lz.lizard_read_device_status(ws) == lz.LIZARD_ERR_INVALID_ARG, offs
        assert (y[:, L:] == 0).all()
    ws = lz.new_workspace(256, "cuda")
    cache = torch.zeros(3, C, N, device="cuda")
    slots = torch.tensor([1, 3], dtype=torch.int64, device="cuda")
    y = lz.lizard_scan_step(x[0, :2], dt[0, :2], A, Bm[0, :2], Cm[0, :2], cache[:3], slots=slots, workspace=ws)
    assert lz.lizard_read_device_status(ws) == lz.LIZARD_ERR_INVALID_ARG
    assert (y[1] == 0).all() and (cache[1] != 0).any() and (cache[[0, 2]] == 0).all()
    cs = torch.zeros(3, 3, C, device="cuda")
    lz.lizard_conv_step(x[0, :2], w, None, cs, slots=slots, workspace=ws)
    assert lz.lizard_read_device_status(ws) == lz.LIZARD_ERR_INVALID_ARG
    assert (cs[1] != 0).any() and (cs[[0, 2]] == 0).all()


# ------------------------------------------------------------------------------------- norm

NORM = [  # T, D, groups, gate ("", first, last), act, post, scale, pre, residual ("", same, f32), stride
    (1, 8, 1, "", "silu", True, True, True, "same", 0),
    (5, 37, 1, "last", "silu", True, True, True, "same", 0),
    (7, 64, 4, "first", "silu", True, False, False, "", 0),
    (3, 96, 3, "last", "sigmoid", True, True, True, "f32", 0),
    (9, 40, 5, "first", "sigmoid", True, True, True, "f32", 104),
    (4, 30, 6, "last", "silu", True, False, True, "same", 61),
    (2, 1000, 1, "", "silu", False, False, True, "same", 0),
    (3, 1536, 12, "last", "silu", True, True, True, "f32", 0),
    (2, 2304, 2, "first", "silu", True, True, True, "same", 0),
    (1300, 16, 1, "last", "silu", True, True, True, "same", 0),
    (2, 8200, 1, "last", "silu", True, True, True, "same", 0),
    (2, 16384, 8, "", "silu", True, True, True, "f32", 0),
    (2, 9001, 1, "first", "silu", True, True, True, "f32", 0),
    (2, 1040, 8, "last", "silu", True, True, True, "same", 0),
    (6, 24, 1, "last", "silu", False, True, False, "same", 0),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(NORM)))
def test_block_norm(lz, dtype, case):
    T, D, groups, gate, act, post, scale, pre, res, stride = NORM[case]
    d = Draw(case, dtype)
    rtp = {"": tdt(dtype), "same": tdt(dtype), "f32": torch.float32}[res]

    def rows(dtype=None):
        t, v = d(1, T, D, dtype=dtype, stride=stride)
        return t[0], v[0]

    none = (None, None)
    vec = lambda on: d(D, dtype=torch.float32, scale=0.3, shift=1.0) if on else none  # noqa: E731
    v = dict(o=rows(), gate=rows() if gate else none, r=rows(rtp) if res else none, w_post=vec(post), scale=vec(scale),
             w_pre=vec(pre))
    dr, dn = rows(rtp), rows() if pre else none
    how = dict(groups=groups, gate_first=gate == "first", eps=1e-4)
    code = lz.LIZARD_ACT_SILU if act == "silu" else lz.LIZARD_ACT_SIGMOID
    t = {k: a[0] for k, a in v.items()}
    f = {k: a[1] for k, a in v.items()}
    o = t.pop("o")
    r_out, n_out = lz.lizard_block_norm_fwd(o, **t, **how, act=code)
    g = lz.lizard_block_norm_bwd(o, **t, **how, act=code, dr_out=dr[0], dn_out=dn[0])
    torch.cuda.synchronize()
    rr, rn = S.norm_fwd(**f, **how, act=act)
    # sums of squares lose at most D/256 + 16 roundings (a thread's, the lanes', the warps')
    cnt = 128 + D / 128
    size = np.abs(rr).max(1, keepdims=True) + (np.abs(f["r"]).max(1, keepdims=True) if res else 0)
    check(r_out, rr, size + np.abs(rr), cnt, "r_out")
    if pre:
        check(n_out, rn, np.abs(rn) + np.abs(rn).max(1, keepdims=True), cnt, "n_out")
    else:
        assert n_out is None
    ref = S.norm_bwd(**f, **how, act=act, dr_out=dr[1], dn_out=dn[1])
    for k in ("do", "dgate", "dr"):
        assert (g[k] is None) == (ref[k] is None), k
        if ref[k] is not None:  # each row's terms are within a few of its largest gradient
            scale_ = np.abs(ref["do"]).max(1, keepdims=True) * 4 + np.abs(ref[k]).max(1, keepdims=True) * 4
            check(g[k], ref[k], scale_, cnt, k)
    for k in ("dw_post", "dscale", "dw_pre"):
        assert (g[k] is None) == (ref[k] is None), k
        if ref[k] is not None:  # T terms of up to the rows' largest
            top = np.abs(ref["dr"]).max() if ref["dr"] is not None else np.abs(dr[1]).max() * 4
            mag = T * (top * (np.abs(rr).max() + 4) + np.abs(ref[k]).max())
            check(g[k], ref[k], mag, cnt + 2 * T, k)


def test_block_norm_in_place(lz):
    """r_out may be r, n_out may be o."""
    d = Draw(2, "bf16")
    o, r = d(33, 128)[0], d(33, 128)[0]
    w = d(128, dtype=torch.float32)[0]
    a, b = lz.lizard_block_norm_fwd(o, r=r, w_post=w, w_pre=w)
    o2, r2 = o.clone(), r.clone()
    lz.lizard_block_norm_fwd(o2, r=r2, w_post=w, w_pre=w, r_out=r2, n_out=o2)
    torch.cuda.synchronize()
    assert torch.equal(a, r2) and torch.equal(b, o2)


# ------------------------------------------------------------------------- streams and graphs


def test_other_stream_and_graph_replay(lz):
    """The calls run on the stream they are given; captured with their buffers they replay on new
    contents, offsets included."""
    d = Draw(4, "bf16")
    L, C, N = 300, 16, 16
    x, dt = d(1, L, C)[0], d(1, L, C)[0]
    Bm, Cm = d(1, L, 1, N)[0], d(1, L, 1, N)[0]
    A = -torch.ones(C, N, device="cuda")
    cu = offsets([100, 200])
    how = dict(cu_seqlens=cu)
    ref = lz.lizard_scan_fwd(x, dt, A, Bm, Cm, **how)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    lz.lizard_scan_fwd(x, dt, A, Bm, Cm, y=y, workspace=ws, stream=s, **how)
    torch.cuda.synchronize()
    assert torch.equal(y, ref)
    y.zero_()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        lz.lizard_scan_fwd(x, dt, A, Bm, Cm, y=y, workspace=ws, **how)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ref)
    cu.copy_(torch.tensor([0, 17, 300]))
    x.mul_(0.5)
    g.replay()
    again = lz.lizard_scan_fwd(x, dt, A, Bm, Cm, **how)
    torch.cuda.synchronize()
    assert torch.equal(y, again) and not torch.equal(y, ref)


def test_gradients_are_deterministic(lz):
    v, n = scan_inputs(10, "bf16")
    t = {k: a[0] for k, a in v.items()}
    how = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"])
    args = (t["x"], t["dt"], t["A"], t["Bm"], t["Cm"])
    _, st = lz.lizard_scan_fwd(*args, save_states=True, **how)
    a, b = (lz.lizard_scan_bwd(*args, t["dy"], st, **how) for _ in range(2))
    torch.cuda.synchronize()
    for k in a:
        if a[k] is not None:
            assert torch.equal(a[k], b[k]), k
