"""The selective block on the GPU where its calls meet odd sizes, other streams and threads, and values
far out."""
import ctypes
import threading

import numpy as np
import pytest

from oracle import selective as S
from test_gpu_selective import Draw, check, offsets, tdt

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lz():
    from gated_linear_sliding_gb300 import lizard

    lizard.load()
    return lizard


# ------------------------------------------------------------------------------- states in place


@pytest.mark.parametrize("B,L,C,N,lens", [(1, 600, 1001, 16, None), (1, 600, 9, 4, None), (3, 1500, 37, 8, None),
                                          (1, 700, 13, 16, [300, 0, 1, 399])])
def test_scan_in_place_state_of_odd_channels(lz, B, L, C, N, lens):
    """h_out is h0, the time axis is cut and the channels are odd: the same bits as with two arrays."""
    d = Draw(11, "f32")
    x, dt = d(B, L, C)[0], d(B, L, C, shift=-1.0)[0]
    Bm, Cm = d(B, L, 1, N)[0], d(B, L, 1, N)[0]
    A = d.dev(-np.exp(d.rng.normal(size=(C, N))))[0]
    h0 = d(B if lens is None else len(lens), C, N)[0]
    cu = offsets(lens)
    h, st = torch.empty_like(h0), h0.clone()
    y = lz.lizard_scan_fwd(x, dt, A, Bm, Cm, h0=h0, h_out=h, cu_seqlens=cu)
    y2 = lz.lizard_scan_fwd(x, dt, A, Bm, Cm, h0=st, h_out=st, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, st)


# ------------------------------------------------------------------------------------- streams


def block_calls(lz, host=False):
    """Each call of the block as f(**more) -> its outputs; the packed ones with offsets on the device or
    as host integers."""
    d = Draw(21, "bf16")
    L, C, N = 640, 64, 16
    cu = [0, 300, 640] if host else offsets([300, 340])
    x, dt, dy = (d(1, L, C)[0] for _ in range(3))
    Bm, Cm = d(1, L, 1, N)[0], d(1, L, 1, N)[0]
    A = d.dev(-np.exp(d.rng.normal(size=(C, N))))[0]
    w = d(C, 4, dtype=torch.float32)[0]
    v = d(C, dtype=torch.float32)[0]
    state, h = d(3, 3, C)[0], d(3, C, N, dtype=torch.float32)[0]
    _, st = lz.lizard_scan_fwd(x, dt, A, Bm, Cm, cu_seqlens=cu, save_states=True)
    rows, last = x[0], (x[0, :3], dt[0, :3], A, Bm[0, :3], Cm[0, :3])

    kept = []

    def own(t):  # a step's state, the caller's: made before the call and alive after it
        kept.append(t.clone())
        torch.cuda.current_stream().synchronize()
        return kept[-1]

    def flat(f):
        def call(**more):
            out = f(**more)
            out = out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,)
            return [t for t in out if t is not None]
        return call

    return {k: flat(f) for k, f in dict(
        conv_fwd=lambda **m: lz.lizard_conv_fwd(x, w, v, act=1, cu_seqlens=cu, **m),
        conv_bwd=lambda **m: lz.lizard_conv_bwd(x, w, v, dy, act=1, cu_seqlens=cu, **m),
        conv_step=lambda **m: lz.lizard_conv_step(rows[:3], w, v, own(state), act=1, **m),
        scan_fwd=lambda **m: lz.lizard_scan_fwd(x, dt, A, Bm, Cm, cu_seqlens=cu, save_states=True, **m),
        scan_bwd=lambda **m: lz.lizard_scan_bwd(x, dt, A, Bm, Cm, dy, st, cu_seqlens=cu, **m),
        scan_step=lambda **m: lz.lizard_scan_step(*last, own(h), **m),
        norm_fwd=lambda **m: lz.lizard_block_norm_fwd(rows, r=rows, w_post=v, w_pre=v, **m),
        norm_bwd=lambda **m: lz.lizard_block_norm_bwd(rows, r=rows, w_post=v, w_pre=v, dr_out=rows, dn_out=rows, **m),
    ).items()}


CALLS = ["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step", "norm_fwd", "norm_bwd"]


def memory_stays(f):
    """A call f on another stream, which is still busy, takes no memory back to the current stream
    before its kernels are done: neither does it see what is written there meanwhile, nor does it
    write there."""
    want = f()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    sizes = (512, 4096, 1 << 14, 1 << 16, 1 << 18, 1 << 20, 2 << 20, 5 << 20, 20 << 20)

    def filled():
        return [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(24 if n <= 1 << 16 else 4)]

    # the streams' pools have blocks of these sizes from here on, and the kernels are loaded: nothing
    # below makes the host wait
    filled()
    f(stream=s)
    f()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)  # 0.1 s
    got = f(stream=s)
    fill = filled()
    torch.cuda.current_stream().synchronize()
    assert not s.query()  # the call's kernels are still to come
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i
    assert all(bool((t == 0x5A).all()) for t in fill)


def outputs_stay(f):
    """A call f on another stream writes no memory that pending work of the current stream still reads."""
    want = f()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    keep = [torch.full(t.shape, 7, dtype=t.dtype, device="cuda") for t in want for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    late = [t.clone() for t in keep]
    del keep
    got = f(stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in late)
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_on_another_stream(lz, name):
    memory_stays(block_calls(lz)[name])


@pytest.mark.parametrize("name", CALLS)
def test_outputs_of_a_call_on_another_stream(lz, name):
    outputs_stay(block_calls(lz)[name])


@pytest.mark.parametrize("name", ["conv_fwd", "conv_bwd", "scan_fwd", "scan_bwd"])
def test_host_offsets_on_another_stream(lz, name):
    """Offsets copied for a call on another stream (the host waits for the copy) are not overwritten by
    the current stream."""
    f = block_calls(lz, host=True)[name]
    want = f()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        got = f(stream=s)
        fill = [torch.full((3,), -1, dtype=torch.int64, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), i
        del fill


# ------------------------------------------------------------------------------- host threads


@pytest.mark.parametrize("widths", [(8192, 5120), (4096, 2056)])
def test_norms_of_two_host_threads(lz, widths):
    """Two host threads whose rows take the same kernels with different amounts of shared memory: every
    call succeeds and gives the bits it gives alone.  The library is called without the binding, so
    that the threads spend their time inside it."""
    d = Draw(31, "f32")
    T, data, want = 4, [], []
    for D in widths:
        o, r, w = d(T, D)[0], d(T, D)[0], d(D)[0]
        how = dict(r=r, w_post=w, w_pre=w)
        g = lz.lizard_block_norm_bwd(o, **how, dr_out=r, dn_out=o)
        want.append([*lz.lizard_block_norm_fwd(o, **how), g["do"], g["dr"], g["dw_post"], g["dw_pre"]])
        data.append((o, r, w))
    torch.cuda.synchronize()
    lib, got, bad, start = lz.load(), [None, None], [0, 0], threading.Barrier(2)

    def work(i):
        (o, r, w), D, s = data[i], widths[i], torch.cuda.Stream()
        dims = lz.lizard_norm_dims(T=T, D=D, groups=1, eps_post=1e-5, eps_pre=1e-5, dtype=0, res_dtype=0, act=1)
        out = [torch.zeros_like(t) for t in want[i]]
        ws = lz.new_workspace(lz.lizard_block_norm_bwd_workspace(dims), "cuda")
        torch.cuda.synchronize()
        p, po, pr, pw = [t.data_ptr() for t in out], o.data_ptr(), r.data_ptr(), w.data_ptr()
        ref, st = ctypes.byref(dims), s.cuda_stream
        start.wait()
        for _ in range(10000):
            bad[i] += lib.lizard_block_norm_fwd(ref, po, None, pr, pw, None, pw, p[0], p[1], st) != 0
            bad[i] += lib.lizard_block_norm_bwd(ref, po, None, pr, pw, None, pw, pr, po, p[2], None, p[3], p[4], None, p[5],
                                                ws.data_ptr(), ws.numel(), st) != 0
        s.synchronize()
        got[i] = out

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert bad == [0, 0]
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


# ------------------------------------------------------------------------------- step sizes


def step_sizes(lz, dt, way):
    """softplus(dt) as the state after one token of x = Bm = 1 from zero."""
    n = dt.numel()
    one = torch.ones(1, 1, n, dtype=dt.dtype, device="cuda")
    A, h = -torch.ones(n, 1, device="cuda"), torch.zeros(1, n, 1, device="cuda")
    bc = torch.ones(1, 1, 1, 1, dtype=dt.dtype, device="cuda")
    if way == "prompt":
        lz.lizard_scan_fwd(one, dt.view(1, 1, n), A, bc, bc, h_out=h)
    else:
        lz.lizard_scan_step(one[0], dt.view(1, n), A, bc[0], bc[0], h)
    torch.cuda.synchronize()
    return h.view(n).double().cpu().numpy()


@pytest.mark.parametrize("way", ["prompt", "step"])
def test_softplus_keeps_its_digits(lz, way):
    """Relative error over arguments from -87 to 20.  In units of 2^-24: four for ex2.approx (2^-22), two
    for rcp.approx (one ulp), one each for the correction's last step, u + 2, u / (2 + u) and the last
    multiply-add, two for the polynomial: twelve.  The remainder's own rounding is below 2^-40."""
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-87, 20, 200_000), rng.uniform(-1, 1, 50_000), rng.uniform(-20, -5, 50_000)])
    v = v.astype(np.float32)
    got = step_sizes(lz, torch.from_numpy(v).cuda(), way)
    w = v.astype(np.float64)
    want = np.maximum(w, 0) + np.log1p(np.exp(-np.abs(w)))
    err = np.abs(got - want) / want * 2.0 ** 24
    assert err.max() <= 12, (err.max(), w[err.argmax()])


@pytest.mark.parametrize("way", ["prompt", "step"])
def test_softplus_far_out(lz, way):
    """A token whose step is masked by the lowest value or minus infinity passes nothing; below 2^-126 a
    step size is zero; NaN stays."""
    f = np.float32
    v = np.array([-np.inf, np.finfo(f).min, -1e30, -200, -128, -103, -88, -87.5, 88, 128, 129, 1e30, np.inf, np.nan, 0], f)
    got = step_sizes(lz, torch.from_numpy(v).cuda(), way)
    w = v.astype(np.float64)
    want = np.maximum(w, 0) + np.log1p(np.exp(-np.abs(w)))
    assert np.isnan(got[13]) and got[12] == np.inf
    assert (got[:5] == 0).all()
    assert (np.abs(got[:8] - want[:8]) <= 2.0 ** -126).all()
    assert (np.abs(got[8:12] / want[8:12] - 1) <= 12 * 2.0 ** -24).all() and abs(got[14] / want[14] - 1) <= 12 * 2.0 ** -24


# ------------------------------------------------------------------------------- long memory


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,N,G", [(24, 16, 1), (10, 5, 2), (7, 1, 1)])
def test_states_token_by_token_are_the_prompts(lz, dtype, C, N, G):
    """250 single tokens move a state to the bits that a prompt of them (one segment) moves it to: the
    same decays, products and sums in the same order.  (A bias of the decays adds up over tokens.)"""
    d = Draw(41, dtype)
    L = 250
    x, dt = d(2, L, C)[0], d(2, L, C, shift=-5.0)[0]
    Bm, Cm = d(2, L, G, N)[0], d(2, L, G, N)[0]
    A = d.dev(-np.exp(d.rng.normal(size=(C, N))))[0]
    bias = d(C, dtype=torch.float32, scale=0.3)[0]
    h0 = d(2, C, N, dtype=torch.float32)[0]
    h, st = torch.empty_like(h0), h0.clone()
    lz.lizard_scan_fwd(x, dt, A, Bm, Cm, dt_bias=bias, h0=h0, h_out=h)
    for t in range(L):
        lz.lizard_scan_step(x[:, t].contiguous(), dt[:, t].contiguous(), A, Bm[:, t].contiguous(), Cm[:, t].contiguous(), st,
                            dt_bias=bias)
    torch.cuda.synchronize()
    assert torch.equal(h, st)


# ------------------------------------------------------------------------------- parameter gradients

PARAM = [  # T, D, groups, gate ("", first, last), residual: more rows than CTAs, so that each adds up several
    (1300, 16, 1, "last", "same"),
    (2000, 128, 1, "", "f32"),
    (400, 37, 1, "last", "same"),
    (1400, 1023, 3, "first", "f32"),   # one column a piece, group sums through shared memory
    (1400, 512, 2, "last", "same"),
    (700, 1040, 8, "first", "same"),
    (700, 2050, 2, "last", "same"),
    (400, 2048, 1, "last", "f32"),
    (400, 3840, 3, "first", "same"),   # eight columns a piece, group sums through shared memory
    (400, 4096, 1, "last", "same"),
    (400, 5000, 1, "last", "f32"),     # sums in shared memory from here on
    (400, 8184, 3, "first", "same"),
    (330, 9000, 3, "last", "f32"),     # in the CTAs' partial sums from here on
    (330, 9001, 1, "first", "same"),
    (310, 16384, 8, "last", "same"),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(PARAM)))
def test_parameter_gradients_of_many_rows(lz, dtype, case):
    """dw_post, dscale and dw_pre where a CTA walks several rows.  A term passes at most 128 roundings
    before the sums over rows (a row's sum: 16 of a thread, ten of the lanes and warps, three such sums;
    the gate's exponential and reciprocal eight; two dozen products), which have T / 8 in a chain at
    most; each is 2^-24 of the term's magnitude, added up over a column's rows.  A lost row is about
    1 / T of that sum, more than twenty times as much."""
    T, D, groups, gate, res = PARAM[case]
    d = Draw(case, dtype)
    rtp = tdt(dtype) if res == "same" else torch.float32
    vec = lambda: d(D, dtype=torch.float32, scale=0.3, shift=1.0)  # noqa: E731
    v = dict(o=d(T, D), gate=d(T, D) if gate else (None, None), r=d(T, D, dtype=rtp), w_post=vec(), scale=vec(), w_pre=vec())
    dr, dn = d(T, D, dtype=rtp), d(T, D)
    t, f = {k: a[0] for k, a in v.items()}, {k: a[1] for k, a in v.items()}
    o = t.pop("o")
    how = dict(groups=groups, gate_first=gate == "first", eps=1e-4)
    g = lz.lizard_block_norm_bwd(o, **t, **how, dr_out=dr[0], dn_out=dn[0])
    torch.cuda.synchronize()
    ref = S.norm_bwd(**f, **how, act="silu", dr_out=dr[1], dn_out=dn[1])
    # the terms' magnitudes
    a = np.abs(S.silu(f["gate"])) if gate else np.ones((T, D))
    u = np.abs(f["o"]) * (a if gate == "first" else 1)
    parts = u.reshape(T, groups, -1)
    unit = (parts / np.sqrt((parts ** 2).mean(-1, keepdims=True) + 1e-4)).reshape(T, D)
    n = unit * np.abs(f["w_post"]) * (a if gate == "last" else 1)
    rr_out, _ = S.norm_fwd(**f, **how, act="silu")
    q = np.sqrt((rr_out ** 2).mean(-1, keepdims=True) + 1e-4)
    rr = np.abs(f["r"]) + np.abs(f["scale"]) * n
    w = np.abs(dn[1] * f["w_pre"])
    grad = np.abs(dr[1]) + w / q + rr * (w * rr).mean(-1, keepdims=True) / q ** 3
    mags = dict(dw_pre=np.abs(dn[1]) * rr / q, dscale=grad * n,
                dw_post=grad * np.abs(f["scale"]) * unit * (a if gate == "last" else 1))
    for k, m in mags.items():
        check(g[k], ref[k], m.sum(0), 128 + T / 8, k)


# ------------------------------------------------------------------------------- captured steps


def test_captured_token_replays_on_new_tokens_and_slots(lz):
    """A token's three calls captured into a graph, replayed on other tokens and slots (one idle, others
    in another order), give the eager calls' bits in outputs and states."""
    d = Draw(51, "bf16")
    B, C, N, slots = 6, 40, 16, 9
    w, v = d(C, 4, dtype=torch.float32)[0], d(C, dtype=torch.float32, shift=1.0)[0]
    A = d.dev(-np.exp(d.rng.normal(size=(C, N))))[0]
    conv, state = d(slots, 3, C)[0], d(slots, C, N, dtype=torch.float32)[0]
    tokens = [dict(x=d(B, C)[0], dt=d(B, C, shift=-2.0)[0], Bm=d(B, 1, N)[0], Cm=d(B, 1, N)[0], z=d(B, C)[0], r=d(B, C)[0],
                   slots=torch.tensor(d.rng.permutation(slots)[:B], device="cuda")) for _ in range(5)]
    tokens[3]["slots"][2] = -1

    def run(t, conv, state):
        x = lz.lizard_conv_step(t["x"], w, v, conv, slots=t["slots"], act=1)
        y = lz.lizard_scan_step(x, t["dt"], A, t["Bm"], t["Cm"], state, D=v, z=t["z"], slots=t["slots"])
        return lz.lizard_block_norm_fwd(y, r=t["r"], w_post=v, scale=v, w_pre=v)

    ec, es = conv.clone(), state.clone()
    want = [run(t, ec, es) for t in tokens]
    gc, gs = conv.clone(), state.clone()
    at = {k: a.clone() for k, a in tokens[0].items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(at, gc, gs)
    for t, ref in zip(tokens, want):
        for k in at:
            at[k].copy_(t[k])
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert torch.equal(gc, ec) and torch.equal(gs, es)


# ------------------------------------------------------------------------------- values not finite


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("L,C,N", [(70, 37, 5), (600, 24, 16)])
def test_a_channel_that_is_not_finite_stays_alone(lz, bad, L, C, N):
    """One channel's inputs hold such values at some tokens: every other channel's results, forward and
    backward, are the bits they are without them, over one segment and over several."""
    d = Draw(61, "bf16")
    t = {k: d(2, L, C)[0] for k in ("x", "dt", "z", "dy")}
    Bm, Cm = d(2, L, 1, N)[0], d(2, L, 1, N)[0]
    A = d.dev(-np.exp(d.rng.normal(size=(C, N))))[0]
    w, v = d(C, 4, dtype=torch.float32)[0], d(C, dtype=torch.float32)[0]

    def results(t):
        h = torch.empty(2, C, N, device="cuda")
        how = dict(D=v, z=t["z"], dt_bias=v)
        y, st = lz.lizard_scan_fwd(t["x"], t["dt"], A, Bm, Cm, h_out=h, save_states=True, **how)
        g = lz.lizard_scan_bwd(t["x"], t["dt"], A, Bm, Cm, t["dy"], st, **how)
        c = lz.lizard_conv_fwd(t["x"], w, v, act=1)
        gc = lz.lizard_conv_bwd(t["x"], w, v, t["dy"], act=1)
        wide = [y, g["dx"], g["ddt"], g["dz"], c, gc["dx"]]
        return wide, [h.transpose(0, 1), g["dA"], g["dD"], g["ddt_bias"], gc["dw"], gc["dbias"]]

    want = results(t)
    channel, keep = 11, [c for c in range(C) if c != 11]
    for k in t:
        t[k][:, ::13, channel] = bad
    got = results(t)
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got[0], want[0])):
        assert torch.equal(a[..., keep], b[..., keep]), i
        assert not torch.isfinite(a[..., channel]).all(), i
    for i, (a, b) in enumerate(zip(got[1], want[1])):
        assert torch.equal(a[keep], b[keep]), i


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mask", ["inf", "lowest"])
def test_masked_tokens(lz, dtype, mask):
    """Tokens whose dt is minus infinity or the lowest value, all of a sequence's among them: outputs,
    states and gradients against 64 bits, with the counts of roundings of the scan's tests."""
    B, L, C, N = 3, 330, 16, 16
    d = Draw(71, dtype)
    low = -np.inf if mask == "inf" else torch.finfo(tdt(dtype)).min
    raw = d.rng.normal(size=(B, L, C)).astype(np.float32)
    raw[d.rng.random((B, L)) < 0.3] = low
    raw[2] = low
    dt, dtv = d.dev(raw, tdt(dtype))
    (x, xv), (z, zv), (dy, dyv) = (d(B, L, C) for _ in range(3))
    (Bm, Bv), (Cm, Cv) = d(B, L, 1, N), d(B, L, 1, N)
    A, Av = d.dev(-np.exp(d.rng.normal(size=(C, N))))
    (b, bv), (h0, hv) = d(C, dtype=torch.float32), d(B, C, N, dtype=torch.float32)
    h = torch.empty_like(h0)
    how = dict(z=z, dt_bias=b, h0=h0)
    y, st = lz.lizard_scan_fwd(x, dt, A, Bm, Cm, h_out=h, save_states=True, **how)
    g = lz.lizard_scan_bwd(x, dt, A, Bm, Cm, dy, st, **how)
    torch.cuda.synchronize()
    assert torch.equal(h[2], h0[2])
    for i in range(B):
        a = (xv[i], dtv[i], Av, Bv[i], Cv[i], np.zeros(C), zv[i], bv, hv[i])
        up = (dyv[i], np.zeros((C, N)))
        (ry, rh), (my, mh) = S.scan_fwd(*a), S.scan_fwd(*a, absolute=True)
        check(y[i], ry, my, 16 * L + 64 + N, f"y {i}")
        check(h[i], rh[-1], mh[-1], 16 * L + 64 + N, f"h {i}")
        r, m = S.scan_bwd(*a, *up), S.scan_bwd(*a, *up, absolute=True)
        for k, gk in (("dx", "dx"), ("ddt", "ddt"), ("dz", "dz"), ("dB", "dBm"), ("dC", "dCm")):
            check(g[gk][i], r[k], m[k], 32 * L + 128 + N + 2 * C, f"{gk} {i}")
