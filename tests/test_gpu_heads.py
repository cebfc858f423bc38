"""The rotation of queries and keys and the linear attention with a decay for each head on the GPU
against their float64 definitions.

Tolerances.  Every output is an fp32 sum rounded once to its type: its error is at most half a step of
the type (eps / 2 relative to the value) plus n roundings of fp32 (2^-24 each) relative to the sum of
its terms' magnitudes, which the definitions give with absolute=True.
Rotation: n counts 32 roundings of a term (the norm's reciprocal root, products, cosine and sine of up to
four units of 1 with an angle of 2^-25 turns) and one for each value of the head in the sum of squares, twice
in the gradient; a weight's gradient one more for each row.
Decays: a term passes two products of d values, one of them in sums over 64 tokens, a rounding and a power for
every tile, and powers of up to 87 / ln 2 = 126 in the exponent, each rounded twice (2 ln 2 126 = 175 at
most where the term is not 0): n = 400 + 2 (dk + dv) + 4 L / 64 + 64.
Tensor cores round a pair's weight or the state to bf16 once (2^-8 of the term) on its way into an output of
bf16; on its way into a state that leaves the call it keeps its 24 bits in three parts (2^-17 is allowed).
"""
import numpy as np
import pytest

from oracle import heads as H

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U32 = 2.0 ** -24
EPS = 1e-6


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
            t = flat.unflatten(-1, t.shape[2:])
        return t, v


def check(got, ref, mag, n, what, part=0.0):
    """part: further roundings relative to the terms' magnitudes."""
    half = torch.finfo(got.dtype).eps / 2
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, what
    assert np.isfinite(got).all(), f"{what}: not finite"
    arith = (n * U32 + part) * mag
    tol = half * (np.abs(ref) + arith) + arith + 1e-37
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (what, int(bad.sum()), got.size, float((np.abs(got - ref) / tol).max()))


# --------------------------------------------------------------------------------- rotation


ROPE = [
    # B, L, Hq, Hkv, d, rot, sections, norm, weights, neighbours, far, stride
    (1, 1, 1, 1, 2, 2, None, True, True, False, 0, 0),
    (1, 1, 1, 0, 1, 0, None, True, True, False, 0, 0),
    (2, 5, 4, 2, 128, 128, None, True, True, False, 0, 0),
    (3, 33, 32, 8, 128, 128, None, True, True, False, 1 << 20, 0),
    (1, 70, 6, 3, 128, 64, None, True, False, True, 0, 0),
    (2, 9, 3, 1, 72, 40, [7, 13], True, True, False, 0, 0),
    (2, 9, 3, 1, 72, 40, [7, 13], True, True, True, 0, 0),
    (1, 65, 5, 5, 80, 64, [8, 12, 12], False, False, True, 40, 0),
    (1, 40, 2, 2, 256, 256, [100, 0, 20, 8], True, True, False, 3, 0),
    (1, 7, 2, 1, 512, 512, None, True, True, False, 0, 0),
    (2, 11, 3, 2, 33, 30, None, True, True, False, 0, 0),
    (2, 11, 3, 2, 33, 30, [3, 12], True, True, True, -9, 0),
    (1, 13, 2, 1, 511, 6, None, True, True, True, 0, 0),
    (2, 17, 4, 2, 64, 64, None, True, True, False, 5, 1024),
    (2, 17, 4, 2, 64, 64, None, True, True, False, 5, 1027),
    (1, 3, 40, 1, 32, 20, None, False, False, False, 0, 0),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,Hq,Hkv,d,rot,sections,norm,weights,near,far,stride", ROPE)
def test_rope(lz, dtype, B, L, Hq, Hkv, d, rot, sections, norm, weights, near, far, stride):
    D = Draw(d + L, dtype)
    strided = dict(stride=stride, at=16) if stride else {}
    q, qn = D(B, L, Hq, d, **strided)
    dq, dqn = D(B, L, Hq, d, **strided)
    k, kn = D(B, L, Hkv, d) if Hkv else (None, None)
    dk, dkn = D(B, L, Hkv, d) if Hkv else (None, None)
    wq, wqn = D(d, dtype=torch.float32, scale=0.2, shift=1.0) if weights else (None, np.ones(d))
    wk, wkn = D(d, dtype=torch.float32, scale=0.2, shift=1.0) if weights and Hkv else (None, np.ones(d))
    freqs, fn = D.dev(10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2)) * 1.7) if rot else (None, np.zeros(0))
    start, pos = 0, None
    if sections is None and far:
        start = far
    pn = start + np.tile(np.arange(L), (B, 1))[..., None]
    if sections is not None:
        pn = D.rng.integers(-3, 50, size=(B, L, len(sections))) + far
        pos = torch.from_numpy(pn).cuda()
    how = dict(positions=pos, sections=sections, start=start, w_q=wq, w_k=wk, norm=norm, eps=EPS, neighbours=near)
    yq, yk = lz.lizard_qk_rope_fwd(q, k, freqs, **how)
    g = lz.lizard_qk_rope_bwd(q, k, freqs, dq, dk, **how)
    torch.cuda.synchronize()
    for name, x, w, dy, y, dx, dw, wt in (("q", qn, wqn, dqn, yq, g["dq"], g["dw_q"], wq), ("k", kn, wkn, dkn, yk, g["dk"], g["dw_k"], wk)):
        if x is None:
            assert y is None and dx is None
            continue
        a = H.angles(pn.reshape(B * L, -1), fn, sections or [rot // 2])
        x, dy = x.reshape(B * L, -1, d), dy.reshape(B * L, -1, d)
        n = 32 + d
        ref, mag = (H.rope_fwd(x, w, a, near, norm, EPS, absolute=t) for t in (False, True))
        check(y.reshape(x.shape), ref, mag, n, name)
        (rdx, rdw), (mdx, mdw) = (H.rope_bwd(x, w, a, near, norm, EPS, dy, absolute=t) for t in (False, True))
        check(dx.reshape(x.shape), rdx, mdx, 2 * n, "d" + name)
        assert (dw is None) == (wt is None)
        if wt is not None:
            check(dw, rdw, mdw, n + B * L * x.shape[1], "dw_" + name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_in_place(lz, dtype):
    D = Draw(5, dtype)
    q, k, dq, dk = D(2, 9, 4, 64)[0], D(2, 9, 2, 64)[0], D(2, 9, 4, 64)[0], D(2, 9, 2, 64)[0]
    freqs = D(32, dtype=torch.float32)[0]
    w = D(64, dtype=torch.float32)[0]
    want = lz.lizard_qk_rope_fwd(q, k, freqs, w_q=w, w_k=w)
    gwant = lz.lizard_qk_rope_bwd(q, k, freqs, dq, dk, w_q=w, w_k=w)
    g = lz.lizard_qk_rope_bwd(q, k, freqs, dq, dk, w_q=w, w_k=w, dq=dq, dk=dk)
    got = lz.lizard_qk_rope_fwd(q, k, freqs, w_q=w, w_k=w, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert got[0] is q and g["dq"] is dq
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and all(torch.equal(gwant[n], g[n]) for n in gwant)


def test_rope_angles_of_far_positions(lz):
    """The angle is that of the exact product: against integers, in 2^-24 of a turn and the rounding of
    cosine and sine."""
    pos = torch.tensor([[0, 1, -1, 12345, 1 << 20, (1 << 31) - 1, -(1 << 33) + 7, (1 << 40) + 1]], device="cuda")
    freqs = torch.tensor([1.0, 0.1, 3e-5, 1e-12, 6.2831855, 700.5, -0.25, 0.0], device="cuda")
    q = torch.zeros(1, 8, 1, 16, device="cuda")
    q[..., :8] = 1.0
    y, _ = lz.lizard_qk_rope_fwd(q, None, freqs, positions=pos, norm=False)
    import math
    from fractions import Fraction

    two_pi = Fraction(2 * 3141592653589793238462643383279502884197169399375105820974944592307816406286209, 10 ** 78)
    for i, p in enumerate(pos[0].tolist()):
        for j, f in enumerate(freqs.tolist()):
            turn = Fraction(f) * p / two_pi
            a = 2 * math.pi * float(turn - math.floor(turn))
            off = 2 * math.pi * (2.0 ** -24 + abs(p) * 2.0 ** -63) + 4 * 2.0 ** -24
            assert abs(y[0, i, 0, j].item() - math.cos(a)) < off and abs(y[0, i, 0, 8 + j].item() - math.sin(a)) < off, (p, f)


def test_rope_values_that_are_not_finite_stay_in_their_row(lz):
    D = Draw(6, "f32")
    q, freqs = D(1, 4, 3, 32)[0], D(8, dtype=torch.float32)[0]
    want, _ = lz.lizard_qk_rope_fwd(q, None, freqs)
    bad = q.clone()
    bad[0, 1, 1, 20] = float("nan")
    bad[0, 2, 0, 3] = float("inf")
    got, _ = lz.lizard_qk_rope_fwd(bad, None, freqs)
    keep = torch.ones(4, 3, dtype=torch.bool)
    keep[1, 1] = keep[2, 0] = False
    assert torch.equal(got[0][keep.cuda()], want[0][keep.cuda()]) and got[0, 1, 1].isnan().all()
    # without a norm, beyond the rotated part, alone
    bad, _ = q.clone(), None
    bad[0, 0, 0, 20] = float("inf")
    got, _ = lz.lizard_qk_rope_fwd(bad, None, freqs, norm=False)
    want, _ = lz.lizard_qk_rope_fwd(q, None, freqs, norm=False)
    assert got[0, 0, 0, 20].item() == float("inf") and int((got != want).sum()) == 1
    freqs[3] = float("inf")
    got, _ = lz.lizard_qk_rope_fwd(q, None, freqs, norm=False)
    assert got[..., [3, 11]].isnan().all() and got.isnan().sum() == 2 * 12


# ----------------------------------------------------------------------------------- decays


DECAY = [
    # B, L, Hq, Hkv, dk, dv, lens, states given
    (1, 1, 1, 1, 1, 1, None, False),
    (2, 3, 2, 1, 8, 16, None, True),
    (1, 64, 4, 1, 64, 64, None, True),
    (2, 65, 4, 2, 128, 128, None, True),
    (1, 63, 8, 8, 128, 128, None, False),
    (1, 257, 4, 1, 128, 128, None, True),
    (1, 700, 3, 1, 128, 64, None, True),
    (3, 130, 6, 2, 40, 72, None, True),
    (1, 300, 16, 1, 64, 128, None, False),
    (1, 200, 5, 1, 80, 96, None, True),
    (2, 100, 2, 2, 33, 57, None, True),
    (1, 90, 2, 1, 160, 192, None, True),
    (1, 70, 2, 1, 128, 136, None, True),
    (1, 777, 4, 2, 128, 128, [1, 300, 0, 64, 65, 7, 340], True),
    (1, 500, 8, 2, 64, 128, [499, 1], True),
    (1, 200, 2, 1, 24, 8, [0, 0, 200, 0], True),
    (1, 130, 4, 4, 128, 128, [1] * 130, True),
    (1, 90, 3, 3, 7, 130, [30, 60], False),
]


def rates(rng, n):
    """Decays of every kind: none, slow, fast, within a tile's reach and far beyond it."""
    some = [0.0, -1e-4, -0.01, -0.3, -3.0, -60.0, -1e6, -np.inf]
    return np.array([some[i] for i in rng.permutation(8)] * ((n + 7) // 8))[:n]


def spans(B, L, lens):
    if lens is None:
        return [(b, 0, L) for b in range(B)]
    ends = np.cumsum(lens)
    return [(0, int(e - n), int(e)) for e, n in zip(ends, lens)]


def offsets(lens):
    return None if lens is None else torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64, device="cuda")


def slack(lz, dims):
    """Roundings relative to the terms: of outputs, of states."""
    return (2.0 ** -8 + 2.0 ** -16, 2.0 ** -17) if lz.lizard_decay_attn_kernel(dims) == 1 else (0.0, 0.0)


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,Hq,Hkv,dk,dv,lens,given", DECAY)
def test_decay(lz, dtype, B, L, Hq, Hkv, dk, dv, lens, given, seed):
    D = Draw(seed + L + dk, dtype)
    q, qn = D(B, L, Hq, dk)
    k, kn = D(B, L, Hkv, dk)
    v, vn = D(B, L, Hkv, dv)
    do, don = D(B, L, Hq, dv)
    l, ln = D.dev(rates(D.rng, Hkv))
    n = len(lens) if lens else B
    s0, s0n = D(n, Hkv, dk, dv, dtype=torch.float32) if given else (None, np.zeros((n, Hkv, dk, dv)))
    ds, dsn = D(n, Hkv, dk, dv, dtype=torch.float32) if given else (None, np.zeros((n, Hkv, dk, dv)))
    cu = offsets(lens)
    s_out, ds0 = torch.full((n, Hkv, dk, dv), 77.0, device="cuda"), torch.full((n, Hkv, dk, dv), 77.0, device="cuda")
    scale = 0.37
    o = lz.lizard_decay_attn_fwd(q, k, v, l, scale=scale, s0=s0, s_out=s_out, cu_seqlens=cu)
    g = lz.lizard_decay_attn_bwd(q, k, v, l, do, scale=scale, s0=s0, ds_out=ds, ds0=ds0, cu_seqlens=cu)
    torch.cuda.synchronize()
    rounds = 464 + 2 * (dk + dv) + L // 16
    part, spart = slack(lz, lz.lizard_decay_dims(B, L, Hq, Hkv, dk, dv, dtype=lz.LIZARD_F32 if dtype == "f32" else lz.LIZARD_BF16))
    for i, (b, a, e) in enumerate(spans(B, L, lens)):
        one = (qn[b, a:e], kn[b, a:e], vn[b, a:e], ln, s0n[i], scale)
        (ro, rs), (mo, ms) = (H.decay_fwd(*one, absolute=t) for t in (False, True))
        check(o[b, a:e], ro, mo, rounds, f"o {i}", part)
        check(s_out[i], rs, ms, rounds, f"s_out {i}", spart)
        rg, mg = (H.decay_bwd(*one, don[b, a:e], dsn[i], absolute=t) for t in (False, True))
        for name, r, m in zip(("dq", "dk", "dv"), rg, mg):
            check(g[name][b, a:e], r, m, rounds, f"{name} {i}", part)
        check(ds0[i], rg[3], mg[3], rounds, f"ds0 {i}", spart)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("stride,at", [(2048, 8), (1029, 16)])
def test_decay_strided(lz, dtype, stride, at):
    """Column ranges of wider rows give the dense call's bits where the same kernels serve both, else its
    values; nothing beside them is written."""
    D = Draw(7, dtype)
    B, L, Hq, Hkv, dk, dv = 2, 150, 4, 2, 64, 128
    dense = [D(B, L, h, d)[0] for h, d in ((Hq, dk), (Hkv, dk), (Hkv, dv), (Hq, dv))]
    l = D.dev([-0.1, -0.02])[0]

    def wide(t):
        rows = torch.full((B, L, stride), 77.0, dtype=t.dtype, device="cuda")
        view = rows[..., at:at + t[0, 0].numel()].unflatten(-1, t.shape[2:])
        return rows, view.copy_(t)

    rows = [wide(t) for t in dense]
    o = lz.lizard_decay_attn_fwd(*dense[:3], l)
    g = lz.lizard_decay_attn_bwd(*dense[:3], l, dense[3])
    out = {n: wide(t) for n, t in (("o", o), ("dq", g["dq"]), ("dk", g["dk"]), ("dv", g["dv"]))}
    for _, v in out.values():
        v.fill_(3.0)
    args = [v for _, v in rows]
    lz.lizard_decay_attn_fwd(*args[:3], l, o=out["o"][1])
    lz.lizard_decay_attn_bwd(*args[:3], l, args[3], dq=out["dq"][1], dk=out["dk"][1], dv=out["dv"][1])
    torch.cuda.synchronize()
    for n, t in (("o", o), ("dq", g["dq"]), ("dk", g["dk"]), ("dv", g["dv"])):
        whole, view = out[n]
        if stride % 8 == 0 or dtype == "f32":
            assert torch.equal(view, t), n
        else:  # two roundings to bf16, of values that differ by the tensor cores' rounding of their terms
            assert (view.float() - t.float()).norm() < 2.0 ** -6 * t.float().norm(), n
        view.fill_(77.0)
        assert (whole == 77.0).all(), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,lens", [(1, 700, None), (2, 64, None), (1, 700, [300, 0, 1, 399])])
def test_decay_states_in_place(lz, dtype, B, L, lens):
    """s_out is s0 and ds0 is ds_out, across segments and sequences: the same bits as with two arrays."""
    D = Draw(8, dtype)
    q, k, v, do = (D(B, L, h, 128)[0] for h in (2, 1, 1, 2))
    l = D.dev([-0.003])[0]
    n = len(lens) if lens else B
    s0, ds = D(n, 1, 128, 128, dtype=torch.float32)[0], D(n, 1, 128, 128, dtype=torch.float32)[0]
    cu = offsets(lens)
    two, dtwo = torch.empty_like(s0), torch.empty_like(s0)
    o = lz.lizard_decay_attn_fwd(q, k, v, l, s0=s0, s_out=two, cu_seqlens=cu)
    g = lz.lizard_decay_attn_bwd(q, k, v, l, do, s0=s0, ds_out=ds, ds0=dtwo, cu_seqlens=cu)
    one, done = s0.clone(), ds.clone()
    o1 = lz.lizard_decay_attn_fwd(q, k, v, l, s0=one, s_out=one, cu_seqlens=cu)
    g1 = lz.lizard_decay_attn_bwd(q, k, v, l, do, s0=s0, ds_out=done, ds0=done, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert torch.equal(o, o1) and torch.equal(one, two) and torch.equal(done, dtwo)
    assert all(torch.equal(g[n], g1[n]) for n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv,dk,dv", [(1, 1, 1, 1, 1), (5, 4, 2, 128, 128), (3, 9, 1, 64, 128), (2, 16, 8, 40, 72),
                                            (4, 3, 3, 33, 57), (2, 2, 1, 160, 192), (70, 8, 8, 32, 36)])
def test_decay_step(lz, dtype, B, Hq, Hkv, dk, dv):
    D = Draw(B + dk, dtype)
    nslots = B + 3
    slots = D.rng.permutation(nslots)[:B].astype(np.int64)
    if B > 2:
        slots[1] = -1
    state, sn = D(nslots, Hkv, dk, dv, dtype=torch.float32)
    (q, qn), (k, kn), (v, vn) = D(B, Hq, dk), D(B, Hkv, dk), D(B, Hkv, dv)
    l, ln = D.dev(rates(D.rng, Hkv))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    o = lz.lizard_decay_attn_step(q, k, v, l, state, scale=0.37, slots=torch.from_numpy(slots).cuda(), workspace=ws)
    assert lz.lizard_read_device_status(ws) == 0
    n = 200 + dk
    for b, slot in enumerate(slots):
        if slot < 0:
            assert (o[b] == 0).all()
            continue
        one = (qn[b][None], kn[b][None], vn[b][None], ln, sn[slot], 0.37)
        (ro, rs), (mo, ms) = (H.decay_fwd(*one, absolute=t) for t in (False, True))
        check(o[b], ro[0], mo[0], n, f"o {b}")
        check(state[slot], rs, ms, n, f"state {b}")
    idle = np.setdiff1d(np.arange(nslots), slots)
    assert np.array_equal(state[torch.from_numpy(idle).cuda()].double().cpu().numpy(), sn[idle])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decay_prompt_then_tokens(lz, dtype):
    """A prompt's last state goes on token by token: the outputs are those of the longer prompt, up to the
    roundings of both."""
    D = Draw(9, dtype)
    L, more, Hq, Hkv, d = 150, 6, 4, 2, 128
    (q, qn), (k, kn), (v, vn) = D(1, L + more, Hq, d), D(1, L + more, Hkv, d), D(1, L + more, Hkv, d)
    l, ln = D.dev([-0.01, -0.2])
    state = torch.empty(1, Hkv, d, d, device="cuda")
    lz.lizard_decay_attn_fwd(q[:, :L], k[:, :L], v[:, :L], l, s_out=state)
    one = (qn[0], kn[0], vn[0], ln, np.zeros((Hkv, d, d)), d ** -0.5)
    (ro, rs), (mo, ms) = (H.decay_fwd(*one, absolute=t) for t in (False, True))
    for t in range(L, L + more):
        o = lz.lizard_decay_attn_step(*(x[:, t].contiguous() for x in (q, k, v)), l, state)
        check(o[0], ro[t], mo[t], 1500, f"o {t}", 2.0 ** -17 if dtype == "bf16" else 0.0)
    check(state[0], rs, ms, 1500, "state", 2.0 ** -17 if dtype == "bf16" else 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decay_values_that_are_not_finite_stay_in_their_sequence_and_head(lz, dtype):
    D = Draw(10, dtype)
    lens, Hq, Hkv, d = [70, 30, 100], 4, 2, 128
    L, cu = sum(lens), offsets(lens)
    q, k, v, do = (D(1, L, h, d)[0] for h in (Hq, Hkv, Hkv, Hq))
    l = D.dev([-0.01, -0.2])[0]
    st = [torch.empty(3, Hkv, d, d, device="cuda") for _ in range(4)]
    o = lz.lizard_decay_attn_fwd(q, k, v, l, s_out=st[0], cu_seqlens=cu)
    g = lz.lizard_decay_attn_bwd(q, k, v, l, do, ds0=st[1], cu_seqlens=cu)
    bad = [t.clone() for t in (q, k, v, do)]
    bad[0][0, 75, 3, 5] = float("nan")  # sequence 1, query heads 2 and 3, state head 1
    bad[1][0, 80, 1, 7] = float("inf")
    bad[2][0, 90, 1, 0] = float("-inf")
    bad[3][0, 99, 2, 1] = float("nan")
    o2 = lz.lizard_decay_attn_fwd(*bad[:3], l, s_out=st[2], cu_seqlens=cu)
    g2 = lz.lizard_decay_attn_bwd(*bad[:3], l, bad[3], ds0=st[3], cu_seqlens=cu)
    torch.cuda.synchronize()
    rows = torch.ones(L, dtype=torch.bool, device="cuda")
    rows[70:100] = False
    for a, b in ((o, o2), (g["dq"], g2["dq"]), (g["dk"], g2["dk"]), (g["dv"], g2["dv"])):
        half = a.shape[2] // 2
        assert torch.equal(a[:, rows], b[:, rows]) and torch.equal(a[:, :, :half], b[:, :, :half])
        assert not torch.isfinite(b[:, 70:100, half:]).all()
    for a, b in ((st[0], st[2]), (st[1], st[3])):
        assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1, 0], b[1, 0])


def test_inconsistent_offsets_and_slots_are_reported(lz):
    D = Draw(11, "bf16")
    q, k, v, do = (D(1, 100, h, 128)[0] for h in (2, 1, 1, 2))
    l = D.dev([-0.1])[0]
    s = torch.zeros(3, 1, 128, 128, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    for cu in ([0, 50, 40, 100], [0, 10, 20, 90], [5, 10, 20, 100], [0, 1 << 40, -7, 100], [0, 0, 0, 200]):
        off = torch.tensor(cu, device="cuda")
        lz.lizard_decay_attn_fwd(q, k, v, l, s_out=s, cu_seqlens=off, workspace=ws)
        assert lz.lizard_read_device_status(ws) == lz.LIZARD_ERR_INVALID_ARG
        lz.lizard_decay_attn_bwd(q, k, v, l, do, ds0=s, cu_seqlens=off, workspace=ws)
        assert lz.lizard_read_device_status(ws) == lz.LIZARD_ERR_INVALID_ARG
    state = torch.ones(3, 1, 128, 128, device="cuda")
    slots = torch.tensor([1, 3, 1 << 40], device="cuda")
    o = lz.lizard_decay_attn_step(q[0, :3], k[0, :3], v[0, :3], l, state, slots=slots, workspace=ws)
    assert lz.lizard_read_device_status(ws) == lz.LIZARD_ERR_INVALID_ARG
    assert (o[1:] == 0).all() and (state[[0, 2]] == 1).all() and (state[1] != 1).any()


def test_repeated_calls_give_the_same_bits(lz):
    D = Draw(12, "bf16")
    q, k, v, do = (D(2, 900, h, 128)[0] for h in (8, 2, 2, 8))
    l = D.dev([-0.1, -0.001])[0]
    freqs, w = D(64, dtype=torch.float32)[0], D(128, dtype=torch.float32)[0]
    runs = []
    for _ in range(3):
        o = lz.lizard_decay_attn_fwd(q, k, v, l)
        g = lz.lizard_decay_attn_bwd(q, k, v, l, do)
        r = lz.lizard_qk_rope_bwd(q, k, freqs, q, k, w_q=w, w_k=w)
        runs.append([o, g["dq"], g["dk"], g["dv"], r["dq"], r["dk"], r["dw_q"], r["dw_k"]])
    torch.cuda.synchronize()
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))
