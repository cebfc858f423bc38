"""The rotation of queries and keys and the linear attention with a decay for each head at the limits of
their arguments: no epsilon, many states, values that are not finite, states that leave a call whole.
Tolerances as for the ordinary sizes, unless a test derives its own."""
import numpy as np
import pytest

from oracle import heads as H
from test_gpu_heads import U32, Draw, check, offsets

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lz():
    from gated_linear_sliding_gb300 import lizard

    lizard.load()
    return lizard


# --------------------------------------------------------------------------------- rotation


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv", [(6, 4), (1, 3), (4, 1), (5, 0)])
@pytest.mark.parametrize("d,rot", [(128, 128), (72, 40), (33, 30)])  # pieces of eight, four and one
def test_rope_without_epsilon(lz, dtype, Hq, Hkv, d, rot):
    """eps = 0 and head counts that leave lanes without a head: the formula's values, the weights' gradients
    (which sum over all heads) among them."""
    D = Draw(Hq + Hkv + d, dtype)
    B, L = 2, 7
    freqs, fn = D.dev(10000.0 ** (-np.arange(rot // 2) / (rot // 2)))
    parts = {}
    for n, h in (("q", Hq), ("k", Hkv)):
        none = (None, None)
        parts[n] = (D(B, L, h, d), D(B, L, h, d), D(d, dtype=torch.float32, scale=0.2, shift=1.0)) if h else (none, none, none)
    how = dict(w_q=parts["q"][2][0], w_k=parts["k"][2][0], eps=0.0)
    y = dict(zip("qk", lz.lizard_qk_rope_fwd(parts["q"][0][0], parts["k"][0][0], freqs, **how)))
    g = lz.lizard_qk_rope_bwd(parts["q"][0][0], parts["k"][0][0], freqs, parts["q"][1][0], parts["k"][1][0], **how)
    a = H.angles(np.tile(np.arange(L), B)[:, None], fn, [rot // 2])
    for n, ((x, xn), (_, dyn), (_, w)) in parts.items():
        if x is None:
            continue
        xn, dyn = xn.reshape(B * L, -1, d), dyn.reshape(B * L, -1, d)
        rounds = 32 + d
        ref, mag = (H.rope_fwd(xn, w, a, False, True, 0.0, absolute=t) for t in (False, True))
        check(y[n].reshape(xn.shape), ref, mag, rounds, n)
        (rdx, rdw), (mdx, mdw) = (H.rope_bwd(xn, w, a, False, True, 0.0, dyn, absolute=t) for t in (False, True))
        check(g["d" + n].reshape(xn.shape), rdx, mdx, 2 * rounds, "d" + n)
        check(g["dw_" + n], rdw, mdw, rounds + B * L * xn.shape[1], "dw_" + n)


# ----------------------------------------------------------------------------------- decays


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [1, 2])
def test_states_in_place_of_many_sequences(lz, dtype, G):
    """More sequences than cuts, some over one cut or several, some that begin or end at one, empty ones among
    them: states in place give the bits of two arrays."""
    D = Draw(14 + G, dtype)
    lens = [64, 0, 30, 34, 0, 1, 126, 1, 64, 320, 63, 2] + [3] * 100 + [0, 200, 64, 90]
    L, Hkv, d, cu = sum(lens), 2, 64, offsets(lens)
    q, k, v, do = (D(1, L, h, d)[0] for h in (G * Hkv, Hkv, Hkv, G * Hkv))
    l = D.dev([-0.003, -0.9])[0]
    s0, ds = (D(len(lens), Hkv, d, d, dtype=torch.float32)[0] for _ in range(2))
    two, dtwo = torch.full_like(s0, 77.0), torch.full_like(s0, 77.0)
    o = lz.lizard_decay_attn_fwd(q, k, v, l, s0=s0, s_out=two, cu_seqlens=cu)
    g = lz.lizard_decay_attn_bwd(q, k, v, l, do, s0=s0, ds_out=ds, ds0=dtwo, cu_seqlens=cu)
    for _ in range(5):
        one, done = s0.clone(), ds.clone()
        o1 = lz.lizard_decay_attn_fwd(q, k, v, l, s0=one, s_out=one, cu_seqlens=cu)
        g1 = lz.lizard_decay_attn_bwd(q, k, v, l, do, s0=s0, ds_out=done, ds0=done, cu_seqlens=cu)
        torch.cuda.synchronize()
        assert torch.equal(o, o1) and torch.equal(one, two) and torch.equal(done, dtwo)
        assert all(torch.equal(g[n], g1[n]) for n in ("dq", "dk", "dv"))


def test_a_workspace_of_just_the_bytes_asked_for(lz):
    """Many sequences with states in place: nothing behind the workspace's last byte is written."""
    D = Draw(16, "bf16")
    lens = [5] * 300 + [1000]
    L, d, cu = sum(lens), 64, offsets(lens)
    q, k, v, do = (D(1, L, h, d)[0] for h in (2, 1, 1, 2))
    l = D.dev([-0.003])[0]
    s0 = D(len(lens), 1, d, d, dtype=torch.float32)[0]
    dims = lz.lizard_decay_dims(1, L, 2, 1, d, d, len(lens), scale=1.0, dtype=lz.LIZARD_BF16)
    for need, call in ((lz.lizard_decay_attn_fwd_workspace(dims), lambda s, w: lz.lizard_decay_attn_fwd(q, k, v, l, s0=s, s_out=s, cu_seqlens=cu, workspace=w)),
                       (lz.lizard_decay_attn_bwd_workspace(dims), lambda s, w: lz.lizard_decay_attn_bwd(q, k, v, l, do, ds_out=s, ds0=s, cu_seqlens=cu, workspace=w))):
        ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        call(s0.clone(), ws[:need])
        assert lz.lizard_read_device_status(ws) == 0 and (ws[need:] == 0x5A).all()


def same_where_finite(got, ref, mag, n, what, part):
    """The definition's values where it has them; where it has none (infinity, NaN), none either."""
    at = np.isfinite(ref)
    assert not np.isfinite(got.double().cpu().numpy()[~at]).any(), f"{what}: finite where the definition is not"
    keep = torch.from_numpy(at).cuda()
    check(got[keep], ref[at], mag[at], n, what, part)


NOT_FINITE = [
    # dtype, B, L, Hq, Hkv, dk, dv, log_decay: fp32 arithmetic, then tensor cores with two heads to a tile, an odd number
    # of them, and one (chunks of 128 tokens), decays within the split of their factors and beyond it, segments of one
    # chunk and of several
    ("f32", 1, 150, 4, 2, 40, 72, [-0.02, -0.9]),
    ("f32", 1, 150, 3, 3, 33, 57, [-0.02, -0.9, 0.0]),
    ("bf16", 1, 200, 2, 1, 136, 24, [-0.1]),
    ("bf16", 1, 150, 4, 2, 64, 128, [-0.02, -0.9]),
    ("bf16", 1, 150, 10, 2, 40, 72, [-0.9, -0.02]),
    ("bf16", 1, 150, 20, 2, 64, 64, [-0.02, -0.9]),
    ("bf16", 1, 150, 4, 2, 120, 24, [-0.02, -0.9]),
    ("bf16", 1, 150, 2, 2, 16, 128, [-0.02, -1e6]),
    ("bf16", 1, 300, 2, 2, 128, 64, [-0.02, -0.9]),
    ("bf16", 1, 450, 76, 76, 32, 32, np.resize([-0.02, -0.9], 76)),
    ("bf16", 4, 200, 60, 20, 32, 32, np.resize([-0.02, -0.9], 20)),
]


@pytest.mark.parametrize("kind", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
@pytest.mark.parametrize("dtype,B,L,Hq,Hkv,dk,dv,decay", NOT_FINITE)
def test_values_that_are_not_finite_reach_what_the_definition_says(lz, dtype, B, L, Hq, Hkv, dk, dv, decay, which, kind):
    """One value of q, k, v or do that is not finite, early and late in a chunk: results that the definition
    leaves finite (tokens before v's, tokens after do's, other heads) have its values."""
    D = Draw(L + dk, dtype)
    x = {n: D(B, L, h, d) for n, h, d in (("q", Hq, dk), ("k", Hkv, dk), ("v", Hkv, dv), ("do", Hq, dv))}
    l, ln = D.dev(np.asarray(decay))
    (s0, s0n), (ds, dsn) = (D(B, Hkv, dk, dv, dtype=torch.float32) for _ in range(2))
    dims = lz.lizard_decay_dims(B, L, Hq, Hkv, dk, dv, dtype=lz.LIZARD_F32 if dtype == "f32" else lz.LIZARD_BF16)
    tensor = lz.lizard_decay_attn_kernel(dims) == 1
    part = 2.0 ** -8 + 2.0 ** -16 if tensor else 0.0
    rounds, scale = 464 + 2 * (dk + dv) + L // 16, 0.37
    for t in (0, 1, 62, 64, 127, 131, L - 1):
        b, h = t % B, t % Hkv
        ends = {n: (a.clone(), w.copy()) for n, (a, w) in x.items()}
        dev, host = ends[which]
        head = h * (dev.shape[2] // Hkv) + t % (dev.shape[2] // Hkv)
        at = -1 - 5 * t % dev.shape[3]
        dev[b, t, head, at] = kind
        host[b, t, head, at] = kind
        s_out, ds0 = torch.empty_like(s0), torch.empty_like(s0)
        args = [ends[n][0] for n in ("q", "k", "v")]
        o = lz.lizard_decay_attn_fwd(*args, l, scale=scale, s0=s0, s_out=s_out)
        g = lz.lizard_decay_attn_bwd(*args, l, ends["do"][0], scale=scale, s0=s0, ds_out=ds, ds0=ds0)
        # the row that holds the value, and the state heads around it
        heads = slice(max(0, h - 1), h + 2)
        G = Hq // Hkv
        qheads = slice(heads.start * G, min(heads.stop, Hkv) * G)
        q, k, v, do = (ends[n][1][b][:, qheads if n in ("q", "do") else heads] for n in ("q", "k", "v", "do"))
        one = (q, k, v, ln[heads], s0n[b, heads], scale)
        with np.errstate(invalid="ignore"):
            (ro, rs), (mo, ms) = (H.decay_fwd(*one, absolute=a) for a in (False, True))
            rg, mg = (H.decay_bwd(*one, do, dsn[b, heads], absolute=a) for a in (False, True))
        same_where_finite(o[b, :, qheads], ro, mo, rounds, f"o {t}", part)
        same_where_finite(s_out[b, heads], rs, ms, rounds, f"s_out {t}", 2.0 ** -17 if tensor else 0.0)
        for n, r, m in zip(("dq", "dk", "dv"), rg, mg):
            same_where_finite(g[n][b][:, qheads if n == "dq" else heads], r, m, rounds, f"{n} {t}", part)
        same_where_finite(ds0[b, heads], rg[3], mg[3], rounds, f"ds0 {t}", 2.0 ** -17 if tensor else 0.0)


@pytest.mark.parametrize("G", [1, 2])
def test_padding_that_is_not_finite(lz, G):
    """A dense batch of ragged rows whose padding was never written: every token in front of it has the
    definition's value."""
    D = Draw(13, "bf16")
    B, L, Hkv, d, lens = 3, 400, 2, 64, (130, 400, 1)
    x, xn = zip(*(D(B, L, h, d) for h in (G * Hkv, Hkv, Hkv)))
    l, ln = D.dev([-0.02, -0.9])
    for b, n in enumerate(lens):
        for t in x:
            t[b, n:] = float("nan")
    got = lz.lizard_decay_attn_fwd(*x, l)
    for b, n in enumerate(lens):
        one = (*(t[b, :n] for t in xn), ln, np.zeros((Hkv, d, d)), d ** -0.5)
        ro, mo = (H.decay_fwd(*one, absolute=t)[0] for t in (False, True))
        check(got[b, :n], ro, mo, 464 + 4 * d + n // 16, f"o {b}", 2.0 ** -8 + 2.0 ** -16)


@pytest.mark.parametrize("G,Hkv", [(1, 2), (2, 2), (1, 80), (2, 80)])
def test_states_in_place_around_values_that_are_not_finite(lz, G, Hkv):
    """Sequences of which two hold such values, in segments and in one, states in place: the others keep their bits, and
    all have those of two arrays."""
    D = Draw(17 + G, "bf16")
    lens = [70, 64, 0, 200, 130, 50]
    L, d, cu = sum(lens), 64, offsets(lens)
    q, k, v, do = (D(1, L, h, d)[0] for h in (G * Hkv, Hkv, Hkv, G * Hkv))
    l = D.dev(np.resize([-0.003, -0.9], Hkv))[0]
    s0, ds = (D(len(lens), Hkv, d, d, dtype=torch.float32)[0] for _ in range(2))
    bv, bdo = v.clone(), do.clone()
    bv[0, 300, :, 3] = float("nan")  # of sequence 3, tokens 134 to 333
    bdo[0, 150, :, 5] = float("inf")
    bv[0, 69, :, 1] = bdo[0, 69, :, 1] = float("inf")  # of sequence 0, tokens 0 to 69

    def run(v, do, in_place):
        a, b = s0.clone(), ds.clone()
        a1, b1 = (a, b) if in_place else (torch.full_like(a, 77.0), torch.full_like(b, 77.0))
        o = lz.lizard_decay_attn_fwd(q, k, v, l, s0=a, s_out=a1, cu_seqlens=cu)
        g = lz.lizard_decay_attn_bwd(q, k, v, l, do, s0=s0, ds_out=b, ds0=b1, cu_seqlens=cu)
        torch.cuda.synchronize()
        return [o, g["dq"], g["dk"], g["dv"]], [a1, b1]

    clean, states = run(v, do, False)
    two, two_s = run(bv, bdo, False)
    one, one_s = run(bv, bdo, True)
    rows = torch.ones(L, dtype=torch.bool, device="cuda")
    rows[134:334] = rows[:70] = False
    others = [1, 2, 4, 5]
    for a, b, c in zip(clean, two, one):
        assert torch.equal(b.nan_to_num(99.0), c.nan_to_num(99.0)) and torch.equal(b.isnan(), c.isnan())
        assert not torch.isfinite(b[:, 134:334]).all() and not torch.isfinite(b[:, :70]).all()
        assert torch.equal(a[:, rows], b[:, rows])
    for a, b, c in zip(states, two_s, one_s):
        assert torch.equal(b.nan_to_num(99.0), c.nan_to_num(99.0)) and torch.equal(b.isnan(), c.isnan())
        assert torch.equal(a[others], b[others]) and not torch.isfinite(b[3]).all() and not torch.isfinite(b[0]).all()


def test_many_sequences_with_values_that_are_not_finite(lz):
    """More of them in a segment than are noted one by one, states in place: the definition's values, infinities among
    them, for all."""
    D = Draw(19, "bf16")
    G, Hkv, d, n, each = 2, 80, 32, 150, 3  # one segment a head
    L, cu = n * each, offsets([each] * n)
    (q, qn), (k, kn), (v, vn), (do, don) = (D(1, L, h, d) for h in (G * Hkv, Hkv, Hkv, G * Hkv))
    l, ln = D.dev(np.resize([-0.003, -0.9], Hkv))
    (s0, s0n), (ds, dsn) = (D(n, Hkv, d, d, dtype=torch.float32) for _ in range(2))
    for t, a in ((v, vn), (do, don)):
        t[0, 1:-30:each, :, 3] = float("inf")
        a[0, 1:-30:each, :, 3] = np.inf
    s, e = s0.clone(), ds.clone()
    o = lz.lizard_decay_attn_fwd(q, k, v, l, scale=0.37, s0=s, s_out=s, cu_seqlens=cu)
    g = lz.lizard_decay_attn_bwd(q, k, v, l, do, scale=0.37, s0=s0, ds_out=e, ds0=e, cu_seqlens=cu)
    part = 2.0 ** -8 + 2.0 ** -16
    for i in (0, 1, 63, 64, 65, 139, 140, 149):
        at, heads = slice(each * i, each * i + each), slice(0, 3)
        one = (qn[0, at, :3 * G], kn[0, at, heads], vn[0, at, heads], ln[heads], s0n[i, heads], 0.37)
        with np.errstate(invalid="ignore"):
            (ro, rs), (mo, ms) = (H.decay_fwd(*one, absolute=a) for a in (False, True))
            rg, mg = (H.decay_bwd(*one, don[0, at, :3 * G], dsn[i, heads], absolute=a) for a in (False, True))
        same_where_finite(o[0, at, :3 * G], ro, mo, 600, f"o {i}", part)
        same_where_finite(s[i, heads], rs, ms, 600, f"s_out {i}", 2.0 ** -17)
        for name, r, m in zip(("dq", "dk", "dv"), rg, mg):
            same_where_finite(g[name][0, at, :3 * G] if name == "dq" else g[name][0, at, heads], r, m, 600, f"{name} {i}", part)
        same_where_finite(e[i, heads], rg[3], mg[3], 600, f"ds0 {i}", 2.0 ** -17)


WHOLE = [
    # B, L, Hq, Hkv, lens, token: states that leave from the walk itself (a packed batch; one segment; two that share an
    # end), and from the ends and their join; with several query heads a state and with one
    (1, 40, 2, 1, None, 3),
    (1, 40, 1, 1, None, 3),
    (1, 60, 2, 1, [20, 40], 25),
    (2, 128, 80, 40, None, 70),
    (2, 128, 40, 40, None, 70),
    (1, 128, 2, 1, None, 5),
    (1, 190, 2, 1, None, 70),
    (1, 190, 1, 1, None, 70),
]


@pytest.mark.parametrize("B,L,Hq,Hkv,lens,token", WHOLE)
def test_states_that_leave_keep_their_24_bits(lz, B, L, Hq, Hkv, lens, token):
    """States of one token's product, on the tensor cores: every entry is a power of the decay times two values,
    which two bf16 parts of the scaled row miss by up to 2^-17, three by up to 2^-26.
    Roundings, in units of 2^-24 of the entry: the decay's log2 (a rounding and its constant's, of an exponent of
    up to 0.19) 0.3, its product with a distance 0.2, the power (two units in the last place) 4, the row times it 1 and times
    the scale 1, two cut-off additions of the parts 4: 11.  For each tile of 64 tokens that the state passes then (three
    at most), and for its join, a power as the one above, its product and an addition: 7.  Together 39.  Two parts miss
    the largest remainders by about 100, which is shown on the same row."""
    d, l = 128, -0.003
    rng = np.random.default_rng(L + Hq)
    ln = np.float64(np.float32(l))
    decay = torch.full((Hkv,), l, device="cuda")
    n, cu = len(lens or []) or B, offsets(lens)
    begin, end = (0, L) if lens is None else (lens[0], L)
    G, h, b = Hq // Hkv, Hkv // 2, B - 1
    seq = b if lens is None else 1
    y, z = (torch.from_numpy(rng.normal(size=d).astype(np.float32)).to("cuda", torch.bfloat16) for _ in range(2))
    units = 11 + 7 * 4
    outer = torch.outer(y.double(), z.double()).cpu().numpy()

    def close(got, far, scale):
        ref = scale * np.exp(ln * far) * outer
        off = np.abs(got.double().cpu().numpy() / ref - 1)
        assert off.max() < units * U32, off.max() / U32
        # the same from two parts of the row
        row = (y.double() * scale * np.exp(ln * far)).float().cpu()
        hi = row.bfloat16().float()
        two = hi.double() + (row - hi).bfloat16().double()
        assert (two / row.double() - 1).abs().max() > units * U32

    q, k, v, do = (torch.zeros(B, L, m, d, dtype=torch.bfloat16, device="cuda") for m in (Hq, Hkv, Hkv, Hq))
    k[b, token, h], v[b, token, h] = y, z
    q[b, token, h * G], do[b, token, h * G] = y, z
    s_out, ds0 = (torch.full((n, Hkv, d, d), 77.0, device="cuda") for _ in range(2))
    assert lz.lizard_decay_attn_kernel(lz.lizard_decay_dims(B, L, Hq, Hkv, d, d, dtype=lz.LIZARD_BF16)) == 1
    lz.lizard_decay_attn_fwd(q, k, v, decay, s_out=s_out, cu_seqlens=cu)
    lz.lizard_decay_attn_bwd(q, k, v, decay, do, scale=0.37, ds0=ds0, cu_seqlens=cu)
    close(s_out[seq, h], end - 1 - token, 1.0)
    close(ds0[seq, h], token + 1 - begin, np.float64(np.float32(0.37)))
    s_out[seq, h] = ds0[seq, h] = 0
    assert not s_out.any() and not ds0.any()
