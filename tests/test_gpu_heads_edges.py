"""The rotation of queries and keys and the linear attention with a decay for each head where their calls
meet other streams, graphs, guards, long arrays and odd ways of cutting the time axis; and a run of them
between the projections and the norm, for prompts, single tokens and training."""
import threading

import numpy as np
import pytest

from oracle import heads as H
from oracle import selective as S
from test_gpu_heads import Draw, check, offsets, rates, slack, spans
from test_gpu_selective_canary import FRONT, GUARD, Guarded
from test_gpu_selective_edges import memory_stays, outputs_stay

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lz():
    from gated_linear_sliding_gb300 import lizard

    lizard.load()
    return lizard


# --------------------------------------------------------------------- cuts of the time axis


CUTS = [
    # B, L, Hq, Hkv, dk, dv, lens: tiles of an odd number of query heads over many segments, one query head
    # (chunks of 128 tokens), two segments shared by two CTAs, segments that sequences begin and end in
    (1, 1100, 5, 1, 64, 64, None),
    (1, 900, 3, 1, 128, 128, None),
    (2, 777, 7, 1, 32, 64, None),
    (1, 1500, 2, 2, 128, 128, None),
    (1, 1283, 1, 1, 64, 128, None),
    (1, 129, 52, 52, 32, 32, None),
    (2, 200, 60, 30, 32, 64, None),
    (1, 1401, 3, 3, 64, 64, [129, 0, 127, 128, 1, 1016]),
    (1, 1000, 6, 2, 64, 64, [1, 62, 1, 64, 500, 371, 1]),
    (1, 640, 1, 1, 128, 128, [640]),
    (1, 700, 2, 1, 192, 160, [333, 367]),
    (1, 450, 3, 1, 100, 130, None),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,Hq,Hkv,dk,dv,lens", CUTS)
def test_decay_over_segments(lz, dtype, B, L, Hq, Hkv, dk, dv, lens):
    """With first states, gradients of the last ones and decays of every kind, tolerances as for the
    shorter ones."""
    D = Draw(L, dtype)
    (q, qn), (k, kn), (v, vn), (do, don) = D(B, L, Hq, dk), D(B, L, Hkv, dk), D(B, L, Hkv, dv), D(B, L, Hq, dv)
    l, ln = D.dev(np.resize([-0.02, -0.001, *rates(D.rng, 8)], Hkv))
    n, cu, scale = len(lens or []) or B, offsets(lens), 0.21
    (s0, s0n), (ds, dsn) = (D(n, Hkv, dk, dv, dtype=torch.float32) for _ in range(2))
    s_out, ds0 = torch.full_like(s0, 77.0), torch.full_like(s0, 77.0)
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
@pytest.mark.parametrize("G", [1, 2])
def test_states_that_grow(lz, dtype, G):
    """Decays above 0, up to e^2.5 a token over 20 tokens: the formula's values."""
    D = Draw(3, dtype)
    L, Hkv, d = 20, 3, 64
    (q, qn), (k, kn), (v, vn), (do, don) = D(1, L, G * Hkv, d), D(1, L, Hkv, d), D(1, L, Hkv, d), D(1, L, G * Hkv, d)
    l, ln = D.dev([0.3, 0.9, 2.5])
    s_out, ds0 = torch.empty(1, Hkv, d, d, device="cuda"), torch.empty(1, Hkv, d, d, device="cuda")
    o = lz.lizard_decay_attn_fwd(q, k, v, l, scale=1.0, s_out=s_out)
    g = lz.lizard_decay_attn_bwd(q, k, v, l, do, scale=1.0, ds0=ds0)
    part, spart = slack(lz, lz.lizard_decay_dims(1, L, G * Hkv, Hkv, d, d, dtype=lz.LIZARD_F32 if dtype == "f32" else lz.LIZARD_BF16))
    one = (qn[0], kn[0], vn[0], ln, np.zeros((Hkv, d, d)), 1.0)
    (ro, rs), (mo, ms) = (H.decay_fwd(*one, absolute=t) for t in (False, True))
    rg, mg = (H.decay_bwd(*one, don[0], np.zeros((Hkv, d, d)), absolute=t) for t in (False, True))
    n = 464 + 4 * d
    check(o[0], ro, mo, n, "o", part)
    check(s_out[0], rs, ms, n, "s_out", spart)
    for name, r, m in zip(("dq", "dk", "dv"), rg, mg):
        check(g[name][0], r, m, n, name, part)
    check(ds0[0], rg[3], mg[3], n, "ds0", spart)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_tokens(lz, dtype):
    """Rows of length 0: states and their gradients pass, weights' gradients are zero."""
    D = Draw(4, dtype)
    q, k, v = (D(2, 1, h, 32)[0][:, :0] for h in (4, 2, 2))
    l = D.dev([-0.1, 0.0])[0]
    s0, s1, s2 = D(2, 2, 32, 32, dtype=torch.float32)[0], *(torch.full((2, 2, 32, 32), 77.0, device="cuda") for _ in range(2))
    assert lz.lizard_decay_attn_fwd(q, k, v, l, s0=s0, s_out=s1).shape == (2, 0, 4, 32)
    g = lz.lizard_decay_attn_bwd(q, k, v, l, q, ds_out=s0, ds0=s2)
    assert torch.equal(s0, s1) and torch.equal(s0, s2) and g["dk"].shape == k.shape
    lz.lizard_decay_attn_fwd(q, k, v, l, s_out=s1)
    assert (s1 == 0).all()
    w, freqs = D(32, dtype=torch.float32)[0], D(16, dtype=torch.float32)[0]
    assert lz.lizard_qk_rope_fwd(q, k, freqs, w_q=w, w_k=w)[0].shape == q.shape
    r = lz.lizard_qk_rope_bwd(q, k, freqs, q, k, w_q=w, w_k=w)
    assert (r["dw_q"] == 0).all() and (r["dw_k"] == 0).all()


# --------------------------------------------------------------------- long arrays


def test_rows_beyond_32_bits(lz):
    """Rows of a wide array whose last elements lie beyond 2^31: the dense call's bits."""
    D = Draw(5, "bf16")
    L, wide = 66000, 32768
    q, k, v, do = (D(1, L, h, 64)[0] for h in (2, 1, 1, 2))
    l, freqs = D.dev([-0.01])[0], D(32, dtype=torch.float32)[0]

    def far(t):
        rows = torch.empty(1, L, wide, dtype=t.dtype, device="cuda")
        return rows[..., wide - t[0, 0].numel():].unflatten(-1, t.shape[2:])

    wq, wo = far(q), far(q)
    wq.copy_(q)
    want, _ = lz.lizard_qk_rope_fwd(q, None, freqs)
    lz.lizard_qk_rope_fwd(wq, None, freqs, q_out=wo)
    assert torch.equal(wo, want)
    want = lz.lizard_qk_rope_bwd(q, None, freqs, do, None)["dq"]
    lz.lizard_qk_rope_bwd(wq, None, freqs, do, None, dq=wo)
    assert torch.equal(wo, want)
    o = lz.lizard_decay_attn_fwd(q, k, v, l)
    lz.lizard_decay_attn_fwd(wq, k, v, l, o=wo)
    assert torch.equal(wo, o)
    g = lz.lizard_decay_attn_bwd(q, k, v, l, do)
    g2 = lz.lizard_decay_attn_bwd(wq, k, v, l, do, dq=wo)
    assert torch.equal(wo, g["dq"]) and torch.equal(g["dk"], g2["dk"]) and torch.equal(g["dv"], g2["dv"])
    wk = far(k)  # k far out, and its gradient
    wk.copy_(k)
    g2 = lz.lizard_decay_attn_bwd(q, wk, v, l, do, dv=far(k))
    assert torch.equal(g["dk"], g2["dk"]) and torch.equal(g["dv"], g2["dv"])


def test_rows_beyond_32_bits_in_fp32_arithmetic(lz):
    D = Draw(6, "bf16")
    L, wide = 66000, 32770  # no multiple of 8: fp32 arithmetic
    q, k, v, do = (D(1, L, h, 36)[0] for h in (2, 1, 1, 2))
    l = D.dev([-0.01])[0]
    dense = [torch.empty(1, L, 74, dtype=q.dtype, device="cuda")[..., :72].unflatten(-1, (2, 36)).copy_(t) for t in (q, do)]
    rows = [torch.empty(1, L, wide, dtype=q.dtype, device="cuda")[..., 32696:32768].unflatten(-1, (2, 36)).copy_(t) for t in (q, do)]
    assert rows[0].data_ptr() % 16 == 0
    o = lz.lizard_decay_attn_fwd(dense[0], k, v, l)
    assert torch.equal(lz.lizard_decay_attn_fwd(rows[0], k, v, l), o)
    g = lz.lizard_decay_attn_bwd(dense[0], k, v, l, dense[1])
    out = torch.empty(1, L, wide, dtype=q.dtype, device="cuda")[..., 32696:32768].unflatten(-1, (2, 36))
    g2 = lz.lizard_decay_attn_bwd(rows[0], k, v, l, rows[1], dq=out)
    assert all(torch.equal(g[n], g2[n]) for n in g if n != "ds0")


def test_slots_beyond_32_bits(lz):
    D = Draw(7, "bf16")
    nslots = (1 << 31) // (128 * 128) + 9
    state = torch.zeros(nslots, 1, 128, 128, device="cuda")
    slots = torch.tensor([nslots - 1, 0, nslots - 5], device="cuda")
    first = D(3, 1, 128, 128, dtype=torch.float32)[0]
    state[slots] = first
    q, k, v = (D(3, h, 128)[0] for h in (4, 1, 1))
    l = D.dev([-0.1])[0]
    o = lz.lizard_decay_attn_step(q, k, v, l, state, slots=slots)
    assert torch.equal(o, lz.lizard_decay_attn_step(q, k, v, l, first)) and torch.equal(state[slots], first)
    state[slots] = 0
    assert not state.any()


# --------------------------------------------------------------------- guards


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,L,Hq,Hkv,d,left,right", [(2, 37, 3, 1, 64, 8, 24), (1, 300, 2, 2, 128, 16, 8), (1, 65, 5, 1, 33, 8, 3),
                                                     (2, 130, 4, 2, 72, 8, 8), (1, 400, 3, 1, 160, 8, 2)])
def test_guards(lz, dtype, B, L, Hq, Hkv, d, left, right):
    """Outputs between guard columns and rows, states between guard states, a workspace of just the bytes
    asked for: nothing else is written, and the values are the dense call's."""
    D = Draw(8, "f32" if dtype is torch.float32 else "bf16")
    q, k, v, do = (D(B, L, h, d)[0] for h in (Hq, Hkv, Hkv, Hq))
    l, freqs, w = D.dev(np.resize([-0.01, -0.4], Hkv))[0], D(d // 4, dtype=torch.float32)[0], D(d, dtype=torch.float32)[0]
    wide = {n: Guarded(B, L, h * d, left, right, dtype, (h, d))
            for n, h in (("q_out", Hq), ("k_out", Hkv), ("rdq", Hq), ("rdk", Hkv), ("o", Hq), ("dq", Hq), ("dk", Hkv), ("dv", Hkv))}
    # the dense form of a call that takes the same kernels: the same row distances
    same = {n: Guarded(B, L, h * d, left, right, dtype, (h, d)) for n, h in (("q_out", Hq), ("k_out", Hkv), ("rdq", Hq), ("rdk", Hkv),
                                                                            ("o", Hq), ("dq", Hq), ("dk", Hkv), ("dv", Hkv))}
    dims = lz.lizard_decay_dims(B, L, Hq, Hkv, d, d, dtype=lz.LIZARD_F32 if dtype is torch.float32 else lz.LIZARD_BF16,
                                **({} if right % 8 == 0 else dict(ldo=Hq * d + left + right)))
    rdims = lz.lizard_rope_dims(B=B, L=L, Hq=Hq, Hkv=Hkv, d=d, rot=2 * (d // 4), axes=1, dtype=dims.dtype, norm=1)
    need = dict(f=lz.lizard_decay_attn_fwd_workspace(dims), b=lz.lizard_decay_attn_bwd_workspace(dims), r=lz.lizard_qk_rope_bwd_workspace(rdims))
    runs = []
    for out in (same, wide):
        ws = {n: torch.full((m + 4096,), 0x5A, dtype=torch.uint8, device="cuda") for n, m in need.items()}
        states = [torch.full((FRONT + B + 1, Hkv, d, d), GUARD, device="cuda") for _ in range(2)]
        lz.lizard_qk_rope_fwd(q, k, freqs, w_q=w, w_k=w, q_out=out["q_out"].view, k_out=out["k_out"].view)
        r = lz.lizard_qk_rope_bwd(q, k, freqs, do, v, w_q=w, w_k=w, dq=out["rdq"].view, dk=out["rdk"].view, workspace=ws["r"][:need["r"]])
        lz.lizard_decay_attn_fwd(q, k, v, l, s_out=states[0][FRONT:-1], o=out["o"].view, workspace=ws["f"][:need["f"]])
        lz.lizard_decay_attn_bwd(q, k, v, l, do, ds0=states[1][FRONT:-1], dq=out["dq"].view, dk=out["dk"].view, dv=out["dv"].view,
                                 workspace=ws["b"][:need["b"]])
        torch.cuda.synchronize()
        for n, a in out.items():
            assert a.intact(), n
        for s in states:
            assert (s[:FRONT] == GUARD).all() and (s[-1] == GUARD).all() and (s[FRONT:-1] != GUARD).any()
        for n, t in ws.items():
            assert (t[need[n]:] == 0x5A).all(), n
        runs.append([out[n].view.clone() for n in out] + states + [r["dw_q"], r["dw_k"]])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    dense = [*lz.lizard_qk_rope_fwd(q, k, freqs, w_q=w, w_k=w)]
    # (another width of pieces or kernel: within a step of the type, and the tensor cores' rounding of terms)
    for a, b in zip(runs[0], dense):
        assert (a.float() - b.float()).norm() <= 2.0 ** -6 * b.float().norm()


# --------------------------------------------------------------------- streams and graphs


def calls(lz, host=False):
    """Each call as f(**more) -> its outputs."""
    D = Draw(9, "bf16")
    L, d = 640, 64
    cu = [0, 300, 640] if host else offsets([300, 340])
    q, k, v, do = (D(1, L, h, d)[0] for h in (4, 2, 2, 4))
    l, freqs, w = D.dev([-0.1, -0.003])[0], D(d // 2, dtype=torch.float32)[0], D(d, dtype=torch.float32)[0]
    s0 = D(2, 2, d, d, dtype=torch.float32)[0]
    kept = []

    def own(t):  # a state of the caller's: made before the call and alive after it
        kept.append(t.clone())
        torch.cuda.current_stream().synchronize()
        return kept[-1]

    def flat(f):
        def call(**more):
            out = f(**more)
            out = out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,)
            return [t for t in out if t is not None]
        return call

    return {n: flat(f) for n, f in dict(
        rope_fwd=lambda **m: lz.lizard_qk_rope_fwd(q, k, freqs, w_q=w, w_k=w, **m),
        rope_bwd=lambda **m: lz.lizard_qk_rope_bwd(q, k, freqs, do, v, w_q=w, w_k=w, **m),
        decay_fwd=lambda **m: lz.lizard_decay_attn_fwd(q, k, v, l, s0=s0, cu_seqlens=cu, **m),
        decay_bwd=lambda **m: lz.lizard_decay_attn_bwd(q, k, v, l, do, s0=s0, ds_out=s0, cu_seqlens=cu, **m),
        decay_step=lambda **m: lz.lizard_decay_attn_step(q[0, :2], k[0, :2], v[0, :2], l, own(s0), **m),
    ).items()}


CALLS = ["rope_fwd", "rope_bwd", "decay_fwd", "decay_bwd", "decay_step"]


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_on_another_stream(lz, name):
    memory_stays(calls(lz)[name])


@pytest.mark.parametrize("name", CALLS)
def test_outputs_of_a_call_on_another_stream(lz, name):
    outputs_stay(calls(lz)[name])


@pytest.mark.parametrize("name", ["decay_fwd", "decay_bwd"])
def test_host_offsets(lz, name):
    want, got = calls(lz)[name](), calls(lz, host=True)[name](stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_calls_of_two_host_threads(lz):
    """Two host threads on two streams, with sizes that take the same kernels: the bits of each alone."""
    D = Draw(10, "bf16")
    jobs = []
    for B, L, G in ((1, 700, 4), (2, 333, 1)):
        q, k, v, do = (D(B, L, h, 128)[0] for h in (2 * G, 2, 2, 2 * G))
        l = D.dev([-0.1, -0.003])[0]

        def job(q=q, k=k, v=v, do=do, l=l, **m):
            g = lz.lizard_decay_attn_bwd(q, k, v, l, do, **m)
            return [lz.lizard_decay_attn_fwd(q, k, v, l, **m), g["dq"], g["dk"], g["dv"]]
        jobs.append(job)
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    got, bad, start = [None, None], [], threading.Barrier(2)

    def work(i):
        try:
            s = torch.cuda.Stream()
            start.wait()
            for _ in range(200):
                got[i] = jobs[i](stream=s)
            s.synchronize()
        except Exception as e:  # reported by the test's thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def graph_of(f):
    f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    return g, out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_calls_replay_on_new_lengths(lz, dtype):
    """Forward and gradients captured with one workspace for two graphs (of different sizes), replayed in
    turn on other values, offsets and decays: the eager bits, states in place among them."""
    D = Draw(11, dtype)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    sets = []
    for L, G, cuts in ((900, 2, [[0, 300, 300, 900], [0, 1, 64, 900], [0, 0, 900, 900]]), (520, 1, [[0, 130, 390, 520], [0, 5, 517, 520], [0, 519, 520, 520]])):
        new = []
        for cut in cuts:
            x = dict(zip("qkvd", (D(1, L, h, 64)[0] for h in (2 * G, 2, 2, 2 * G))))
            x.update(l=D.dev(-np.exp(D.rng.uniform(-7, 1, 2)))[0], cu=torch.tensor(cut, device="cuda"), s0=D(3, 2, 64, 64, dtype=torch.float32)[0],
                     ds=D(3, 2, 64, 64, dtype=torch.float32)[0])
            new.append(x)
        at = {n: t.clone() for n, t in new[0].items()}

        def run(x, **m):
            s, ds = x["s0"].clone(), x["ds"].clone()
            o = lz.lizard_decay_attn_fwd(x["q"], x["k"], x["v"], x["l"], s0=s, s_out=s, cu_seqlens=x["cu"], **m)
            g = lz.lizard_decay_attn_bwd(x["q"], x["k"], x["v"], x["l"], x["d"], s0=x["s0"], ds_out=ds, ds0=ds, cu_seqlens=x["cu"], **m)
            return [o, s, g["dq"], g["dk"], g["dv"], ds]
        sets.append((new, [run(x) for x in new], at, *graph_of(lambda at=at, run=run: run(at, workspace=ws))))
    for i in range(3):
        for new, want, at, g, out in sets:
            for n in at:
                at[n].copy_(new[i][n])
            g.replay()
        torch.cuda.synchronize()
        for _, want, _, _, out in sets:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i])), i
    assert lz.lizard_read_device_status(ws) == 0


def test_captured_token_replays_on_new_slots_and_positions(lz):
    D = Draw(12, "bf16")
    B, slots, d = 6, 9, 64
    freqs, w, l = D(d // 2, dtype=torch.float32)[0], D(d, dtype=torch.float32)[0], D.dev([-0.1, -0.003])[0]
    state = D(slots, 2, d, d, dtype=torch.float32)[0]
    tokens = [dict(q=D(B, 1, 4, d)[0], k=D(B, 1, 2, d)[0], v=D(B, 1, 2, d)[0], at=torch.tensor(D.rng.integers(0, 1 << 40, (B, 1)), device="cuda"),
                   slots=torch.tensor(D.rng.permutation(slots)[:B], device="cuda")) for _ in range(5)]
    tokens[3]["slots"][2] = -1

    def run(t, state):
        q, k = lz.lizard_qk_rope_fwd(t["q"], t["k"], freqs, positions=t["at"], w_q=w, w_k=w)
        return lz.lizard_decay_attn_step(q[:, 0], k[:, 0], t["v"][:, 0], l, state, slots=t["slots"])

    eager = state.clone()
    want = [run(t, eager) for t in tokens]
    at = {n: a.clone() for n, a in tokens[0].items()}
    mine = state.clone()
    g, out = graph_of(lambda: run(at, mine))
    mine.copy_(state)
    for t, ref in zip(tokens, want):
        for n in at:
            at[n].copy_(t[n])
        g.replay()
        assert torch.equal(out, ref)
    assert torch.equal(mine, eager)


# --------------------------------------------------------------------- a run of them


class Layer:
    """Projections, rotation, attention and the norm with its gate and residual, of 4 query heads on 2."""

    def __init__(self, lz, seed):
        self.lz, self.D = lz, Draw(seed, "bf16")
        self.Hq, self.Hkv, self.d, self.width = 4, 2, 64, 256
        D, f32 = self.D, torch.float32
        self.W = D((4 + 2 + 2) * 64 + 256, 256, scale=1 / 16)[0]
        self.freqs, self.fn = D.dev(10000.0 ** (-np.arange(32) / 32))
        (self.w_q, self.wqn), (self.w_k, self.wkn), (self.w_post, self.wpn), (self.w_pre, self.wen) = (
            D(n, dtype=f32, scale=0.1, shift=1.0) for n in (64, 64, 256, 256))
        self.l, self.ln = D.dev([-0.02, -0.4])

    def rotated(self, x, start):
        q, k, v, g = self.lz.lizard_qkvg_proj(x, self.W, 4, 2, 64, 128)
        how = dict(start=start, w_q=self.w_q, w_k=self.w_k)
        return (q, k, v, g), self.lz.lizard_qk_rope_fwd(q, k, self.freqs, **how)

    def finish(self, o, g, x):
        rows = (-1, 256)
        return self.lz.lizard_block_norm_fwd(o.reshape(rows), gate=g.reshape(rows), r=x.reshape(rows), w_post=self.w_post, w_pre=self.w_pre, groups=4)


def double(t):
    return t.double().cpu().numpy()


def test_a_prompt_and_its_tokens(lz):
    """A layer's calls over a prompt, then token by token from the state that it leaves: each call against the
    definition of its own inputs, and the tokens' results against those of the longer prompt."""
    layer = Layer(lz, 20)
    L, more, d = 150, 5, 64
    x, _ = layer.D(1, L + more, 256)
    state = torch.empty(1, 2, d, d, device="cuda")
    raw, (q, k) = layer.rotated(x[:, :L].contiguous(), 0)
    o = lz.lizard_decay_attn_fwd(q, k, raw[2], layer.l, s_out=state)
    layer.finish(o, raw[3], x[:, :L].contiguous())

    def rope_right(raw, out, w, at, what):
        a = H.angles(np.asarray(at)[:, None], layer.fn, [32])
        ref, mag = (H.rope_fwd(double(raw), w, a, False, True, 1e-6, absolute=t) for t in (False, True))
        check(out, ref, mag, 32 + d, what)

    rope_right(raw[0][0], q[0], layer.wqn, range(L), "q")
    rope_right(raw[1][0], k[0], layer.wkn, range(L), "k")
    one = (double(q[0]), double(k[0]), double(raw[2][0]), layer.ln, np.zeros((2, d, d)), d ** -0.5)
    (ro, rs), (mo, ms) = (H.decay_fwd(*one, absolute=t) for t in (False, True))
    n = 464 + 4 * d + L // 16
    check(o[0], ro, mo, n, "o", 2.0 ** -8 + 2.0 ** -16)
    check(state[0], rs, ms, n, "state", 2.0 ** -17)

    raw_all, (qa, ka) = layer.rotated(x, 0)
    whole = layer.finish(lz.lizard_decay_attn_fwd(qa, ka, raw_all[2], layer.l), raw_all[3], x)
    for t in range(L, L + more):
        xt = x[:, t:t + 1].contiguous()
        raw, (q, k) = layer.rotated(xt, t)
        rope_right(raw[0][0], q[0], layer.wqn, [t], f"q {t}")
        before = double(state[0])
        o = lz.lizard_decay_attn_step(q[:, 0], k[:, 0], raw[2][:, 0], layer.l, state)
        one = (double(q[0]), double(k[0]), double(raw[2][0]), layer.ln, before, d ** -0.5)
        (ro, rs), (mo, ms) = (H.decay_fwd(*one, absolute=f) for f in (False, True))
        check(o, ro, mo, 200 + d, f"o {t}")
        check(state[0], rs, ms, 200 + d, f"state {t}")
        r, y = layer.finish(o, raw[3], xt)
        o64, g64, x64 = (double(a).reshape(1, 256) for a in (o, raw[3], xt))
        rr, ry = S.norm_fwd(o64, g64, x64, layer.wpn, None, layer.wen, groups=4, gate_first=False, act="silu", eps=1e-5)
        for a, ref in ((r, rr), (y, ry)):
            # one rounding to bf16, and fp32 sums of 256 terms with a dozen roundings each
            assert np.abs(double(a) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 300 * 2.0 ** -24 * np.abs(ref).max()
        for a, b in zip((r, y), whole):
            # the prompt's attention rounds pairs and states to bf16 where the token's keeps fp32, two calls round
            # their outputs: a few times 2^-9 of a row's norm
            b = b.view(1, L + more, 256)[:, t].float()
            assert (a.float() - b).norm() <= 2.0 ** -6 * b.norm()


def test_a_training_step_captured(lz):
    """The layer's forward and gradients, captured and replayed on other inputs: the eager bits."""
    layer = Layer(lz, 21)
    B, L = 2, 300
    data = [(layer.D(B, L, 256)[0], layer.D(B * L, 256)[0], layer.D(B * L, 256)[0]) for _ in range(2)]

    def step(x, dr, dn):
        rows = (-1, 256)
        raw, (q, k) = layer.rotated(x, 0)
        o = lz.lizard_decay_attn_fwd(q, k, raw[2], layer.l)
        out = layer.finish(o, raw[3], x)
        n = lz.lizard_block_norm_bwd(o.view(rows), gate=raw[3].view(rows), r=x.view(rows), w_post=layer.w_post, w_pre=layer.w_pre, groups=4,
                                     dr_out=dr, dn_out=dn)
        g = lz.lizard_decay_attn_bwd(q, k, raw[2], layer.l, n["do"].view(o.shape))
        r = lz.lizard_qk_rope_bwd(raw[0], raw[1], layer.freqs, g["dq"], g["dk"], w_q=layer.w_q, w_k=layer.w_k)
        dx, dW = lz.lizard_qkvg_proj_bwd(x, layer.W, r["dq"], r["dk"], g["dv"], n["dgate"].view(raw[3].shape))
        return [*out, n["dr"], n["dw_post"], n["dw_pre"], r["dw_q"], r["dw_k"], dx, dW]

    want = [step(*d) for d in data]
    at = [t.clone() for t in data[0]]
    g, out = graph_of(lambda: step(*at))
    for d, ref in reversed(list(zip(data, want))):
        for a, b in zip(at, d):
            a.copy_(b)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert all(torch.isfinite(t).all() for t in out)


def test_gradients_of_rotation_and_attention_are_the_differences(lz):
    """fp32: the loss sum(c o) + sum(e s_out) along random directions of every input, by central differences in
    64 bits, against the gradients of the two calls in a row.  A gradient's error is that of its calls (their
    tests), with the rotated queries and keys off by 32 + d roundings each; the differences' own is below h^2 of
    the terms' magnitude."""
    D = Draw(22, "f32")
    L, Hq, Hkv, d, scale = 90, 4, 2, 16, 0.25
    f32 = torch.float32
    names = dict(q=D(1, L, Hq, d), k=D(1, L, Hkv, d), v=D(1, L, Hkv, d), w_q=D(d, dtype=f32, shift=1.0), w_k=D(d, dtype=f32, shift=1.0),
                 s0=D(1, Hkv, d, d, dtype=f32))
    t, n = {i: a[0] for i, a in names.items()}, {i: a[1] for i, a in names.items()}
    (c, cn), (e, en), (l, ln), (freqs, fn) = D(1, L, Hq, d), D(1, Hkv, d, d, dtype=f32), D.dev([-0.05, -0.7]), D(d // 2, dtype=f32)
    a = H.angles(np.arange(L)[:, None], fn, [d // 2])

    def loss(x):
        q, k = (H.rope_fwd(x[i][0], x[w], a, False, True, 1e-6) for i, w in (("q", "w_q"), ("k", "w_k")))
        o, s = H.decay_fwd(q, k, x["v"][0], ln, x["s0"][0], scale)
        return (cn[0] * o).sum() + (en[0] * s).sum()

    q, k = lz.lizard_qk_rope_fwd(t["q"], t["k"], freqs, w_q=t["w_q"], w_k=t["w_k"])
    ds0 = torch.empty_like(t["s0"])
    g = lz.lizard_decay_attn_bwd(q, k, t["v"], l, c, scale=scale, s0=t["s0"], ds_out=e, ds0=ds0)
    r = lz.lizard_qk_rope_bwd(t["q"], t["k"], freqs, g["dq"], g["dk"], w_q=t["w_q"], w_k=t["w_k"])
    got = dict(q=r["dq"], k=r["dk"], v=g["dv"], w_q=r["dw_q"], w_k=r["dw_k"], s0=ds0)
    # the magnitudes of the terms
    mq, mk = (H.rope_fwd(n[i][0], n[w], a, False, True, 1e-6, absolute=True) for i, w in (("q", "w_q"), ("k", "w_k")))
    mags = H.decay_bwd(mq, mk, n["v"][0], ln, n["s0"][0], scale, cn[0], en[0], absolute=True)
    (gq, gwq), (gk, gwk) = (H.rope_bwd(n[i][0], n[w], a, False, True, 1e-6, m, absolute=True) for i, w, m in (("q", "w_q", mags[0]), ("k", "w_k", mags[1])))
    mag = dict(q=gq, k=gk, v=mags[2], w_q=gwq, w_k=gwk, s0=mags[3])
    rounds, h = 464 + 4 * d + L // 16 + 4 * (32 + d) + L * Hq, 1e-5
    for i in names:
        u = D.rng.normal(size=n[i].shape)
        diff = (loss({**n, i: n[i] + h * u}) - loss({**n, i: n[i] - h * u})) / (2 * h)
        size = (mag[i].reshape(u.shape) * np.abs(u)).sum()
        assert abs((double(got[i]) * u).sum() - diff) <= (rounds * 2.0 ** -24 + 1e-8) * size, i


# --------------------------------------------------------------------- refusals of the binding


def test_refusals(lz):
    D = Draw(13, "bf16")
    q, k, v = (D(1, 8, h, 32)[0] for h in (4, 2, 2))
    l, freqs, w = D.dev([-0.1, -0.2])[0], D(16, dtype=torch.float32)[0], D(32, dtype=torch.float32)[0]
    bad = (ValueError, TypeError, lz.LizardError)
    fwd, rope, step = lz.lizard_decay_attn_fwd, lz.lizard_qk_rope_fwd, lz.lizard_decay_attn_step
    state = torch.zeros(1, 2, 32, 32, device="cuda")
    for f in (lambda: fwd(q[0], k[0], v[0], l), lambda: fwd(q, k[:, :7], v, l), lambda: fwd(q, k.float(), v, l), lambda: fwd(q, k, v, l[:1]),
              lambda: fwd(q, k, v, l.double()), lambda: fwd(q, k, v, l.cpu()), lambda: fwd(q[:, :, :3], k, v, l),
              lambda: fwd(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, l), lambda: fwd(q, k, v, l, s0=state[:, :1]),
              lambda: fwd(q, k, v, l, s0=state.bfloat16()), lambda: fwd(q, k, v, l, scale=float("nan")),
              lambda: fwd(q, k, v, l, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
              lambda: fwd(q.expand(2, -1, -1, -1), k.expand(2, -1, -1, -1), v.expand(2, -1, -1, -1), l, cu_seqlens=[0, 8]),
              lambda: rope(q, k, freqs[:15], norm=False, sections=[8, 8], positions=torch.zeros(1, 8, 2, dtype=torch.int64, device="cuda")),
              lambda: rope(q, k, freqs, sections=[8, 8]), lambda: rope(q, k, freqs, w_q=w[:8]), lambda: rope(q, k, freqs, w_q=w, norm=False),
              lambda: rope(q, k, freqs, positions=torch.zeros(1, 8, dtype=torch.int32, device="cuda")),
              lambda: rope(q, k, torch.zeros(17, device="cuda")), lambda: rope(q, None, freqs, k_out=k),
              lambda: step(q[:, 0], k[:, 0], v[:, 0], l, state[:, :, :16]), lambda: step(q[:, 0], k[:, 0], v[:, 0], l, state.half()),
              lambda: step(q[0], k[0], v[0], l, state), lambda: step(q[:, 0], k[:, 0], v[:, 0], l, state, slots=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(bad):
            f()


# --------------------------------------------------------------------- long sums, repeated calls


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("H,L", [(160, 20000), (3, 20000)])
def test_states_of_long_sequences_do_not_drift(lz, dtype, G, H, L):
    """With next to no decay and positive terms a state is a sum of L of them: rounded to nearest its errors do not
    add up in one direction.  Uncut (160 states) and in segments.  A sum's L / 64 additions err by 2^-24 each at random,
    16 times that at most in 20000 tokens' 313; the split of the terms (2^-16) at random over L of them is below 2^-22.
    The power of a tile's length, which is the same for every tile, is within two units of the exact one (exp2f's bound:
    2^-23 below 1), and a term passes L / 128 of them on average: 1.9e-5 in one direction.  (Cut off after every addition
    of 16 rows, the states would be 8e-5 too small.)  fp32 arithmetic adds token by token, G L of them: an error of at
    most 2^-24 of a sum that grows in proportion has a deviation of 2^-24 / 3 of the last one, six deviations of all are
    2^-23 sqrt(G L)."""
    D = Draw(14, dtype)
    d, power = 16, L / 128 * 2.0 ** -23
    most = power + (2.0 ** -17 if dtype == "bf16" else 2.0 ** -23 * (G * L) ** 0.5)
    k, v = (torch.rand(1, L, H, d, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).add(0.5).to(D.dtype) for i in (1, 2))
    q = torch.zeros(1, L, G * H, d, dtype=D.dtype, device="cuda")
    s, l = torch.empty(1, H, d, d, device="cuda"), torch.full((H,), -1e-9, device="cuda")
    lz.lizard_decay_attn_fwd(q, k, v, l, s_out=s)
    ref = torch.einsum("lhi,lhj->hij", k[0].double(), v[0].double())
    err = (s[0].double() - ref) / ref + 0.5e-9 * L  # the decay's own: half of L of it on average
    assert err.mean().abs() < 2.0 ** -21 + power and err.abs().max() < most
    # backwards: dS = sum of q do^T
    g0 = torch.empty_like(s)
    lz.lizard_decay_attn_bwd(k.repeat_interleave(G, 2), k, v, l, v.repeat_interleave(G, 2), scale=1.0, ds0=g0)
    err = (g0[0].double() - G * ref) / (G * ref) + 0.5e-9 * L
    assert err.mean().abs() < 2.0 ** -21 + power and err.abs().max() < most


@pytest.mark.parametrize("Hq,Hkv,d,L", [(6, 2, 64, 130), (12, 3, 128, 300), (5, 1, 64, 700), (4, 4, 128, 400)])
@pytest.mark.parametrize("fast", [True, False])
def test_many_calls_give_the_same_bits(lz, Hq, Hkv, d, L, fast):
    """Whatever the memory held before."""
    D = Draw(15, "bf16")
    q, k, v, do = (D(2, L, h, d)[0] for h in (Hq, Hkv, Hkv, Hq))
    l, s0, want = D.dev(np.full(Hkv, -1e6 if fast else -0.01))[0], D(2, Hkv, d, d, dtype=torch.float32)[0], None
    for _ in range(40):
        torch.full((16 << 20,), float("nan"), device="cuda")
        s, ds = torch.empty_like(s0), torch.empty_like(s0)
        o = lz.lizard_decay_attn_fwd(q, k, v, l, s0=s0, s_out=s)
        g = lz.lizard_decay_attn_bwd(q, k, v, l, do, s0=s0, ds_out=s0, ds0=ds)
        got = [o, s, g["dq"], g["dk"], g["dv"], ds]
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
