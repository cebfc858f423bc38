"""Pins of the selective block's float64 definitions: closed forms and central differences."""
import numpy as np
import pytest

from oracle import selective as S


def _diff(f, v, eps=1e-6):
    """Central differences of the scalar f with respect to v, in place."""
    g = np.zeros_like(v)
    it = np.nditer(v, flags=["multi_index", "zerosize_ok"])
    for _ in it:
        i = it.multi_index
        keep = v[i]
        v[i] = keep + eps
        hi = f()
        v[i] = keep - eps
        lo = f()
        v[i] = keep
        g[i] = (hi - lo) / (2 * eps)
    return g


def _close(got, want):
    # central differences of step 1e-6: truncation 1e-12, rounding 2^-53 / 1e-6 = 1e-10 of the
    # function's value (below 1e2 here)
    np.testing.assert_allclose(got, want, rtol=1e-6, atol=1e-7)


def test_conv_of_an_impulse_is_its_taps():
    w = np.arange(8.0).reshape(2, 4) + 1
    x = np.zeros((6, 2))
    x[1] = 1
    y, tail, _ = S.conv_fwd(x, w, np.zeros(2), np.zeros((3, 2)), act=False)
    np.testing.assert_array_equal(y[1:5], w.T[::-1])
    np.testing.assert_array_equal(tail, x[3:])


@pytest.mark.parametrize("L,K", [(1, 4), (2, 4), (5, 3), (4, 1)])
@pytest.mark.parametrize("act", [False, True])
def test_conv_gradients_by_differences(L, K, act):
    rng = np.random.default_rng(L * 10 + K)
    x, w, b = rng.normal(size=(L, 2)), rng.normal(size=(2, K)), rng.normal(size=2)
    st, dy, ds = rng.normal(size=(K - 1, 2)), rng.normal(size=(L, 2)), rng.normal(size=(K - 1, 2))

    def f():
        y, tail, _ = S.conv_fwd(x, w, b, st, act)
        return (y * dy).sum() + (tail * ds).sum()

    dx, dw, db, dst = S.conv_bwd(x, w, b, st, act, dy, ds)
    for got, v in ((dx, x), (dw, w), (db, b), (dst, st)):
        _close(got, _diff(f, v))


def test_scan_closed_forms():
    """One token: y = C d x B + D x; constant inputs: the geometric sum; A = 0: a running sum."""
    d, x, B, C, A = 0.3, 2.0, 0.7, -1.1, -0.9
    one = dict(B=np.full((5, 1, 1), B), Cm=np.full((5, 1, 1), C), D=np.zeros(1), z=None,
               dt_bias=np.zeros(1), h0=np.zeros((1, 1)), use_softplus=False)
    y, h = S.scan_fwd(np.full((5, 1), x), np.full((5, 1), d), np.full((1, 1), A), **one)
    a = np.exp(d * A)
    np.testing.assert_allclose(h[1:, 0, 0], d * x * B * (1 - a ** np.arange(1, 6)) / (1 - a), rtol=1e-14)
    np.testing.assert_allclose(y[:, 0], C * h[1:, 0, 0], rtol=1e-14)
    _, h = S.scan_fwd(np.full((5, 1), x), np.full((5, 1), d), np.zeros((1, 1)), **one)
    np.testing.assert_allclose(h[1:, 0, 0], d * x * B * np.arange(1, 6), rtol=1e-14)


@pytest.mark.parametrize("L,C,N,G", [(1, 2, 1, 1), (4, 4, 3, 2)])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("sp", [False, True])
def test_scan_gradients_by_differences(L, C, N, G, gate, sp):
    rng = np.random.default_rng(L + 7 * N)
    v = dict(x=rng.normal(size=(L, C)), dt=rng.uniform(0.1, 1, (L, C)), A=-rng.uniform(0.1, 2, (C, N)),
             B=rng.normal(size=(L, G, N)), Cm=rng.normal(size=(L, G, N)), D=rng.normal(size=C),
             z=rng.normal(size=(L, C)) if gate else None, dt_bias=rng.normal(size=C) * 0.1,
             h0=rng.normal(size=(C, N)))
    dy, dh = rng.normal(size=(L, C)), rng.normal(size=(C, N))

    def f():
        y, h = S.scan_fwd(**v, use_softplus=sp)
        return (y * dy).sum() + (h[-1] * dh).sum()

    o = S.scan_bwd(**v, dy=dy, dh_out=dh, use_softplus=sp)
    for k, g in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("Cm", "dC"), ("D", "dD"), ("z", "dz"),
                 ("dt_bias", "ddt_bias"), ("h0", "dh0")):
        if v[k] is not None:
            _close(o[g], _diff(f, v[k]))


@pytest.mark.parametrize("gate", ["", "first", "last"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("groups,post,pre,res", [(1, True, True, True), (3, True, False, True), (2, False, True, False)])
def test_norm_gradients_by_differences(gate, act, groups, post, pre, res):
    rng = np.random.default_rng(groups)
    T, D = 2, 6
    v = dict(o=rng.normal(size=(T, D)), gate=rng.normal(size=(T, D)) if gate else None,
             r=rng.normal(size=(T, D)) if res else None, w_post=rng.normal(size=D) if post else None,
             scale=rng.normal(size=D) if res else None, w_pre=rng.normal(size=D) if pre else None)
    how = dict(groups=groups, act=act, gate_first=gate == "first", eps=1e-3)
    dr, dn = rng.normal(size=(T, D)), rng.normal(size=(T, D)) if pre else None

    def f():
        r_out, n_out = S.norm_fwd(**v, **how)
        return (r_out * dr).sum() + ((n_out * dn).sum() if pre else 0)

    g = S.norm_bwd(**v, **how, dr_out=dr, dn_out=dn)
    for k, name in (("o", "do"), ("gate", "dgate"), ("r", "dr"), ("w_post", "dw_post"), ("scale", "dscale"),
                    ("w_pre", "dw_pre")):
        assert (g[name] is None) == (v[k] is None)
        if v[k] is not None:
            _close(g[name], _diff(f, v[k]))


def test_norm_of_a_row_has_unit_mean_square():
    rng = np.random.default_rng(0)
    r_out, n_out = S.norm_fwd(rng.normal(size=(3, 8)), None, None, np.ones(8), None, np.ones(8), 2, "silu", False, 0.0)
    np.testing.assert_allclose((r_out.reshape(3, 2, 4) ** 2).mean(-1), 1, rtol=1e-14)
    np.testing.assert_allclose((n_out ** 2).mean(-1), 1, rtol=1e-14)
