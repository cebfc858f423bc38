"""The rotation of queries and keys and the linear attention with a decay for each head at the limits of
their arguments: no epsilon, many states, values that are not finite, states that leave a call whole.
Tolerances as for the ordinary sizes, unless a test derives its own."""
import numpy as np
import pytest

from oracle import heads as H
from test_gpu_heads import Draw, check

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
