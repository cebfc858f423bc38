"""The selective block's calls write their outputs and nothing else: outputs as column ranges of wider
rows, between guard columns and guard rows, equal the dense outputs bit for bit and leave the guards
as they were."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

GUARD = 77.0


@pytest.fixture(scope="module")
def lz():
    from gated_linear_sliding_gb300 import lizard

    lizard.load()
    return lizard


FRONT = 8  # guard rows or entries before: eight of any width end on a 16-byte boundary


class Guarded:
    """A [B, L, width] view of a buffer whose other places hold GUARD."""

    def __init__(self, B, L, width, left, right, dtype, inner=None):
        self.buf = torch.full((FRONT + B * L + 1, left + width + right), GUARD, dtype=dtype, device="cuda")
        rows = self.buf[FRONT:-1].view(B, L, -1)
        self.flat = rows[..., left:left + width]
        self.view = self.flat if inner is None else self.flat.unflatten(-1, inner)

    def intact(self):
        keep = self.flat.clone()
        self.flat.fill_(GUARD)
        ok = bool((self.buf == GUARD).all())
        self.flat.copy_(keep)
        return ok


def rand(*shape, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,L,C,N,G,left,right", [(2, 37, 40, 16, 1, 8, 24), (1, 300, 24, 24, 2, 8, 3), (3, 19, 37, 5, 1, 8, 2),
                                                  (1, 130, 200, 3, 4, 16, 8)])
def test_scan_guards(lz, dtype, B, L, C, N, G, left, right):
    k = dict(dtype=dtype)
    x, dt, z, dy = (rand(B, L, C, seed=i, **k) for i in range(4))
    Bm, Cm = (rand(B, L, G, N, seed=i, **k) for i in (5, 6))
    A = -torch.exp(rand(C, N, dtype=torch.float32, seed=7))
    h = torch.full((FRONT + B + 1, C, N), GUARD, device="cuda")
    y, st = lz.lizard_scan_fwd(x, dt, A, Bm, Cm, z=z, save_states=True, h_out=h[FRONT:-1])
    assert (h[:FRONT] == GUARD).all() and (h[-1] == GUARD).all()
    dense = lz.lizard_scan_bwd(x, dt, A, Bm, Cm, dy, st, z=z)
    wide = {n: Guarded(B, L, C, left, right, dtype) for n in ("y", "dx", "ddt", "dz")}
    wide.update({n: Guarded(B, L, G * N, left, right, dtype, (G, N)) for n in ("dBm", "dCm")})
    lz.lizard_scan_fwd(x, dt, A, Bm, Cm, z=z, y=wide["y"].view)
    lz.lizard_scan_bwd(x, dt, A, Bm, Cm, dy, st, z=z, **{n: w.view for n, w in wide.items() if n != "y"})
    torch.cuda.synchronize()
    assert torch.equal(wide["y"].view, y)
    for n, w in wide.items():
        assert n == "y" or torch.equal(w.view, dense[n]), n
        assert w.intact(), n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,L,C,K,left,right", [(2, 37, 40, 4, 8, 24), (1, 200, 33, 2, 8, 1), (3, 5, 8, 8, 8, 8)])
def test_conv_guards(lz, dtype, B, L, C, K, left, right):
    x, dy = rand(B, L, C, dtype=dtype, seed=1), rand(B, L, C, dtype=dtype, seed=2)
    w, b = rand(C, K, dtype=torch.float32, seed=3), rand(C, dtype=torch.float32, seed=4)
    state = torch.full((FRONT + B + 1, K - 1, C), GUARD, dtype=dtype, device="cuda")
    y = lz.lizard_conv_fwd(x, w, b, act=1, state_out=state[FRONT:-1])
    dense = lz.lizard_conv_bwd(x, w, b, dy, act=1)
    wy, wd = Guarded(B, L, C, left, right, dtype), Guarded(B, L, C, left, right, dtype)
    lz.lizard_conv_fwd(x, w, b, act=1, y=wy.view)
    lz.lizard_conv_bwd(x, w, b, dy, act=1, dx=wd.view)
    torch.cuda.synchronize()
    assert (state[:FRONT] == GUARD).all() and (state[-1] == GUARD).all()
    assert torch.equal(wy.view, y) and torch.equal(wd.view, dense["dx"])
    assert wy.intact() and wd.intact()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,D,left,right", [(5, 40, 8, 24), (70, 4096, 8, 8), (3, 77, 8, 3), (700, 16, 8, 8)])
def test_norm_guards(lz, dtype, T, D, left, right):
    o, r = rand(T, D, dtype=dtype, seed=1), rand(T, D, dtype=torch.float32, seed=2)
    w = rand(D, dtype=torch.float32, seed=3)
    a, b = lz.lizard_block_norm_fwd(o, r=r, w_post=w, w_pre=w)
    ra, nb = Guarded(1, T, D, left, right, torch.float32), Guarded(1, T, D, left, right, dtype)
    lz.lizard_block_norm_fwd(o, r=r, w_post=w, w_pre=w, r_out=ra.view[0], n_out=nb.view[0])
    torch.cuda.synchronize()
    assert torch.equal(ra.view[0], a) and torch.equal(nb.view[0], b)
    assert ra.intact() and nb.intact()


def test_step_guards(lz):
    """Single tokens write their rows of y and their slots."""
    B, C, N, K = 5, 37, 6, 4
    slots = torch.tensor([3, -1, 0, 6, 1], dtype=torch.int64, device="cuda")
    k = dict(dtype=torch.bfloat16)
    x, dt, z = (rand(B, C, seed=i, **k) for i in range(3))
    Bm, Cm = rand(B, 1, N, seed=4, **k), rand(B, 1, N, seed=5, **k)
    A = -torch.ones(C, N, device="cuda")
    state = torch.full((FRONT + 8, C, N), GUARD, device="cuda")
    y = Guarded(1, B, C, 8, 3, torch.bfloat16)
    lz.lizard_scan_step(x, dt, A, Bm, Cm, state[FRONT:-1], z=z, slots=slots, y=y.view[0])
    torch.cuda.synchronize()
    touched = [FRONT + s for s in slots.tolist() if s >= 0]
    assert y.intact()
    for i in range(FRONT + 8):
        assert (i in touched) != bool((state[i] == GUARD).all()), i
    cs = torch.full((9, K - 1, C), GUARD, dtype=torch.bfloat16, device="cuda")
    cy = Guarded(1, B, C, 8, 3, torch.bfloat16)
    lz.lizard_conv_step(x, rand(C, K, dtype=torch.float32, seed=6), None, cs, slots=slots, y=cy.view[0])
    torch.cuda.synchronize()
    assert cy.intact()
    for i in range(9):
        assert (i in slots.tolist()) != bool((cs[i] == GUARD).all()), i
