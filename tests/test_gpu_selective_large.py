"""Tensors of more than 2^31 elements: the last tokens' results equal those of a call on the last
tokens alone that continues the earlier ones' state."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

L, C, TAIL = 540_032, 4096, 208  # 2.2e9 elements; the tail begins on a chunk of 16 tokens


@pytest.fixture(scope="module")
def lz():
    from gated_linear_sliding_gb300 import lizard

    lizard.load()
    return lizard


@pytest.fixture(scope="module")
def data():
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free device memory")
    assert L * C > 2 ** 31
    g = torch.Generator("cuda").manual_seed(1)
    out = {n: torch.empty(1, L, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for n in ("x", "dt", "dy")}
    yield out
    out.clear()
    torch.cuda.empty_cache()


def tail(t):
    return t[:, -TAIL:].contiguous()


def test_conv(lz, data):
    w = torch.randn(C, 4, device="cuda")
    y = lz.lizard_conv_fwd(data["x"], w, act=1)
    state = data["x"][:, -TAIL - 3:-TAIL].contiguous()
    assert torch.equal(tail(y), lz.lizard_conv_fwd(tail(data["x"]), w, act=1, state_in=state))
    del y
    dx = lz.lizard_conv_bwd(data["x"], w, None, data["dy"], act=1)["dx"]
    part = lz.lizard_conv_bwd(tail(data["x"]), w, None, tail(data["dy"]), act=1, state_in=state)["dx"]
    assert torch.equal(tail(dx), part)


def test_norm(lz, data):
    w = torch.randn(C, device="cuda")
    o, r = data["x"][0], data["dt"][0]
    how = dict(w_post=w, w_pre=w)
    a, b = lz.lizard_block_norm_fwd(o, r=r, **how)
    c, d = lz.lizard_block_norm_fwd(o[-TAIL:].contiguous(), r=r[-TAIL:].contiguous(), **how)
    assert torch.equal(a[-TAIL:], c) and torch.equal(b[-TAIL:], d)
    del b
    g = lz.lizard_block_norm_bwd(o, r=r, dr_out=data["dy"][0], dn_out=a, **how)
    p = lz.lizard_block_norm_bwd(o[-TAIL:].contiguous(), r=r[-TAIL:].contiguous(), dr_out=data["dy"][0, -TAIL:].contiguous(),
                                 dn_out=a[-TAIL:].contiguous(), **how)
    assert torch.equal(g["do"][-TAIL:], p["do"]) and torch.equal(g["dr"][-TAIL:], p["dr"])


def test_scan(lz, data):
    """The two ways sum in another order: half a bf16 step each, and the roundings of 208 tokens of
    fp32 (16 each) relative to the largest value."""
    N = 16
    g = torch.Generator("cuda").manual_seed(2)
    Bm, Cm = (torch.randn(1, L, 1, N, generator=g, device="cuda").bfloat16() for _ in range(2))
    A = -torch.arange(1, N + 1, device="cuda").float().repeat(C, 1)
    y, states = lz.lizard_scan_fwd(data["x"], data["dt"], A, Bm, Cm, save_states=True)
    cut = L - TAIL
    h = torch.empty(1, C, N, device="cuda")
    lz.lizard_scan_fwd(data["x"][:, :cut], data["dt"][:, :cut], A, Bm[:, :cut], Cm[:, :cut], h_out=h)
    part = (tail(data["x"]), tail(data["dt"]), A, tail(Bm), tail(Cm))
    y2, st2 = lz.lizard_scan_fwd(*part, h0=h, save_states=True)

    def close(a, b):
        tol = 2 * 2.0 ** -8 * b.abs() + 16 * TAIL * 2.0 ** -24 * b.abs().max()
        assert ((a - b).abs() <= tol).all()

    close(tail(y).float(), y2.float())
    del y
    got = lz.lizard_scan_bwd(data["x"], data["dt"], A, Bm, Cm, data["dy"], states)
    want = lz.lizard_scan_bwd(*part, tail(data["dy"]), st2, h0=h)
    for k in ("dx", "ddt", "dBm", "dCm"):
        close(tail(got[k]).float(), want[k].float())
