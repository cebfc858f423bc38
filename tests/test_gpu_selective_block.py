"""The example block (examples/selective_block.py): prompt, packed prompt, single tokens and the
training step agree with each other and with differences."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def mod():
    import selective_block

    return selective_block


def inputs(B, L, dm, dtype, n=2, seed=3):
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(B, L, dm, generator=g, device="cuda").to(dtype) for _ in range(n)]


SIZES = dict(dm=48, C=64, N=16, G=2, K=4, heads=4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 40])
def test_prompt_then_tokens_is_the_whole_prompt(mod, dtype, L):
    """The token after a prompt goes through the single-token calls.  fp32: the two paths add the
    same terms, rounded at most 16 times a token each (2^-24), through a block whose outputs are
    of order one; bf16: each of the block's seven intermediate tensors may round to the other
    neighbour (2^-8 of values up to 4)."""
    tp = torch.float32 if dtype == "f32" else torch.bfloat16
    blk = mod.SelectiveBlock(dtype=tp, **SIZES)
    u, r = inputs(3, L + 3, 48, tp)
    rr, uu = blk.prompt(u, r)
    conv = torch.zeros(3, 3, 64, dtype=tp, device="cuda")
    state = torch.zeros(3, 64, 16, device="cuda")
    blk.prompt(u[:, :L].contiguous(), r[:, :L].contiguous(), conv_state=conv, state=state)
    # the states move to slots of a cache, in another order
    slots = torch.tensor([4, 1, 2], dtype=torch.int64, device="cuda")
    cc, cs = torch.zeros(6, 3, 64, dtype=tp, device="cuda"), torch.zeros(6, 64, 16, device="cuda")
    cc[slots], cs[slots] = conv, state
    for t in range(L, L + 3):
        r1, u1 = blk.step(u[:, t], r[:, t].contiguous(), cc, cs, slots=slots)
        tol = 16 * (L + 3) * 2.0 ** -24 * 64 if dtype == "f32" else 7 * 4 * 2.0 ** -8
        assert (r1.float() - rr[:, t].float()).abs().max() <= tol
        assert (u1.float() - uu[:, t].float()).abs().max() <= tol


def test_packed_prompt_equals_each_alone(mod):
    blk = mod.SelectiveBlock(dtype=torch.float32, **SIZES)
    lens = [5, 1, 70, 0, 130]
    u, r = inputs(1, sum(lens), 48, torch.float32)
    conv = torch.zeros(len(lens), 3, 64, device="cuda")
    state = torch.zeros(len(lens), 64, 16, device="cuda")
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    rr, _ = blk.prompt(u, r, cu_seqlens=cu, conv_state=conv, state=state)
    for i, n in enumerate(lens):
        if n == 0:
            assert (state[i] == 0).all()
            continue
        c1, s1 = torch.zeros(1, 3, 64, device="cuda"), torch.zeros(1, 64, 16, device="cuda")
        r1, _ = blk.prompt(u[:, cu[i]:cu[i + 1]].contiguous(), r[:, cu[i]:cu[i + 1]].contiguous(), conv_state=c1, state=s1)
        tol = 16 * n * 2.0 ** -24 * 64
        assert (r1 - rr[:, cu[i]:cu[i + 1]]).abs().max() <= tol
        assert (s1[0] - state[i]).abs().max() <= tol * 4
        # the projections are two products of different shapes: 48 terms each, in either order
        terms = (u[:, cu[i]:cu[i + 1]].abs() @ blk.W_in.abs().t()).max().item()
        assert (c1[0] - conv[i]).abs().max() <= 2 * 48 * 2.0 ** -24 * terms


def test_training_gradients_by_differences(mod):
    """Central differences along random directions, fp32.  The function value is a sum of 2 x 24 x 96
    terms of order one computed to about 2^-20 relative; with a step of 1e-2 its rounding gives
    an error of 96 x 48 x 2^-20 / 2e-2 = 0.2 on slopes of order 100, and the third derivatives'
    part is of order 1e-4 of the slope."""
    blk = mod.SelectiveBlock(dtype=torch.float32, **SIZES)
    u, r, dr, du = inputs(2, 24, 48, torch.float32, n=4)

    def value():
        rr, uu = blk.prompt(u, r)
        return ((rr.double() * dr.double()).sum() + (uu.double() * du.double()).sum()).item()

    *_, g = blk.train(u, r, dr, du)
    places = dict(u=u, r=r, W_in=blk.W_in, W_out=blk.W_out, **blk.p)
    gen = torch.Generator("cuda").manual_seed(9)
    for name, t in places.items():
        v = torch.randn(t.shape, generator=gen, device="cuda")
        v /= v.norm()
        slope = (g[name].double() * v.double()).sum().item()
        keep, eps = t.clone(), 1e-2
        t.copy_(keep + eps * v)
        hi = value()
        t.copy_(keep - eps * v)
        lo = value()
        t.copy_(keep)
        size = g[name].double().norm().item()
        assert abs((hi - lo) / (2 * eps) - slope) <= 0.2 + 2e-3 * size, name


def test_training_step_repeats_bit_for_bit_in_a_graph(mod):
    """The whole step, forward and backward, captured into a CUDA graph while an earlier eager
    step's tensors are alive, gives the eager step's gradients."""
    blk = mod.SelectiveBlock(**SIZES)
    u, r, dr, du = inputs(2, 80, 48, torch.bfloat16, n=4)
    eager = blk.train(u, r, dr, du)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        blk.train(u, r, dr, du)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = blk.train(u, r, dr, du)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])
    for k in ("w", "bias", "A", "D", "dt_bias", "w_post", "scale", "w_pre"):
        assert torch.equal(out[2][k], eager[2][k]), k


def test_example_runs(mod, capsys):
    mod.main()
    assert "gradients:" in capsys.readouterr().out
