"""The token mixer's calls on a stream of their own: workspaces and outputs that the binding allocates
belong to that stream."""
import pytest

from test_gpu_selective_edges import memory_stays, outputs_stay

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

B, L, H, DH, W = 2, 256, 2, 64, 32


@pytest.fixture(scope="module")
def lz():
    from gated_linear_sliding_gb300 import lizard

    lizard.load()
    return lizard


@pytest.fixture(scope="module")
def calls(lz):
    g = torch.Generator("cuda").manual_seed(3)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    q, k, v, ga, dy = (normal(B, L, H, DH) for _ in range(5))
    Wf, sinks = normal(H, DH, DH // 2), normal(H, 4, dtype=torch.float32)
    args = (q, k, v, ga, Wf, sinks)
    lse = torch.empty(B, L, H, device="cuda")
    y = lz.lizard_attn_fwd(*args, W, lse=lse)
    packed = tuple(t.flatten(0, 1) for t in (q, k, v, ga)) + (Wf, sinks)
    cu = [0, 100, B * L]
    plse = torch.empty(B * L, H, device="cuda")
    py = lz.lizard_attn_fwd_varlen(*packed, W, cu, lse=plse)
    x, Wp = normal(B, L, 128), normal(4 * H * DH, 128)
    kept = []

    def step(**m):  # the states are the caller's and alive after the call
        S, z = (torch.zeros(s, device="cuda") for s in ((B, H, DH, DH), (B, H, DH)))
        kc, vc = (torch.zeros(B, H, W + 1, DH, dtype=q.dtype, device="cuda") for _ in range(2))
        kept.append((S, z, kc, vc))
        torch.cuda.current_stream().synchronize()
        tok = tuple(t[:, 0] for t in (q, k, v, ga))
        tok = tuple(t.contiguous() for t in tok)
        kept.append(tok)
        torch.cuda.current_stream().synchronize()
        return [lz.lizard_decode_step(0, *tok, Wf, sinks, S, z, kc, vc, W, **m)]

    yield dict(
        fwd=lambda **m: [lz.lizard_attn_fwd(*args, W, **m)],
        fwd_varlen=lambda **m: [lz.lizard_attn_fwd_varlen(*packed, W, cu, **m)],
        bwd=lambda **m: list(lz.lizard_attn_bwd(*args, y, lse, dy, W, **m).values()),
        bwd_varlen=lambda **m: list(lz.lizard_attn_bwd_varlen(*packed, py, plse, dy.flatten(0, 1), W, cu, **m).values()),
        decode=step,
        proj=lambda **m: list(lz.lizard_qkvg_proj(x, Wp, H, H, DH, DH, **m)),
        proj_bwd=lambda **m: list(lz.lizard_qkvg_proj_bwd(x, Wp, q, k, v, ga, **m)),
    )


CALLS = ["fwd", "fwd_varlen", "bwd", "bwd_varlen", "decode", "proj", "proj_bwd"]


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_on_another_stream(calls, name):
    memory_stays(calls[name])


@pytest.mark.parametrize("name", CALLS)
def test_outputs_of_a_call_on_another_stream(calls, name):
    outputs_stay(calls[name])
