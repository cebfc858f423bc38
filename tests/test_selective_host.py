"""The selective block without a GPU: workspace layouts and what the binding checks and does before a
launch."""
import pytest

from gated_linear_sliding_gb300 import _build
from gated_linear_sliding_gb300 import lizard as lz

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return lz.load()


@pytest.mark.parametrize("B,C,N,L", [(1, 1001, 16, 600), (1, 9, 4, 600), (3, 37, 8, 1500), (2, 5, 64, 700), (1, 7, 3, 400),
                                     (1, 1000, 16, 600)])
def test_copied_states_begin_on_16_bytes(lib, B, C, N, L):
    """Where h_out is h0 and the time axis is cut, the states are copied to the workspace's end and
    read from there in pieces of four values."""
    d = lz.lizard_scan_dims(B=B, L=L, C=C, N=N, G=1, dtype=0, softplus=1)
    ws = lz.lizard_scan_fwd_workspace(d)
    assert ws > 256 + 4 * B * C * N  # cut into segments
    assert (ws - 4 * B * C * N) % 16 == 0


@pytest.mark.parametrize("dtype,res", [(torch.bfloat16, torch.float16), (torch.bfloat16, torch.float64),
                                       (torch.bfloat16, torch.int16), (torch.float32, torch.bfloat16),
                                       (torch.float32, torch.float64)])
def test_residual_stream_of_another_type_is_refused(dtype, res):
    """The library knows the residual stream as o's type or fp32; anything else would be read as one
    of them."""
    o, r = torch.zeros(3, 8, dtype=dtype), torch.zeros(3, 8, dtype=res)
    for call in (lambda: lz.lizard_block_norm_fwd(o, r=r),
                 lambda: lz.lizard_block_norm_fwd(o, r_out=r),
                 lambda: lz.lizard_block_norm_bwd(o, r=r, dr_out=r),
                 lambda: lz.lizard_block_norm_bwd(o, dr_out=r)):
        with pytest.raises(ValueError, match="residual stream: dtype"):
            call()


class OnDevice:
    """Stands for a CUDA tensor of a device."""
    is_cuda = True

    def __init__(self, index, *shape):
        self.device, self.shape, self.dtype = torch.device("cuda", index), torch.Size(shape), torch.float32

    def is_contiguous(self):
        return True


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Kernels are launched on the current device; a tensor of another one must not get there."""
    monkeypatch.setattr(lz, "_gpus", lambda: 2, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def no_launch(*a):
        raise AssertionError("reached the library")

    monkeypatch.setattr(lz, "load", no_launch)
    x0, x1 = OnDevice(0, 1, 5, 8), OnDevice(1, 1, 5, 8)
    w0, w1 = OnDevice(0, 8, 4), OnDevice(1, 8, 4)
    b0, b1 = OnDevice(0, 1, 5, 1, 4), OnDevice(1, 1, 5, 1, 4)
    o0, o1 = OnDevice(0, 5, 8), OnDevice(1, 5, 8)
    q0, q1 = OnDevice(0, 1, 5, 2, 64), OnDevice(1, 1, 5, 2, 64)
    for call in (lambda: lz.lizard_conv_fwd(x1, w1),
                 lambda: lz.lizard_conv_fwd(x0, w1),
                 lambda: lz.lizard_conv_fwd(x0, w0, workspace=w1),
                 lambda: lz.lizard_conv_bwd(x0, w0, None, x1),
                 lambda: lz.lizard_conv_step(o0, w0, None, OnDevice(1, 5, 3, 8)),
                 lambda: lz.lizard_scan_fwd(x0, x0, w0, b0, b0, z=x1),
                 lambda: lz.lizard_scan_bwd(x0, x0, w0, b0, b1, x0, w0),
                 lambda: lz.lizard_scan_step(o0, o0, w0, b0, b0, OnDevice(1, 5, 8, 4)),
                 lambda: lz.lizard_block_norm_fwd(o0, r=o1),
                 lambda: lz.lizard_block_norm_bwd(o1, dr_out=o1),
                 lambda: lz.lizard_attn_fwd(q0, q0, q0, q1, w0, w0, 4)):
        with pytest.raises(ValueError, match="current device is cuda:0"):
            call()


class AsCuda(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    is_cuda = True


def as_cuda(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(AsCuda)


@pytest.mark.parametrize("kind", ["host", "strided"])
def test_workspaces_that_kernels_cannot_use_are_refused(monkeypatch, kind):
    """The library takes a workspace's address and size; it cannot see that it is on the host or has
    gaps."""
    u8 = torch.uint8
    ws = torch.zeros(1 << 16, dtype=u8) if kind == "host" else as_cuda(1 << 17, dtype=u8)[::2]

    class Library:  # sizes are asked for, launches are not to come
        def __getattr__(self, name):
            return lambda *a: 0 if name.endswith(("_workspace", "_bytes")) else pytest.fail(f"reached {name}")

    monkeypatch.setattr(lz, "load", Library)
    x, w, b = as_cuda(1, 5, 8), as_cuda(8, 4), as_cuda(1, 5, 1, 4)
    o, state, bs, h = as_cuda(5, 8), as_cuda(5, 3, 8), as_cuda(5, 1, 4), as_cuda(5, 8, 4)
    q, Wf, sinks = as_cuda(1, 5, 2, 64), as_cuda(2, 64, 32), as_cuda(2, 4)
    t, S, z, kc = as_cuda(1, 2, 64), as_cuda(1, 2, 64, 64), as_cuda(1, 2, 64), as_cuda(1, 2, 5, 64)
    xb, W, qb = (as_cuda(*n, dtype=torch.bfloat16) for n in ((1, 5, 16), (512, 16), (1, 5, 2, 64)))
    for call in (lambda: lz.lizard_conv_fwd(x, w, workspace=ws),
                 lambda: lz.lizard_conv_bwd(x, w, None, x, workspace=ws),
                 lambda: lz.lizard_conv_step(o, w, None, state, workspace=ws),
                 lambda: lz.lizard_scan_fwd(x, x, w, b, b, workspace=ws),
                 lambda: lz.lizard_scan_bwd(x, x, w, b, b, x, as_cuda(0, dtype=u8), workspace=ws),
                 lambda: lz.lizard_scan_step(o, o, w, bs, bs, h, workspace=ws),
                 lambda: lz.lizard_block_norm_bwd(o, dr_out=o, workspace=ws),
                 lambda: lz.lizard_attn_fwd(q, q, q, q, Wf, sinks, 4, workspace=ws),
                 lambda: lz.lizard_attn_bwd(q, q, q, q, Wf, sinks, q, as_cuda(1, 5, 2), q, 4, workspace=ws),
                 lambda: lz.lizard_decode_step(0, t, t, t, t, Wf, sinks, S, z, kc, kc, 4, workspace=ws),
                 lambda: lz.lizard_qkvg_proj(xb, W, 2, 2, 64, 64, q=qb, k=qb, v=qb, g=qb, workspace=ws),
                 lambda: lz.lizard_qkvg_proj_bwd(xb, W, qb, qb, qb, qb, dW=as_cuda(512, 16), workspace=ws)):
        with pytest.raises(ValueError, match="workspace must be"):
            call()
