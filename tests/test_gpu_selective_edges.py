"""The selective block on the GPU where its calls meet odd sizes, other streams and threads, and values
far out."""
import numpy as np
import pytest

from test_gpu_selective import Draw, check, offsets

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lz():
    from gated_linear_sliding_gb300 import lizard

    lizard.load()
    return lizard


# ------------------------------------------------------------------------------- states in place


@pytest.mark.parametrize("B,L,C,N,lens", [(1, 600, 1001, 16, None), (1, 600, 9, 4, None), (3, 1500, 37, 8, None),
                                          (1, 700, 13, 16, [300, 0, 1, 399])])
def test_scan_in_place_state_of_odd_channels(lz, B, L, C, N, lens):
    """h_out is h0, the time axis is cut and the channels are odd: the same bits as with two arrays."""
    d = Draw(11, "f32")
    x, dt = d(B, L, C)[0], d(B, L, C, shift=-1.0)[0]
    Bm, Cm = d(B, L, 1, N)[0], d(B, L, 1, N)[0]
    A = d.dev(-np.exp(d.rng.normal(size=(C, N))))[0]
    h0 = d(B if lens is None else len(lens), C, N)[0]
    cu = offsets(lens)
    h, st = torch.empty_like(h0), h0.clone()
    y = lz.lizard_scan_fwd(x, dt, A, Bm, Cm, h0=h0, h_out=h, cu_seqlens=cu)
    y2 = lz.lizard_scan_fwd(x, dt, A, Bm, Cm, h0=st, h_out=st, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, st)
