"""Gradients of no rows are zeros whatever their size: past 2^32 pieces of 16 bytes too."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_large_gradient_of_no_rows():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep
    N, K = 2 ** 17 + 8, 2 ** 17       # 64 GiB and a little
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GiB")
    gw = torch.full((N, K), 1.0, device="cuda")
    gb = torch.full((N,), 1.0, device="cuda")
    sh = ep.ep_linear_shape(0, K, N, ep.EP_ACT_NONE, 0, 0, 1)
    P = ctypes.c_void_p
    rc = ep.load().ep_linear_backward(ctypes.byref(sh), None, None, None, None, None, P(gw.data_ptr()), P(gb.data_ptr()),
                                      None, 0, P(torch.cuda.current_stream().cuda_stream))
    assert rc == ep.EP_OK
    assert not gb.any()
    for part in gw.split(2 ** 13):
        assert not part.any()
    del gw, part
    torch.cuda.empty_cache()
