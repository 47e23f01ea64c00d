"""A call that CUDA refuses says so, and the next one is not blamed for it."""
import contextlib

import pytest
import torch

import test_gpu_few as few
import test_gpu_norm_residual as nr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import binding
    return binding


@contextlib.contextmanager
def refusing_stream():
    """A stream whose capture has been spoilt (by waiting for it): it takes no launch until the capture is ended."""
    from cuda.bindings import runtime as rt
    s = torch.cuda.Stream()
    mode = rt.cudaStreamCaptureMode.cudaStreamCaptureModeRelaxed
    assert int(rt.cudaStreamBeginCapture(s.cuda_stream, mode)[0]) == 0
    assert int(rt.cudaStreamSynchronize(s.cuda_stream)[0]) != 0
    rt.cudaGetLastError()
    try:
        yield s.cuda_stream
    finally:
        rt.cudaStreamEndCapture(s.cuda_stream)
        rt.cudaGetLastError()


@pytest.mark.parametrize("first", ["few", "norm", "norm_backward", "mx"])
def test_next_call_is_not_blamed(B, first):
    p = few.make(B, "bf16", 2, 256, 32, 2, 128, seed=5)
    d = nr.make(4, 512, "channel", True, seed=5)
    _, _, rstd = nr.forward(B, d, 4, 512, "channel", 1.0)
    x = torch.randn((4, 64), device="cuda").to(torch.bfloat16)
    q = torch.empty((4, 32), dtype=torch.uint8, device="cuda")
    s = torch.empty((4, 2), dtype=torch.uint8, device="cuda")
    calls = {"few": lambda **kw: few.call(B, p, **kw),
             "norm": lambda **kw: nr.forward(B, d, 4, 512, "channel", 1.0, **kw),
             "norm_backward": lambda **kw: nr.backward(B, d, 4, 512, "channel", 1.0, rstd, **kw),
             "mx": lambda **kw: B.moe_quantize_mx(x, q, s, **kw)}
    for c in calls.values():
        c()
    torch.cuda.synchronize()
    for c in calls.values():
        with refusing_stream() as stream, pytest.raises(B.MoeError) as err:
            calls[first](stream=stream)
        assert err.value.status == B.MOE_ERR_CUDA
        c()
    torch.cuda.synchronize()
    few.check(B, p)
