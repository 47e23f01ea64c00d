"""What the calls that look their tensors over take for a byte: torch's own types too.  No GPU is needed:
a tensor that passes the look at its type is refused for where it is."""
import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import build
    build.build()
    from sigmoid_top_routing_warp_b200 import binding
    return binding


def test_byte_types(B):
    for t in (torch.uint8, torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.float4_e2m1fn_x2):
        v = torch.zeros(64, dtype=torch.uint8).view(t)
        with pytest.raises(ValueError, match="current CUDA device"):
            B._look("f", (("q", v, torch.uint8, 64),))
        with pytest.raises(ValueError, match="elements"):
            B._look("f", (("q", v, torch.uint8, 32),))
    for t in (torch.int8, torch.float8_e5m2, torch.bool):
        with pytest.raises(TypeError, match="q must be"):
            B._look("f", (("q", torch.zeros(64, dtype=torch.uint8).view(t), torch.uint8, 64),))
    with pytest.raises(TypeError, match="x must be"):
        B._look("f", (("x", torch.zeros(64, dtype=torch.uint8), torch.bfloat16, 64),))


def test_addresses_and_none_pass(B):
    assert B._look("f", (("x", 4096, torch.bfloat16, 8), ("y", None, torch.uint8, 8))) == [4096, None]
