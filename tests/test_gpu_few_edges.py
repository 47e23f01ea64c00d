"""The few-token layer (moe_forward_few) where its inputs or its shape reach an edge:
stages of several widths in one slot of its ring."""
import pytest
import torch

from test_gpu_few import KINDS, call, check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import binding
    return binding


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [4, 9, 16])
def test_wide_and_narrow_stages_share_slots(B, kind, T):
    """Two experts with every token between experts with a few: the activations of a narrow stage lie
    where a full stage's weights land next.  The same bits from every call, and right ones."""
    bias = torch.zeros(32, device="cuda")
    bias[[11, 30]] = 3.0
    p = make(B, kind, T, 2304, 32, 6, 256, bias=bias, seed=61)
    call(B, p)
    check(B, p)
    first = p["out"].clone()
    for _ in range(50):
        call(B, p)
        assert torch.equal(p["out"], first)
