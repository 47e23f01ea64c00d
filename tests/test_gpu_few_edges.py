"""The few-token layer (moe_forward_few) where its inputs or its shape reach an edge:
stages of several widths in one slot of its ring, a call that
gives up."""
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


@pytest.mark.parametrize("kind", KINDS)
def test_a_stalled_call_leaves_nothing_behind(B, kind):
    """A call that gives up waits for its own copies first: with shared and routed experts, a call of another
    size that follows at once gives its bits."""
    p = make(B, kind, 3, 1024, 32, 4, 256, n_shared=2, seed=67)
    q = make(B, kind, 8, 640, 32, 4, 128, seed=71)
    call(B, p)
    call(B, q)
    first, other = p["out"].clone(), q["out"].clone()
    p["cfg"].flags = B.MOE_FLAG_TEST_STALL
    call(B, p)
    q["out"].zero_()
    call(B, q)
    with pytest.raises(B.MoeError) as err:
        B.moe_check_device_status(p["ws"])
    assert err.value.status == B.MOE_ERR_TIMEOUT
    B.moe_check_device_status(q["ws"])
    assert torch.equal(q["out"], other)
    p["cfg"].flags = 0
    call(B, p)
    check(B, p)
    assert torch.equal(p["out"], first)
