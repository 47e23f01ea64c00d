"""The norms around a block, with gate and residual scale: values that are not finite, and more rows
than any grid has blocks."""
import math

import pytest
import torch

from test_gpu_norm_residual import (MODES, backward, cfg_of, check_backward, check_forward, forward,
                                    make)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import binding
    return binding


@pytest.mark.parametrize("H", [264, 2568, 6152, 9000, 16384])
@pytest.mark.parametrize("gate", MODES)
def test_without_the_next_norm_h_reaches_no_gradient(B, H, gate):
    """D is dh' alone then: an infinity or a NaN in h leaves every gradient as the formula has it."""
    T = 5
    d = make(T, H, gate, False, seed=11)
    _, _, rstd = forward(B, d, T, H, gate, 0.75)
    d["h"][1, 3] = math.inf
    d["h"][2, H - 1] = -math.inf
    d["h"][4, 77] = math.nan
    got = backward(B, d, T, H, gate, 0.75, rstd)
    torch.cuda.synchronize()
    check_backward(d, T, H, gate, 0.75, rstd, got)


@pytest.mark.parametrize("H", [264, 2568, 6152])
def test_non_finite_rows_stay_in_their_rows(B, H):
    """With the next norm an infinity in h or in a gradient belongs to the gradients of its row and to
    the sums over the rows."""
    T = 7
    d = make(T, H, "token", True, seed=12)
    _, _, rstd = forward(B, d, T, H, "token", 1.0)
    clean = backward(B, d, T, H, "token", 1.0, rstd)
    d["h"][2, 5] = math.inf
    d["du"][4, 6] = math.nan
    got = backward(B, d, T, H, "token", 1.0, rstd)
    torch.cuda.synchronize()
    for n in ("dh", "dy", "dgate"):
        for t in (0, 1, 3, 5, 6):
            assert torch.equal(got[n][t], clean[n][t])
        assert not bool(got[n][2].isfinite().any()) and not bool(got[n][4].isfinite().any())


def test_no_rows_leave_zero_sums(B):
    """With no rows the sums are zero whatever the gate and the weights are."""
    H = 64
    d = make(0, H, "channel", True)
    d["gate"][3], d["gate"][5], d["gamma_post"][7] = math.inf, math.nan, -math.inf
    got = backward(B, d, 0, H, "channel", 1.0, torch.empty((2, 0), device="cuda"))
    torch.cuda.synchronize()
    for n in ("dgamma_post", "dgamma_pre", "dgate"):
        assert torch.equal(got[n], torch.zeros(H, device="cuda"))


@pytest.mark.parametrize("T,H", [(9700, 64), (9603, 264), (9480, 512), (4801, 1288), (2401, 2560)])
@pytest.mark.parametrize("gate", MODES)
def test_rows_walked_at_several_blocks_an_sm(B, T, H, gate):
    """Short rows get several blocks of an SM, each with eight rows at least in the backward pass: with
    more rows than that every block walks on, forward too, and the workspace is used to its end and no
    further."""
    d = make(T, H, gate, gate != "none", seed=13)
    h_out, u, rstd = forward(B, d, T, H, gate, 0.75)
    cfg = cfg_of(B, T, H)
    n = B.norm_residual_workspace_size(cfg)
    assert T // 8 >= n // (8 * H) > 148              # rows of partial sums: two of H floats a block
    room = torch.full((n + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
    got = backward(B, d, T, H, gate, 0.75, rstd, ws=room[:n])
    torch.cuda.synchronize()
    check_forward(d, T, H, 0.75, h_out, u, rstd)
    check_backward(d, T, H, gate, 0.75, rstd, got)
    assert bool((room[n:] == 0xa5).all())
