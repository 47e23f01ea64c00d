"""Operators called from several host threads."""
import ctypes
import sys
import threading

import pytest
import torch

import test_gpu_few as few
import test_gpu_norm_residual as nr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import binding
    return binding


def in_new_threads(*jobs):
    """Runs each job in a thread of its own; raises what one raised."""
    raised = []

    def work(job):
        try:
            job()
        except Exception as e:                      # noqa: BLE001 (raised below)
            raised.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if raised:
        raise raised[0]


@pytest.mark.parametrize("kind", few.KINDS)
def test_first_call_of_a_thread_makes_tensor_maps(B, kind):
    """A thread whose first CUDA call is one of ours."""
    p = few.make(B, kind, 2, 256, 32, 2, 128, seed=3)
    few.call(B, p)
    first = p["out"].clone()
    p["out"].zero_()
    torch.cuda.synchronize()
    s = torch.cuda.current_stream().cuda_stream
    in_new_threads(lambda: few.call(B, p, stream=s))
    torch.cuda.synchronize()
    assert torch.equal(p["out"], first)


def in_turn_with_another_size(B, calls, n):
    """n calls of each (function, arguments, stream) in a thread of its own, back to back: what they gave."""
    start, failed = threading.Barrier(len(calls)), [[] for _ in calls]

    def many(f, args, stream, bad):
        start.wait()
        for i in range(n):
            if f(*args, stream.cuda_stream) != B.MOE_OK and len(bad) < 3:
                bad.append(B.get_last_error())
            if i % 500 == 499:
                stream.synchronize()
        stream.synchronize()

    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        in_new_threads(*(lambda c=c, b=b: many(*c, b) for c, b in zip(calls, failed)))
    finally:
        sys.setswitchinterval(interval)
    return failed


@pytest.mark.parametrize("kind", few.KINDS)
def test_few_tokens_of_two_sizes(B, kind):
    """Two threads, each on its own stream and workspace: every call goes through, with the bits of a
    call alone."""
    ps = [few.make(B, kind, 2, 256, E, 2, 128, seed=E) for E in (32, 1024)]
    first, calls = [], []
    for p in ps:
        few.call(B, p)
        first.append(p["out"].clone())
        p["out"].zero_()
        t = [p["x"], p["w_router"], p["bias"], *p["w13"][:2], *p["w2"][:2], *p["w13s"][:2], *p["w2s"][:2],
             p["out"], p["idx"], p["w"], p["ws"]]
        p["c"] = p["cfg"].c()
        calls.append((B.lib().moe_forward_few, [ctypes.byref(p["c"])] +
                      [None if v is None else v.data_ptr() for v in t] + [p["ws"].numel()],
                      torch.cuda.Stream()))
    torch.cuda.synchronize()
    assert in_turn_with_another_size(B, calls, 5000) == [[], []]
    for p, f in zip(ps, first):
        B.moe_check_device_status(p["ws"])
        assert torch.equal(p["out"], f)


@pytest.mark.parametrize("sizes", [(2568, 5120), (5128, 6144), (6152, 8192), (8200, 16384)])
def test_norms_of_two_sizes(B, sizes):
    T, forward, backward, ref, keep = 1, [], [], [], []
    for H in sizes:
        d = nr.make(T, H, "token", True, seed=2)
        h_out, u, rstd = nr.forward(B, d, T, H, "token", 1.0)
        want = {"h_out": h_out, "u": u, **nr.backward(B, d, T, H, "token", 1.0, rstd)}
        got = {n: torch.zeros_like(v) for n, v in want.items()}
        ref.append((want, got))
        cfg, ws = nr.cfg_of(B, T, H), B.alloc_norm_residual_workspace(nr.cfg_of(B, T, H))
        c = cfg.c()
        keep.append((c, d, rstd, ws))
        p = lambda v: v.data_ptr()  # noqa: E731
        head = [ctypes.byref(c), p(d["h"]), p(d["y"]), p(d["gamma_post"]), p(d["gate"]), B.MOE_GATE_TOKEN, 1.0]
        forward.append((B.lib().moe_norm_residual, head + [
            nr.EPS, p(d["gamma_pre"]), p(got["h_out"]), p(got["u"]), None], torch.cuda.Stream()))
        backward.append((B.lib().moe_norm_residual_backward, head + [
            p(d["gamma_pre"]), p(rstd), p(d["dh_out"]), p(d["du"]), p(got["dh"]), p(got["dy"]), p(got["dgate"]),
            p(got["dgamma_post"]), p(got["dgamma_pre"]), p(ws), ws.numel()], torch.cuda.Stream()))
    torch.cuda.synchronize()
    assert in_turn_with_another_size(B, forward, 20000) == [[], []]
    assert in_turn_with_another_size(B, backward, 20000) == [[], []]
    for want, got in ref:
        for n in want:
            assert torch.equal(want[n], got[n]), n
