"""Operators called from several host threads."""
import threading

import pytest
import torch

import test_gpu_few as few

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
