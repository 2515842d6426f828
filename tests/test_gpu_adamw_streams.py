"""GPU tests of the memory around an AdamW plan: what it releases while another
stream still works on it, gradients of captured calls, and gradients inside its
workspace."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import precision_state_amd as ps  # noqa: E402

N = 5_000_000         # a size of its own in the allocator's cache
SLEEP = 800_000_000   # clock cycles, a third of a second, before the work on the stream that arrays are used on


def fresh(*sizes):
    return [torch.zeros(n, device="cuda") for n in sizes]


def pointers_handed_out(n, count):
    """The next allocations of n floats on the current stream (after a first call they come from the cache)."""
    taken = [torch.empty(n, device="cuda") for _ in range(count)]
    return {x.data_ptr() for x in taken}


@pytest.mark.parametrize("how", ["stream", "integer", "current"])
def test_released_arrays_wait_for_the_stream_that_uses_them(how):
    hp = [ps.HParams(algo=ps.ALGO_ADAM, lr=1e-3)]
    side = torch.cuda.Stream()
    w, g, m, v = fresh(N, N, N, N)
    g.fill_(1e-3)
    new = torch.full((N,), 1e-3, device="cuda")
    plan = ps.AdamWPlan([ps.AdamWTensor(w, g, m, v)])
    torch.cuda.synchronize()
    pointers_handed_out(N, 8)
    old, state = g.data_ptr(), {x.data_ptr() for x in (w, m, v)}
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    # No work for the default stream from here on: it may share a hardware queue with this one and wait for it.
    kw = {"stream": dict(stream=side), "integer": dict(stream=side.cuda_stream), "current": {}}[how]
    with torch.cuda.stream(side if how == "current" else torch.cuda.current_stream()):
        plan.step(hp, 1, **kw)
        plan.set_grads([new], **kw)
        plan.step(hp, 2, **kw)
    del g
    assert old not in pointers_handed_out(N, 3)
    assert not side.query()                                 # its work was still to come
    del w, m, v, plan
    assert not state & pointers_handed_out(N, 4)
    assert not side.query()
    side.synchronize()


def test_a_plan_made_on_a_side_stream_and_run_on_the_default_one():
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        w, g, m, v = fresh(N, N, N, N)
        plan = ps.AdamWPlan([ps.AdamWTensor(w, g, m, v)])
        pointers_handed_out(N, 8)
    side.synchronize()
    state = {x.data_ptr() for x in (w, g, m, v)} | {plan.workspace.data_ptr()}
    torch.cuda._sleep(SLEEP)
    plan.step([ps.HParams(algo=ps.ALGO_ADAM, lr=1e-3)], 1)
    del w, g, m, v, plan
    with torch.cuda.stream(side):
        assert not state & pointers_handed_out(N, 5)
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()


def test_gradients_inside_the_workspace_are_refused():
    w, g, m, v = fresh(64, 64, 64, 64)
    plan = ps.AdamWPlan([ps.AdamWTensor(w, g, m, v)])
    inside = plan.workspace[256:512].view(torch.float32)
    with pytest.raises(ps.PSError, match="grad overlaps the workspace"):
        plan.set_grads([inside])
    g.fill_(2.0)
    plan.grad_norm()                                        # the gradients from before still count
    assert float(plan.norm) == 16.0


def test_captured_set_grads_replays_with_gradients_that_nobody_else_holds():
    """The graph sets its own gradients, eager calls others, in turn; the plan alone holds all of them."""
    n = 100_000
    w, first, m, v = fresh(n, n, n, n)
    first.fill_(2.0 ** -6)
    plan = ps.AdamWPlan([ps.AdamWTensor(w, first, m, v)])
    del first
    captured = torch.full((n,), 2.0 ** -7, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.set_grads([captured])
        plan.grad_norm()
    del captured
    root = np.sqrt(np.float64(n))

    def norm_is(level):
        noise = [torch.full((n,), 1e3, device="cuda") for _ in range(6)]    # into whatever memory is free
        torch.cuda.synchronize()
        del noise
        assert float(plan.norm) == float(np.float32(root * level))          # sums and scale are exact
    plan.grad_norm()
    norm_is(2.0 ** -6)                                      # the ones before the first replay
    for level in (2.0 ** -3, 2.0 ** -4, 2.0 ** -5):
        graph.replay()
        norm_is(2.0 ** -7)
        plan.set_grads([torch.full((n,), level, device="cuda")])
        plan.grad_norm()
        norm_is(level)
