"""What an AdamW plan keeps alive, checked without a GPU: host arrays that say
they are on one, and entry points that only record the pointers they were
given. An array of numpy memory is gone when its weak reference is."""
import gc
import types
import weakref

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import precision_state_amd as ps  # noqa: E402

DEVICE = torch.device("cuda", 0)


class OnGpu(torch.Tensor):
    device = property(lambda self: DEVICE)
    get_device = lambda self: 0  # noqa: E731
    recorded = []

    def record_stream(self, stream):
        OnGpu.recorded.append((self.data_ptr(), stream.cuda_stream))


def array(n, dtype=np.float32):
    """A tensor on the pretended GPU, and a weak reference to its memory."""
    a = np.zeros(n, dtype)
    return torch.from_numpy(a).as_subclass(OnGpu), weakref.ref(a)


def gone(*refs):
    gc.collect()
    return [r() is None for r in refs]


class Entries:
    """The C entry points; `capturing`: the streams under capture."""

    def __init__(self):
        self.grads = []
        self.capturing = set()
        self.current = 0

    ps_adamw_workspace_size = staticmethod(ps.lib().ps_adamw_workspace_size)
    ps_last_error = staticmethod(ps.lib().ps_last_error)

    def ps_adamw_plan_create(self, arr, n, ws, size, stream, out):
        out._obj.value = 1
        return 0

    def ps_adamw_set_grads(self, h, arr, n, stream):
        self.grads.append(list(arr))
        return 0

    def ps_adamw_grad_norm(self, h, max_norm, scale, stream):
        return 0

    def ps_adamw_step(self, h, groups, n, step, clipped, rounding, stream):
        return 0

    def ps_adamw_plan_destroy(self, h):
        return 0


class FakeStream:
    def __init__(self, raw):
        self.cuda_stream = raw


@pytest.fixture
def entries(monkeypatch):
    e = Entries()

    class on_stream:
        def __init__(self, s):
            self.raw = s.cuda_stream

        def __enter__(self):
            self.old, e.current = e.current, self.raw

        def __exit__(self, *exc):
            e.current = self.old

    def external(raw, device):
        assert raw != 0                                     # torch makes a new stream of a 0
        return FakeStream(raw)
    cuda = types.SimpleNamespace(current_device=lambda: 0, Stream=FakeStream, ExternalStream=external,
                                 default_stream=lambda device: FakeStream(0), stream=on_stream,
                                 is_current_stream_capturing=lambda: e.current in e.capturing)

    class FakeTorch:
        def __getattr__(self, name):
            return getattr(torch, name)

        @staticmethod
        def empty(n, dtype, device):
            return torch.empty(n, dtype=dtype).as_subclass(OnGpu)
    fake = FakeTorch()
    fake.cuda = cuda
    OnGpu.recorded = []
    monkeypatch.setattr(ps, "torch", fake)
    monkeypatch.setattr(ps, "_lib", e)
    monkeypatch.setattr(ps, "_current_raw_stream", lambda index: e.current)
    return e


def record(n=300):
    t, refs = {}, {}
    for k in ("param", "grad", "m", "v"):
        t[k], refs[k] = array(n)
    return ps.AdamWTensor(**t), refs


def test_plans_of_one_list_keep_their_own_gradients(entries):
    rec, refs = record()
    a, b = ps.AdamWPlan([rec]), ps.AdamWPlan([rec])
    new, new_ref = array(300)
    a.set_grads([new])
    rec.grad = None
    assert gone(refs["grad"]) == [False]                    # b's tables still point to them
    b.set_grads([None])
    assert gone(refs["grad"]) == [True]                     # nobody's do
    del new
    assert gone(new_ref) == [False]
    a.close()
    assert gone(new_ref, refs["param"]) == [True, False]
    b.close()
    del rec
    assert gone(refs["param"], refs["m"], refs["v"]) == [True] * 3


def test_set_grads_leaves_the_callers_records_alone(entries):
    rec, _ = record()
    before = rec.grad
    plan = ps.AdamWPlan([rec])
    plan.set_grads([array(300)[0]])
    assert rec.grad is before
    plan.set_grads([None])
    assert rec.grad is before


def test_a_plan_keeps_what_its_tables_address(entries):
    """The caller's record gets other tensors, and a tensor another storage."""
    rec, refs = record()
    plan = ps.AdamWPlan([rec])
    rec.param.data = torch.zeros(300)
    rec.grad.data = torch.zeros(300)
    rec.param = rec.grad = rec.m = rec.v = None
    assert gone(*refs.values()) == [False] * 4
    g, g_ref = array(300)
    plan.set_grads([g])
    g.data = torch.zeros(300)
    del g
    assert gone(g_ref, *refs.values()) == [False, False, True, False, False]
    del plan
    assert gone(g_ref, *refs.values()) == [True] * 5


def test_gradients_of_a_captured_call_live_as_long_as_the_plan(entries):
    """A replay puts a captured call's pointers into the tables again, and until the first replay the tables hold the
    ones from before."""
    rec, refs = record()
    plan = ps.AdamWPlan([rec])
    rec.grad = None
    captured, captured_ref = array(300)
    entries.capturing.add(7)
    plan.set_grads([captured], stream=FakeStream(7))
    del captured
    assert gone(refs["grad"], captured_ref) == [False, False]
    later, later_ref = array(300)
    plan.set_grads([later])
    assert gone(refs["grad"], captured_ref) == [True, False]
    entries.current = 7                                     # the current stream is under capture
    captured, captured_ref2 = array(300)
    plan.set_grads([captured])
    del captured, later
    assert gone(captured_ref, captured_ref2, later_ref) == [False] * 3
    entries.capturing.clear()
    del plan
    assert gone(captured_ref, captured_ref2, later_ref) == [True] * 3


def test_released_arrays_are_recorded_on_the_plans_streams(entries):
    """The allocator must not hand out what the plan lets go before the streams that the plan ran on are done with it."""
    rec, _ = record()
    plan = ps.AdamWPlan([rec])
    first, kept = rec.grad.data_ptr(), [x.data_ptr() for x in (rec.param, rec.m, rec.v)]
    hp = [ps.HParams(algo=ps.ALGO_ADAM)]
    plan.grad_norm(stream=FakeStream(5))
    plan.step(hp, 1, stream=6)
    assert OnGpu.recorded == []                             # nothing has been released
    second, _ = array(300)
    plan.set_grads([second])                                # on stream 0
    assert sorted(OnGpu.recorded) == [(first, 0), (first, 5), (first, 6)]
    OnGpu.recorded.clear()
    plan.set_grads([second])                                # the same array: kept
    assert OnGpu.recorded == []
    workspace = plan.workspace.data_ptr()
    plan.close()
    assert sorted(OnGpu.recorded) == sorted((p, s) for p in kept + [second.data_ptr(), workspace] for s in (0, 5, 6))
    OnGpu.recorded.clear()
    plan.close()
    assert OnGpu.recorded == []


def test_nothing_is_recorded_where_all_is_on_one_stream(entries):
    """Memory that is given and used on one stream is handed out in its order."""
    rec, _ = record()
    entries.current = 4
    plan = ps.AdamWPlan([rec])
    for _ in range(3):
        plan.set_grads([array(300)[0]])
        plan.grad_norm()
        plan.step([ps.HParams(algo=ps.ALGO_ADAM)], 1, stream=4)
    plan.close()
    assert OnGpu.recorded == []


def test_gradients_given_on_another_stream_are_recorded(entries):
    rec, _ = record()
    plan = ps.AdamWPlan([rec])
    plan.grad_norm()
    entries.current = 8                                     # the gradient is this stream's, the calls are on stream 0
    g, _ = array(300)
    plan.set_grads([g], stream=0)
    assert OnGpu.recorded == [(rec.grad.data_ptr(), 0)]
    OnGpu.recorded.clear()
    plan.set_grads([None], stream=0)
    assert OnGpu.recorded == [(g.data_ptr(), 0)]


def test_a_plan_that_is_let_go_records_its_arrays(entries):
    rec, _ = record()
    plan = ps.AdamWPlan([rec])
    entries.current = 9
    plan.step([ps.HParams(algo=ps.ALGO_ADAM)], 1)
    captured, _ = array(300)
    entries.capturing.add(9)
    plan.set_grads([captured])
    entries.capturing.clear()
    workspace = plan.workspace.data_ptr()
    del plan
    gc.collect()
    arrays = [x.data_ptr() for x in (rec.param, rec.grad, rec.m, rec.v, captured)]
    assert sorted(OnGpu.recorded) == sorted((p, 9) for p in arrays + [workspace])


def test_control_block_fields_have_the_names_of_the_docstring(entries):
    plan = ps.AdamWPlan([record()[0]])
    names = ps.AdamWPlan.__doc__.split("in stream order:")[1].split(".")[0].replace("\n", " ").split(",")
    assert len(names) == 6
    for name in names:
        field = getattr(plan, name.strip())
        assert isinstance(field, torch.Tensor) and field.dim() == 0, name
