"""Further host-side refusals and the plans' handling of streams and devices; these run without a GPU."""
import ctypes

import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

P = ctypes.c_void_p(256)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from semi_autoregressive_drafting_gb300 import _build, _lib
    _build.build()
    return _lib.load()


@pytest.mark.parametrize("T,ok", [(3.5e-39, False), (2.95e-39, False), (4.2e-39, False), (4.3e-39, True),
                                  (1e-38, True), (3e38, True)])
def test_temperature_whose_scale_overflows(lib, T, ok):
    # log2(e) / T is infinite from about 4.24e-39 down, 1 / T only from 2.94e-39
    want = 0 if ok else 1
    assert lib.dspark_token_logprobs(0, 100, T, 0, P, 100, P, 2, P, P, P, P, P, P, P, BIG, None) == want
    assert lib.dspark_token_logprobs_grad(0, 100, T, 0, P, 100, P, P, P, P, P, P, 100, None) == want


class _Stream:
    def __init__(self, handle):
        self.cuda_stream, self.waits = handle, []

    def wait_stream(self, other):
        self.waits.append(other.cuda_stream)


@pytest.fixture
def streams(monkeypatch):
    """Recorded uses of tensors by stream, with stand-ins for the streams themselves."""
    from contextlib import nullcontext
    uses = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: uses.append((t.data_ptr(), s.cuda_stream)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return uses


def _plan(stream):
    """A plan as the constructors leave it: an input, a caller's workspace, a caller's output."""
    x, y, z = torch.zeros(4), torch.zeros(5), torch.zeros(6)
    ws = ds.Workspace.__new__(ds.Workspace)
    ws.buf, ws.nbytes = torch.zeros(256, dtype=torch.uint8), 256
    out = ds.LogprobOutput(y, z, y, y, None, None)
    plan = ds._Plan()
    plan._set("dspark_embedding", (0,), stream, out, (x, ws), torch.device("cuda", 0))
    calls = []
    plan._fn = lambda *a: calls.append(a) or 0
    return plan, calls, {t.data_ptr() for t in (x, y, z, ws.buf)}


def test_what_a_plan_uses_is_recorded_on_its_stream(lib, streams):
    plan, _, used = _plan(_Stream(7))
    assert {p for p, s in streams if s == 7} == used


def test_a_run_on_another_stream_follows_the_plans_and_is_recorded(lib, streams):
    own, other = _Stream(7), _Stream(9)
    plan, calls, used = _plan(own)
    plan.run()
    plan.run(own)
    assert not own.waits and [c[-1] for c in calls] == [7, 7]
    plan.run(other)
    plan.run(other)
    assert [c[-1] for c in calls] == [7, 7, 9, 9]
    assert other.waits == [7]                       # the workspace was cleared on the plan's stream
    assert {p for p, s in streams if s == 9} == used


def test_a_captured_run_waits_for_nothing_outside_the_graph(lib, streams, monkeypatch):
    plan, calls, _ = _plan(_Stream(7))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    other = _Stream(9)
    plan.run(other)
    assert not other.waits and calls[-1][-1] == 9
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    plan.run(other)
    assert other.waits == [7]


# ------------------------------------------------------------------ devices
class _Tensor:
    """A tensor of a device that this machine need not have."""

    is_cuda = True

    def __init__(self, index, shape=(4, 8), dtype=torch.float32):
        self.device, self.shape, self.dtype = torch.device("cuda", index), torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def stride(self, d=None):
        st = [1]
        for n in reversed(self.shape[1:]):
            st.insert(0, st[0] * n)
        return tuple(st) if d is None else st[d]

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        raise AssertionError("no address is taken before the refusal")

    def __getattr__(self, name):
        raise AssertionError(f"{name} is looked at before the refusal")


def _calls(dev):
    x = lambda *shape, dtype=torch.float32: _Tensor(dev, shape, dtype)
    t = x(4, dtype=torch.int32)
    return [lambda: ds.token_logprobs(x(4, 8), t),
            lambda: ds.token_logprobs_grad(x(4, 8), t, x(4, 2), grad_logp=x(4), out=x(4, 8)),
            lambda: ds.embedding(x(9, 8), t),
            lambda: ds.embedding_grad(x(4, 8), t, 9),
            lambda: ds.bias_grad(x(4, 16), x(4, 8), x(16, 8))]


@pytest.mark.parametrize("which", range(5))
def test_tensors_of_a_device_that_is_not_current_are_refused(lib, monkeypatch, which):
    """The library launches on the current device: nothing of another may reach it."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        _calls(1)[which]()


def test_a_workspace_of_another_device_is_refused(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    ws = ds.Workspace.__new__(ds.Workspace)
    ws.buf, ws.nbytes = _Tensor(1, (256,), torch.uint8), 256
    with pytest.raises(ValueError, match="one device"):
        ds._same_device(_Tensor(0), ws)


def test_a_run_under_another_device_is_refused(lib, streams, monkeypatch):
    plan, calls, _ = _plan(_Stream(7))
    plan._index = 1
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        plan.run()
    assert not calls
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    plan.run()
    assert len(calls) == 1
