"""ExpertTrainLayer's plumbing on the CPU, with the calls themselves left out: what it allocates and in which order, and
what it refuses."""
import pytest
import torch

import asynchronous_moe_expert_amd as M
from asynchronous_moe_expert_amd import _native as N

T, E, K, H, I = 6, 4, 2, 64, 32
CALLS = ("moe_route", "moe_sort_rows", "moe_expert_matmul", "moe_swiglu", "moe_merge_rows", "moe_merge_rows_backward",
         "moe_expert_matmul_backward", "moe_swiglu_backward", "moe_route_backward")


@pytest.fixture
def calls(monkeypatch):
    """The names of the calls that a run makes, in order; none of them does anything."""
    made = []
    for name in CALLS:
        monkeypatch.setattr(N, name, lambda *a, name=name, **k: made.append(name))
    return made


class Stream:
    def __init__(self, handle, calls):
        self.cuda_stream, self.calls = handle, calls

    def wait_stream(self, other):
        self.calls.append(f"{self.cuda_stream} waits for {other.cuda_stream}")

    def record_stream(self, *a):
        pass


def layer(dtype=M.MOE_F32, **how):
    return M.ExpertTrainLayer(E, H, I, K, dtype, T, device="cpu", **how)


def inputs(dtype=torch.float32):
    x, logits = torch.zeros(T, H, dtype=dtype), torch.zeros(T, E)
    return [x, logits, torch.zeros(E, 2 * I, H, dtype=dtype), torch.zeros(E, H, I, dtype=dtype), torch.zeros(T, H, dtype=dtype)]


def gradients(dtype=torch.float32):
    x, logits, w_gu, w_d, _ = inputs(dtype)
    return [torch.zeros_like(x), x, logits, w_gu, w_d]


@pytest.fixture
def streams(monkeypatch, calls):
    """A current stream (handle 5) and another one (77)."""
    current, other = Stream(5, calls), Stream(77, calls)
    monkeypatch.setattr(N, "_raw_stream", lambda index: 5)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda at=None: current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: Stream(handle, calls))
    monkeypatch.setattr(N, "_capturing", lambda s: False, raising=False)
    return current, other


@pytest.mark.parametrize("raw", [True, False])
def test_buffers_made_late_are_not_used_before_the_current_stream_is_done_with_them(calls, streams, raw):
    """The allocator hands out what was freed on the current stream, whose work may still be using it."""
    one, stream = layer(), 77 if raw else streams[1]
    one.run(*inputs(), train=True, stream=stream)
    assert calls[0] == "77 waits for 5" and calls[1:].count("77 waits for 5") == 0
    del calls[:]
    one.backward(*gradients(), stream=stream)
    assert calls[0] == "77 waits for 5" and calls[1:].count("77 waits for 5") == 0
    del calls[:]
    one.run(*inputs(), train=True, stream=stream)  # they are there
    one.backward(*gradients(), stream=stream)
    assert not [c for c in calls if "waits" in c]


def test_no_wait_where_there_is_one_stream_or_nothing_to_make(calls, streams):
    for stream in (None, 5, streams[0]):
        one = layer()
        one.run(*inputs(), train=True, stream=stream)
        one.backward(*gradients(), stream=stream)
    one = layer()
    one.run(*inputs(), stream=77)  # not a training run
    assert not [c for c in calls if "waits" in c]


def test_a_capture_that_cannot_wait_is_refused(calls, streams, monkeypatch):
    monkeypatch.setattr(N, "_capturing", lambda s: s.cuda_stream == 77, raising=False)
    one = layer()
    with pytest.raises(M.MoeError, match="captured"):
        one.run(*inputs(), train=True, stream=77)
    assert not calls
    one.run(*inputs(), train=True)
    one.run(*inputs(), train=True, stream=77)


def test_later_buffers_are_made_where_the_layer_is(calls, monkeypatch):
    """A device without a number is the current one when the layer is built, whatever it is later on."""
    real, asked = torch.empty, []

    def empty(*size, device=None, **k):
        asked.append(torch.device(device))
        return real(*size, device="meta" if torch.device(device).type == "cuda" else device, **k)

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "zeros", lambda *size, device=None, **k: empty(*size, device=device, **k))
    one = M.ExpertTrainLayer(E, H, I, K, M.MOE_F32, T, device="cuda")
    monkeypatch.undo()
    made = []
    monkeypatch.setattr(torch, "empty", lambda *size, device=None, **k: made.append(torch.device(device)) or
                        real(*size, device="meta", **k))
    one._rows(H)
    assert asked and made == [one.y.device]
