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


def _bad(good, T_rows=True):
    """Tensors like `good` that a call has to refuse."""
    rows, columns = good.shape[-2:]
    lead = good.shape[:-2]
    new = lambda *s, **k: torch.zeros(*s, dtype=k.get("dtype", good.dtype))  # noqa: E731
    yield "type", new(*good.shape, dtype=torch.float16)
    yield "shape", new(*lead, rows, columns + 8)
    yield "shape", new(*lead, rows + 1, columns)
    yield "strides", new(*lead, columns, rows).transpose(-1, -2)
    yield "overlap", new(*lead, 1, columns).expand(good.shape)
    yield "alignment", new(*lead, rows, columns + 1)[..., :columns]
    flat = new(good.numel() + 1)
    yield "alignment", flat[1:].view(good.shape)
    yield "device", torch.empty(good.shape, dtype=good.dtype, device="meta")
    if lead:
        yield "overlap", new(1, rows, columns).expand(good.shape)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("which", range(5))
def test_a_refused_backward_makes_no_call_and_may_be_made_again(calls, which, dtype):
    """The gradients of the weights may be added to: nothing of them may have been before a later call refuses."""
    one = layer(M.MOE_F32 if dtype == torch.float32 else M.MOE_BF16)
    one.run(*inputs(dtype), train=True)
    good = gradients(dtype)
    for why, t in _bad(good[which]):
        if which == 2 and why == "alignment":  # logits have none
            continue
        del calls[:]
        with pytest.raises(M.MoeError, match="ExpertTrainLayer"):
            one.backward(*good[:which], t, *good[which + 1:], accumulate=True)
        assert not calls, why
    if which in (3, 4) and dtype == torch.float32:
        with pytest.raises(M.MoeError, match="ExpertTrainLayer"):
            one.backward(*good[:which], good[which].bfloat16(), *good[which + 1:])
    one.backward(*good, accumulate=True)
    assert calls[-1] == "moe_route_backward"


def test_gradients_of_every_kind_that_the_calls_take(calls):
    """bf16 layers: f32 gradients of weights, f32 dx; halves of larger tensors, padded rows, logits in any pitch."""
    one = layer(M.MOE_BF16)
    dout, dx, dlogits, dw_gu, dw_d = gradients(torch.bfloat16)
    wide = torch.zeros(E, 2 * I, H + 8)[..., :H]
    both = torch.zeros(E, 2 * H, I)[:, H:]
    for made in ((dout, dx, dlogits, dw_gu.float(), dw_d), (dout.float(), dx.float(), dlogits, wide, both),
                 (dout, dx, torch.zeros(T, E + 3)[:, 1:E + 1], wide.bfloat16(), dw_d.float())):
        one.run(*inputs(torch.bfloat16), train=True)
        one.backward(*made)
    none = M.ExpertTrainLayer(E, H, I, K, M.MOE_BF16, 0, device="cpu")
    none.run(*[t[:0] if t.shape[0] == T else t for t in inputs(torch.bfloat16)], train=True)
    none.backward(dout[:0], dx[:0], dlogits[:0], dw_gu, dw_d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.uint8])
@pytest.mark.parametrize("which", range(5))
def test_a_refused_run_makes_no_call(calls, which, dtype):
    """A run that is refused leaves what the last one keeps for backward()."""
    fp8 = dtype == torch.uint8
    one = layer({torch.float32: M.MOE_F32, torch.bfloat16: M.MOE_BF16, torch.uint8: M.MOE_FP8_E4M3}[dtype])
    good = inputs(dtype)
    if fp8:
        good[4] = good[4].bfloat16()
    scales = dict(x_scale=torch.zeros(T, 1), s_gu=torch.zeros(E, 1, 1), s_d=torch.zeros(E, 1, 1)) if fp8 else {}
    one.run(*good, train=not fp8, **scales)
    for why, t in _bad(good[which]):
        if which == 1 and why not in ("shape", ):  # the rest is moe_route's, the first call
            continue
        del calls[:]
        with pytest.raises(M.MoeError, match="ExpertTrainLayer"):
            one.run(*good[:which], t, *good[which + 1:], **scales)
        assert not calls, why
    if not fp8:
        one.backward(*gradients(dtype))
        return
    for name, t in scales.items():
        for bad in (t.double(), t[1:], t.expand(*t.shape[:-1], 2), t[None], torch.empty(t.shape, device="meta"),
                    t.view(-1)[1:], None, torch.zeros(E * 2, *t.shape[1:])[::2]):
            if name == "x_scale" and bad is not None and bad.dim() == 2 and bad.shape[0] > T:
                continue
            del calls[:]
            with pytest.raises(M.MoeError, match="ExpertTrainLayer"):
                one.run(*good, **dict(scales, **{name: bad}))
            assert not calls
    one.run(*good, **dict(scales, x_scale=torch.zeros(T + 3, 1), s_d=torch.zeros(E)))
    one.run(good[0].view(torch.float8_e4m3fn), *good[1:], **scales)


def test_rows_of_every_layout_that_the_calls_take(calls):
    one = layer(M.MOE_BF16)
    x, logits, w_gu, w_d, out = inputs(torch.bfloat16)
    wide = torch.zeros(T, H + 16, dtype=torch.bfloat16)[:, 8:H + 8]
    one.run(wide, torch.zeros(T, E + 1)[:, 1:], torch.zeros(E, 2 * I, H + 8, dtype=torch.bfloat16)[..., :H],
            torch.zeros(E, 2 * H, I, dtype=torch.bfloat16)[:, H:], torch.zeros(T, H + 4)[:, 4:])
    one.run(torch.zeros(H, 1, dtype=torch.bfloat16).t(), logits[:1], w_gu, w_d, out[:1])  # one row has no pitch


def test_packed_weights_are_not_written_before_the_current_stream_is_done_with_their_memory(calls, streams, monkeypatch):
    monkeypatch.setattr(N, "moe_pack_ffn_weights", lambda *a, **k: calls.append("pack"))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    one = M.ExpertLayer(E, H, I, K, M.MOE_F32, M.MOE_F32, T, device="cpu")
    w = torch.zeros(E, I, H), torch.zeros(E, I, H), torch.zeros(E, H, I)
    one.load_weights(*w, stream=streams[1])
    assert calls == ["77 waits for 5", "pack"]
    one.load_weights(*w)
    assert calls == ["77 waits for 5", "pack", "pack"]


def test_rows_far_apart(calls):
    """A product takes rows at most 16 MiB apart; a training run multiplies a copy of x and takes any."""
    one = layer()
    x, logits, w_gu, w_d, out = inputs()
    far = torch.empty(2 * (1 << 22) + 64).as_strided((2, H), ((1 << 22) + 8, 1))
    one.run(far, logits[:2], w_gu, w_d, out[:2], train=True)
    one.backward(out[:2], far, logits[:2], w_gu, w_d)
    del calls[:]
    with pytest.raises(M.MoeError, match="too far apart"):
        one.run(far, logits[:2], w_gu, w_d, out[:2])
    assert not calls
