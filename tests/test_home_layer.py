"""ExpertLayer's plumbing on the CPU: what it hands to the allocator and what it refuses, with the calls
themselves left out."""
import pytest
import torch

import asynchronous_moe_expert_amd as M
from asynchronous_moe_expert_amd import _native as N

T, E, K, H, I = 5, 8, 2, 64, 128


@pytest.fixture
def calls(monkeypatch):
    """The names of the calls that run() makes; none of them does anything."""
    made = []
    for name in ("moe_route", "moe_sort_rows", "moe_expert_ffn_grouped", "moe_merge_rows", "moe_pack_ffn_weights"):
        monkeypatch.setattr(N, name, lambda *a, name=name, **k: made.append(name))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)  # that of tensors on the CPU
    return made


def layer(**how):
    made = M.ExpertLayer(E, H, I, K, M.MOE_F32, M.MOE_F32, T, device="cpu", **how)
    made.load_weights(torch.zeros(E, I, H), torch.zeros(E, I, H), torch.zeros(E, H, I))
    return made


@pytest.mark.parametrize("raw", [True, False])
def test_a_run_on_another_stream_records_what_it_works_on(calls, monkeypatch, raw):
    class Stream:
        cuda_stream = 77

    recorded = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s.cuda_stream)))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: Stream())
    monkeypatch.setattr(N, "_raw_stream", lambda index: 5)
    one, x, logits, out = layer(), torch.zeros(T, H), torch.zeros(T, E), torch.zeros(T, H)
    one.s_gate = torch.zeros(3)
    for stream in (None, 5):  # the current one
        one.run(x, logits, out, stream=stream)
    assert not recorded
    one.run(x, logits, out, stream=77 if raw else Stream())
    for t in (x, one.w_gu, one.w_d, one.s_gate, one.workspace, one.y, one.row_slot, one.offsets):
        assert (t.data_ptr(), 77) in recorded


@pytest.mark.parametrize("E,K", [(257, 4), (512, 8), (0, 1), (8, 0), (8, 9), (64, 33)])
def test_sizes_that_no_call_takes_are_refused_when_the_layer_is_built(E, K):
    with pytest.raises(M.MoeError, match="256 experts"):
        M.ExpertLayer(E, H, I, K, M.MOE_F32, M.MOE_F32, 4, device="cpu")


def test_the_largest_sizes_are_taken():
    for E, K in ((256, 32), (1, 1), (256, 1)):
        M.ExpertLayer(E, H, I, K, M.MOE_F32, M.MOE_F32, 4, device="cpu")


def test_a_refused_run_makes_no_call(calls):
    one, x, logits, out = layer(), torch.zeros(T, H), torch.zeros(T, E), torch.zeros(T, H)
    del calls[:]
    for bad, text in (((x, logits, out[:3]), "out"), ((x, logits, torch.zeros(T, H + 8)), "out"),
                      ((x[:1].expand(T, H), logits, out), "overlap"), ((x, logits[:2], out), "logits")):
        with pytest.raises(M.MoeError, match=text):
            one.run(*bad)
    with pytest.raises(M.MoeError, match="load_weights"):
        M.ExpertLayer(E, H, I, K, M.MOE_F32, M.MOE_F32, T, device="cpu").run(x, logits, out)
    assert not calls


def test_one_token_may_have_any_pitch(calls, monkeypatch):
    """The row of a [H][1] column's transpose is one run of H elements whatever its stride says."""
    seen = []
    monkeypatch.setattr(N, "moe_expert_ffn_grouped", lambda *a, gather, **k: seen.append(gather[2]))
    x = torch.arange(float(H)).view(H, 1).t()
    assert x.stride() == (1, 1)
    layer().run(x, torch.zeros(1, E), torch.zeros(1, H))
    assert seen[0].stride() == (H, 1) and torch.equal(seen[0], x)
