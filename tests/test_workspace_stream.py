"""A workspace that a call takes for itself is taken on the call's stream:
torch's memory is handed out in the order of one stream, so the current
stream's may still be in use by what is pending there."""
import contextlib
import ctypes

import pytest
import torch

from scaled_fp8_gemm_amd import fp8sg as F


class FakeStream:
    cuda_stream = 0x1230


@pytest.fixture
def taken(monkeypatch):
    """Allocations by the stream that they were made on, without a device."""
    log, now, empty = [], [None], torch.empty

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        yield
        now.pop()

    def fake_empty(*a, **k):
        log.append(now[-1])
        return empty(*a, **{**k, "device": "cpu"})
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", fake_empty)
    monkeypatch.setattr(F, "fp8_workspace_init", lambda *a: None)
    return log


def test_workspaces_are_taken_on_the_calls_stream(taken):
    s = FakeStream()
    F.workspace(stream=s)
    assert taken == [s]
    F._Ws(None, s)
    x, e = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    f = torch.zeros(16)
    # refused after the workspace is there: these are not on a GPU
    with pytest.raises(ValueError, match="on the GPU"):
        F.fp8_layernorm_bwd(x, x, f, f, f, x, f, f, stream=s)
    with pytest.raises(ValueError, match="on the GPU"):
        F.fp8_moe_sort(e, 8, 1, e, e, e, e, stream=s)
    assert taken == [s] * 4
    del taken[:]
    F.workspace()
    F._Ws(None, None)
    assert taken == [None] * 2


def test_raw_handles(taken, monkeypatch):
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: ("external", h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    for handle in (0x50, ctypes.c_void_p(0x50), 0, ctypes.c_void_p(0)):
        F.workspace(stream=handle)
    assert taken == [("external", 0x50)] * 2 + ["default"] * 2


def test_a_raw_handle_needs_a_workspace():
    x, e = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    f = torch.zeros(16)
    for call in (lambda: F._Ws(None, 77),
                 lambda: F.fp8_layernorm_bwd(x, x, f, f, f, x, f, f, stream=77),
                 lambda: F.fp8_moe_sort(e, 8, 1, e, e, e, e, stream=77)):
        with pytest.raises(ValueError, match="raw handle"):
            call()


@pytest.mark.gpu
def test_workspaces_come_from_the_streams_own_memory():
    def pool(t):
        for seg in torch.cuda.memory_snapshot():
            if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
                return seg["stream"]
    s = torch.cuda.Stream()
    assert pool(F.workspace(stream=s)) == s.cuda_stream
    assert pool(F.workspace(stream=s.cuda_stream)) == s.cuda_stream
    assert pool(F._Ws(None, s).t) == s.cuda_stream
    with torch.cuda.stream(s):
        assert pool(F.workspace(stream=0)) == torch.cuda.default_stream().cuda_stream
    assert pool(F.workspace()) == torch.cuda.current_stream().cuda_stream


@pytest.mark.gpu
def test_calls_on_a_side_stream_with_workspaces_of_their_own():
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn((300, 1003), generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(1003, device="cuda")
    e = torch.randint(0, 8, (300, 2), generator=g, device="cuda", dtype=torch.int32)

    def run(stream):
        n = lambda dt, *s: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        r = F.moe_rows(600, 8, 16)
        o = [n(torch.bfloat16, 300, 1003), n(torch.float32, 300), n(torch.float32, 300),
             n(torch.uint8, 300, 1003), n(torch.float32, 1), n(torch.bfloat16, 300, 1003),
             n(torch.float32, 1003), n(torch.float32, 1003), n(torch.int32, 9), n(torch.int32, 8),
             n(torch.int32, 300, 2), n(torch.int32, r)]
        torch.cuda.synchronize()
        F.fp8_layernorm_fwd(x, w, w, 1e-5, *o[:3], yq=F.cast_out(o[3], 0, 0, None, w[:1], o[4]),
                            stream=stream)
        F.fp8_layernorm_bwd(dy, x, o[1], o[2], w, *o[5:8], stream=stream)
        F.fp8_moe_sort(e, 8, 16, *o[8:], stream=stream)
        torch.cuda.synchronize()
        return o
    for a, b in zip(run(None), run(torch.cuda.Stream())):
        assert torch.equal(a, b)
