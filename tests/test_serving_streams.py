"""Where the binding makes an attention call's workspace when the caller gives
none (no GPU: the library's call and the streams are stand-ins)."""
import contextlib
import types

import pytest
import torch

from place_partial_rope_gb300 import binding


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def calls(monkeypatch):
    """What happens, in order; `current` is the stand-in for torch's current stream."""
    log = types.SimpleNamespace(current="default", made_on=[], launched_on=[])

    @contextlib.contextmanager
    def on(stream):
        before, log.current = log.current, stream
        yield
        log.current = before

    class Workspace:
        nbytes = 64
        device = torch.device("cpu")

        def __init__(self):
            log.made_on.append(log.current)

        def data_ptr(self):
            return 1 << 40

        def is_contiguous(self):
            return True

        def record_stream(self, stream):
            pass

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(binding, "tree_attention_workspace", lambda q, cache, max_q: Workspace())
    monkeypatch.setattr(binding, "_launch", lambda fn, args, stream, device: log.launched_on.append(stream))
    return log


def attend(stream):
    cpu = torch.device("cpu")
    cache = types.SimpleNamespace(device=cpu, k_dim=64, v_dim=64, heads=1, _ref=0)
    q = torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    binding.rope_partial_tree_attention(q, cache, i32(0, 2), i32(9), i32(0).view(1, 1), torch.empty_like(q),
                                        stream=stream)


def test_a_workspace_belongs_to_the_stream_that_uses_it(calls):
    """Memory that the allocator hands out on one stream may still be in use
    there, which a call on another stream does not wait for."""
    side = Stream(77)
    attend(side)
    assert calls.made_on == [side] and calls.launched_on == [side]
    assert calls.current == "default"


def test_a_raw_handle_is_a_stream_too(calls):
    attend(1234)
    assert calls.made_on == [("external", 1234)] and calls.launched_on == [1234]


def test_the_current_stream_needs_nothing(calls):
    attend(None)
    assert calls.made_on == ["default"] and calls.launched_on == [None]


@pytest.mark.gpu
def test_calls_on_other_streams_without_a_workspace():
    """A side stream, its raw handle and the default stream's handle 0: the same
    results."""
    from test_tree_gpu import Case
    c = Case("bf16", "fp8", [7, 3], [150, 3333], 2, 3, 64, 64, page=16, seed=6)
    want = c.run()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        torch.cuda.synchronize()
        out, lse = c.run(stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
