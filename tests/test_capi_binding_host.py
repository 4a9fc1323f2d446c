"""The binding's own steps on every call: the current stream's handle and the arguments' addresses. No GPU is needed."""
import importlib.util
import sys

import pytest

from decode_attention_mfa_gb300 import capi


@pytest.fixture
def fresh(monkeypatch):
    """The binding as a program finds it before its first call, with a stand-in for torch's streams (handle 7 on device 3)."""
    import torch
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", {3: 7}.__getitem__, raising=False)
    spec = importlib.util.spec_from_file_location("capi_fresh", capi.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_a_first_stream_lookup_interrupted_anywhere_by_another(fresh):
    """A second call at every instruction of the first, as another thread may make it."""
    found = []

    def trace(frame, event, arg):
        if frame.f_code is not fresh._stream.__code__:
            return None
        frame.f_trace_opcodes = True
        if event == "opcode":
            before = fresh.__dict__.copy()
            found.append(fresh._stream(None))
            for name, value in before.items():  # as if it had not been made
                fresh.__dict__[name] = value
        return trace

    old = sys.gettrace()
    sys._getframe().f_trace_opcodes = True  # (Python 3.12 asks for it before the trace begins)
    sys.settrace(trace)
    try:
        handle = fresh._stream(None)
    finally:
        sys.settrace(old)
    assert handle == 7 and len(found) > 10 and set(found) == {7}


@pytest.mark.parametrize("name", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_the_stream_lookup_without_torchs_private_names(fresh, monkeypatch, name):
    import torch
    monkeypatch.delattr(torch._C, name)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 4)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: type("Stream", (), {"cuda_stream": 10 + device}))
    assert fresh._stream(None) == 14 and fresh._stream(None) == 14


def test_addresses_and_tensors_are_taken_without_an_exception():
    """Addresses as integers are as usual as tensors (a row of a table, a part of a workspace): neither is found by failing."""
    import torch

    class Address(int):
        pass

    raised = []

    def trace(frame, event, arg):
        if event == "exception":
            raised.append(arg)
        return trace

    t = torch.zeros(4)
    old = sys.gettrace()
    sys.settrace(trace)
    try:
        got = [capi._ptr(x) for x in (4096, 0, None, t)]
    finally:
        sys.settrace(old)
    assert got == [4096, 0, None, t.data_ptr()] and not raised
    assert capi._ptr(Address(8)) == 8
    with pytest.raises(AttributeError):
        capi._ptr("text")
