"""The binding's first calls from several threads, on the CPU: what it looks up
once is whole for every thread, wherever another one's first call stands."""
import sys
import threading

import pytest
import torch

import trellis_coded_bit_prefill_amd as tp


def interleaved(monkeypatch, names, function, call):
    """The results of call(), made by a second thread between any two steps of the first thread's first call of
    `function` (its lookups `names` not yet made)."""
    got, at = [], 0
    while True:
        for name in names:
            monkeypatch.setattr(tp, name, None)
        steps = 0

        def other():
            try:
                got.append(call())
            except Exception as e:  # (of the second thread)
                got.append(e)

        def trace(frame, event, arg):
            nonlocal steps
            if frame.f_code is not function.__code__:
                return None
            frame.f_trace_opcodes = True
            if event == "opcode":
                steps += 1
                if steps == at + 1:
                    thread = threading.Thread(target=other)
                    thread.start()
                    thread.join()
            return trace

        sys.settrace(trace)
        try:
            call()
        finally:
            sys.settrace(None)
        if steps <= at:
            return got
        at += 1


def test_stream_handle(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 7 + index, raising=False)
    got = interleaved(monkeypatch, ("_current_device", "_raw_stream"), tp._stream_handle,
                      lambda: tp._stream_handle(torch.device("cuda", 0)))
    assert len(got) > 20 and set(got) == {7}


def test_new_tensors(monkeypatch):
    got = interleaved(monkeypatch, ("_empty", "_f32", "_bf16"), tp._new, lambda: tp._new((2, 3), "bf16", "cpu"))
    assert len(got) > 10 and all(getattr(t, "dtype", t) == torch.bfloat16 for t in got)


def test_kinds(monkeypatch):
    got = interleaved(monkeypatch, ("_types", "_grad_enabled", "_forward_ad"), tp._kinds,
                      lambda: (tp._kinds()[3], tp._grad_enabled(), tp._forward_ad._current_level))
    assert len(got) > 10 and set(got) == {((torch.float32,), True, -1)}
