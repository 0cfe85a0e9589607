"""The benchmark makes its inputs and workspaces on the current stream and calls
the library on another. The first call has to wait for what was queued: memory that the
input generator freed may be the workspace, with its last writes still pending."""

from __future__ import annotations

import contextlib
import os
import sys
import types

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bench  # noqa: E402


class FirstCall(Exception):
    pass


def _fake_cuda(monkeypatch, log):
    class Event:
        def __init__(self, **_):
            pass

        def record(self, *_):
            pass

    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(torch.cuda, "Stream", lambda *_: object())
    monkeypatch.setattr(torch.cuda, "set_device", lambda *_: None)
    monkeypatch.setattr(torch.cuda, "stream", lambda *_: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *_: log.append("wait"))


def _first(log):
    def call(*_, **__):
        log.append("call")
        raise FirstCall

    return call


def test_side_workload_waits_for_its_inputs(monkeypatch):
    log = []
    _fake_cuda(monkeypatch, log)
    monkeypatch.setattr(bench, "make_sets", lambda *_: log.append("inputs") or [
        {"target": None, "draft": None, "tokens": None, "uniforms": None}] * 2)
    sv = types.SimpleNamespace(SV_BF16=0, SV_F32=1, spec_verify=_first(log),
                               new_workspace=lambda *_: log.append("workspace"))
    with pytest.raises(FirstCall):
        bench.time_sub_workload(sv, "c1", "cpu", None)
    assert log == ["inputs", "workspace", "wait", "call"]
