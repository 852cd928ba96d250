"""CPU: the binding takes the current stream from PyTorch's public call where the faster name is missing."""
import importlib.util
import types

import torch

from conditional_sparse_attention_b200 import oda


def test_the_public_call_serves_where_the_raw_one_is_missing(monkeypatch):
    with monkeypatch.context() as m:
        m.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
        m.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=4096))
        m.setattr(torch.cuda, "current_device", lambda: 0)
        fresh = importlib.util.module_from_spec(importlib.util.find_spec(oda.__name__))
        fresh.__spec__.loader.exec_module(fresh)
        assert fresh._s(None).value == 4096
        assert fresh._s(8192).value == 8192
        assert fresh._s(types.SimpleNamespace(cuda_stream=512)).value == 512


def test_the_raw_call_is_asked_for_the_current_device(monkeypatch):
    monkeypatch.setattr(oda, "_raw_stream", lambda device: 100 + device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert oda._s(None).value == 103
