"""The current stream without torch's private shortcuts."""
import importlib.util

import torch

from rope_frequency_chunk_b200 import fasa as F


def load(monkeypatch, without):
    for name in without:
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location("fasa_again", F.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Stream:
    cuda_stream = 1234


def test_public_functions_serve_where_the_shortcuts_are_gone(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: {3: Stream}[device])
    m = load(monkeypatch, ["_cuda_getDevice", "_cuda_getCurrentRawStream"])
    assert m._stream(None) == 1234
    assert m._stream(Stream()) == 1234 and m._stream(77) == 77

    class T:
        def get_device(self):
            return 3

    called = []

    class Lib:
        def fasa_any(self, *a):
            called.append(a)
            return 0

    m._lib = Lib()
    m._launch("fasa_any", T(), None, 5)
    assert called == [(5, 1234)]
