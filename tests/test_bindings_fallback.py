"""The bindings without the private functions of torch that they prefer (no GPU needed)."""
import importlib.util
import types

import torch

import kda_linear_attention_02_b200 as kda


def load_copy():
    """A second copy of the package's __init__, as it would be imported now."""
    spec = importlib.util.spec_from_file_location("kda_copy", kda.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_private_functions_of_torch_may_be_missing(monkeypatch):
    class Without(types.ModuleType):
        def __getattr__(self, name):
            if name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
                raise AttributeError(name)
            return getattr(real, name)
    real = torch._C
    monkeypatch.setattr(torch, "_C", Without("torch._C"))
    m = load_copy()
    asked = []

    class Stream:
        cuda_stream = 1234
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: asked.append(dev) or Stream)
    assert m._raw_stream(3) == 1234 and asked == [3]
    assert m._current_device is torch.cuda.current_device


def test_private_functions_of_torch_are_used_where_they_are():
    m = load_copy()
    assert m._raw_stream is torch._C._cuda_getCurrentRawStream and m._current_device is torch._C._cuda_getDevice
