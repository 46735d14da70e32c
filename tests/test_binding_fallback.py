"""The binding on a torch without the private names it prefers: every call needs a stream's
handle and the current device, and falls back to the public functions."""
import importlib.util
import types

import torch

import mxfp8_block_scaled_05_gb300 as m


def test_public_functions_serve_without_the_private_names(monkeypatch):
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    asked = []

    def current_stream(device=None):
        asked.append(device)
        return types.SimpleNamespace(cuda_stream=0x77)
    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    spec = importlib.util.spec_from_file_location("binding_without_private_names", m.__file__)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod._stream() == 0x77 and asked == [3]
    assert mod._stream(types.SimpleNamespace(cuda_stream=5)) == 5

    class Tensor:                     # what _require asks a tensor
        is_cuda, dtype, device = True, torch.uint8, "cuda:3"

        def is_contiguous(self):
            return True

        def get_device(self):
            return 3
    mod._require(Tensor(), torch.uint8, "t")
