"""The binding's own decisions (no GPU: the library and the devices are stand-ins)."""
import contextlib

import torch

from kimi_delta_attention_gb300 import _gdr


def test_norm_workspace_goes_by_device(monkeypatch):
    """The size depends on a device's processors: asked for on the tensor's device, and kept per
    device, whichever is current."""
    processors, now = {0: 100, 1: 152}, [0]

    class Library:
        def kda_layer_norm_bwd_workspace_size(self, rows, D):
            return 256 + 8 * D * min(rows, processors[now[0]])

    @contextlib.contextmanager
    def device(index):
        was, now[0] = now[0], index
        yield
        now[0] = was

    monkeypatch.setattr(_gdr, "load_library", Library)
    monkeypatch.setattr(torch.cuda, "device", device)
    _gdr._norm_workspace_bytes.cache_clear()
    try:
        for current in (0, 1):
            now[0] = current
            for index in (0, 1):
                assert _gdr._norm_workspace_bytes(1000, 64, index) == 256 + 8 * 64 * processors[index]
            assert now[0] == current
    finally:
        _gdr._norm_workspace_bytes.cache_clear()
