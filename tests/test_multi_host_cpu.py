"""Host side of the many-adapter layer and the many-tensor AdamW, on the CPU with fakes of the library."""
import contextlib

import pytest
import torch

from bit_nf4_quantized_blockwise_b200 import _lib


class _Sizes:
    """A library whose workspace sizes depend on the current device, as they do where the number of SMs differs."""

    def __init__(self):
        self.current, self.queries = 0, 0

    @contextlib.contextmanager
    def device(self, index):
        before, self.current = self.current, index
        try:
            yield
        finally:
            self.current = before

    def qlora_multi_linear_fwd_workspace_size(self, *sizes):
        self.queries += 1
        return 1000 * (self.current + 1) + sizes[2]

    def qlora_multi_linear_bwd_workspace_size(self, *sizes):
        return 7 + self.qlora_multi_linear_fwd_workspace_size(*sizes)


def test_workspace_sizes_are_those_of_the_call_s_device(monkeypatch):
    fake = _Sizes()
    monkeypatch.setattr(_lib, "lib", lambda: fake)
    monkeypatch.setattr(torch.cuda, "device", fake.device)
    _lib._multi_ws_size.cache_clear()
    try:
        for _ in range(2):
            for dev in (0, 1, 3):
                assert _lib._multi_ws_size(False, dev, 256, 128, 40, 4, 16) == 1000 * (dev + 1) + 40
                assert _lib._multi_ws_size(True, dev, 256, 128, 40, 4, 16) == 1000 * (dev + 1) + 47
        assert fake.queries == 6 and fake.current == 0
    finally:
        _lib._multi_ws_size.cache_clear()
