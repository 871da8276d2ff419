"""The rounding of the 8-bit AdamW state: refusals that need no GPU, and the struct's layout."""
import ctypes

import pytest
import torch

import bit_nf4_quantized_blockwise_b200 as q
from bit_nf4_quantized_blockwise_b200._lib import qlora_adamw_state_t, qlora_adamw_t

ERR_UNSUP = 4
P = ctypes.c_void_p
FAKE = 0x10000  # never dereferenced


def test_step_refuses_other_roundings():
    from bit_nf4_quantized_blockwise_b200 import build
    build.build()
    L = q.lib()
    assert ctypes.sizeof(qlora_adamw_state_t) == 48
    size = L.qlora_multi_adamw_plan_size(1, 256)
    for bits, rounding in ((8, 2), (8, -1), (32, 1)):
        st = qlora_adamw_state_t(FAKE, FAKE, FAKE, FAKE, FAKE, bits, rounding)
        h = qlora_adamw_t(1e-3, 0.9, 0.999, 1e-8, 0.0, 0.3, 0)
        grads = (P * 1)(None)
        assert L.qlora_multi_adamw_step(P(FAKE), size, 1, 256, grads, 0, ctypes.byref(st), ctypes.byref(h),
                                        None) == ERR_UNSUP


def test_class_refuses_other_roundings():
    p = torch.zeros(4)
    with pytest.raises(ValueError, match="rounding"):
        q.MultiAdamW([p], state_bits=8, rounding="up")
    with pytest.raises(ValueError, match="rounding"):
        q.MultiAdamW([p], rounding="stochastic")
