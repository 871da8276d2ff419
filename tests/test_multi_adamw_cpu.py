"""Checks of the many-tensor AdamW step that need no GPU: the state layout, and
that bad arguments are refused before anything is launched."""
import ctypes

import pytest
import torch

import bit_nf4_quantized_blockwise_b200 as q
from bit_nf4_quantized_blockwise_b200._lib import qlora_adamw_state_t, qlora_adamw_t, qlora_adamw_tensor_t

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUP, _, _, _, ERR_WS = range(9)
P = ctypes.c_void_p
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    from bit_nf4_quantized_blockwise_b200 import build
    build.build()
    return q.lib()


def _table(*rows):
    t = (qlora_adamw_tensor_t * len(rows))()
    for e, (p, c, n) in zip(t, rows):
        e.param, e.copy, e.n = p, c, n
    return t


def test_state_starts_every_tensor_in_a_new_block(L):
    t = _table((FAKE, None, 1), (FAKE, None, 256), (FAKE, None, 257))
    assert L.qlora_multi_adamw_state_elems(ctypes.cast(t, P), 3) == 256 + 256 + 512
    assert L.qlora_multi_adamw_state_elems(ctypes.cast(_table((FAKE, None, 0)), P), 1) == 0
    assert L.qlora_multi_adamw_state_elems(None, 1) == 0
    assert L.qlora_multi_adamw_plan_size(0, 256) == 0 and L.qlora_multi_adamw_plan_size(3, 0) == 0
    assert L.qlora_multi_adamw_plan_size(3, 1024) > 0


def test_plan_refusals(L):
    size = L.qlora_multi_adamw_plan_size(1, 256)

    def plan(rows, n=1, ws=FAKE, nbytes=size):
        return L.qlora_multi_adamw_plan(ctypes.cast(_table(rows), P), n, P(ws), nbytes, None)
    assert L.qlora_multi_adamw_plan(None, 1, P(FAKE), size, None) == ERR_NULL
    assert plan((FAKE, None, 4), n=0) == ERR_SHAPE
    assert plan((FAKE, None, 0)) == ERR_SHAPE
    assert plan((None, None, 4)) == ERR_NULL
    assert plan((FAKE + 2, None, 4)) == ERR_ALIGN
    assert plan((FAKE, FAKE + 1, 4)) == ERR_ALIGN
    assert plan((FAKE, None, 4), nbytes=size - 1) == ERR_WS
    assert plan((FAKE, None, 4), ws=None) == ERR_WS
    assert plan((FAKE, None, 4), ws=FAKE + 8) == ERR_ALIGN


def test_step_refusals(L):
    size = L.qlora_multi_adamw_plan_size(1, 256)
    n0 = L.qlora_launch_count()

    def step(g=FAKE, gd=0, bits=32, elems=256, count=1, nbytes=size, state=None, **hp):
        st = qlora_adamw_state_t(FAKE, FAKE, FAKE, FAKE, FAKE, bits)
        for k, v in (state or {}).items():
            setattr(st, k, v)
        h = qlora_adamw_t(1e-3, 0.9, 0.999, 1e-8, 0.0, 0.3, 0)
        for k, v in hp.items():
            setattr(h, k, v)
        grads = (P * 1)(g)
        return L.qlora_multi_adamw_step(P(FAKE), nbytes, count, elems, grads, gd, ctypes.byref(st), ctypes.byref(h), None)
    assert step(bits=16) == ERR_UNSUP
    assert step(gd=2) == ERR_UNSUP
    assert step(bits=8, state={"m_scale": None}) == ERR_NULL
    assert step(state={"steps": None}) == ERR_NULL
    assert step(state={"m": FAKE + 4}) == ERR_ALIGN
    assert step(elems=255) == ERR_SHAPE and step(count=0) == ERR_SHAPE
    assert step(nbytes=size - 1) == ERR_WS
    assert step(g=FAKE + 2) == ERR_ALIGN and step(g=FAKE + 1, gd=1) == ERR_ALIGN
    for bad in ({"beta1": 1.0}, {"beta2": -0.1}, {"eps": 0.0}, {"lr": -1.0}, {"weight_decay": -1.0},
                {"max_grad_norm": float("nan")}):
        assert step(**bad) == ERR_UNSUP
    assert step(g=None) == OK  # no gradient at all: nothing to do
    assert L.qlora_launch_count() == n0


def test_class_refusals():
    p = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        q.MultiAdamW([p])
    with pytest.raises(ValueError, match="empty"):
        q.MultiAdamW([])
    with pytest.raises(ValueError, match="state_bits"):
        q.MultiAdamW([p], state_bits=16)
    with pytest.raises(ValueError, match="copies"):
        q.MultiAdamW([p], copies=[])
