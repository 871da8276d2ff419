"""Checks of the many-adapter layer that need no GPU: arguments that do not fit
the weight, the bank or the plan are refused before anything is launched."""
import ctypes

import pytest
import torch

import bit_nf4_quantized_blockwise_b200 as q
from bit_nf4_quantized_blockwise_b200._lib import AdapterPlan, NF4Weight, qlora_adapters_t, qlora_nf4_t

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUP, ERR_CB, ERR_CUDA, ERR_TIMEOUT, ERR_WS = range(9)
P = ctypes.c_void_p
FAKE = 0x10000  # never dereferenced
O, H, M, N, R = 256, 512, 16, 3, 8
BF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    from bit_nf4_quantized_blockwise_b200 import build
    build.build()
    return q.lib()


def _wq():
    w = qlora_nf4_t()
    w.codes = w.absmax_fp8 = w.dq_scale = w.dq_mean = FAKE
    w.o, w.h, w.block, w.dq_block = O, H, 64, 256
    w.codebook = (ctypes.c_float * 16)(*[float(v) for v in range(-7, 9)])
    return w


def test_plan_refusals(L):
    size = L.qlora_adapter_plan_size(M, N)
    assert size > 0
    for bad in ((0, N), (M, 0), (M, 65536), (-1, N), ((1 << 28) + 1, N)):
        assert L.qlora_adapter_plan_size(*bad) == 0
    n0 = L.qlora_launch_count()
    assert L.qlora_adapter_plan(P(FAKE), 0, N, P(FAKE), size, None) == ERR_SHAPE
    assert L.qlora_adapter_plan(P(FAKE), M, 0, P(FAKE), size, None) == ERR_UNSUP
    assert L.qlora_adapter_plan(None, M, N, P(FAKE), size, None) == ERR_NULL
    assert L.qlora_adapter_plan(P(FAKE), M, N, None, size, None) == ERR_WS
    assert L.qlora_adapter_plan(P(FAKE), M, N, P(FAKE), size - 1, None) == ERR_WS
    assert L.qlora_adapter_plan(P(FAKE + 2), M, N, P(FAKE), size, None) == ERR_ALIGN
    assert L.qlora_adapter_plan(P(FAKE), M, N, P(FAKE + 8), size, None) == ERR_ALIGN
    assert L.qlora_launch_count() == n0


@pytest.mark.parametrize("bad", [
    (O, H, 64, 0, R), (O, H, 0, N, R), (O, H, 0, 0, R), (O, H, -1, N, R), (O, H, (1 << 28) + 1, N, R),
    (O, H, M, 65536, R), (O, H, M, N, 0), (O, H, M, N, 12), (O, H, M, N, 264), (O, H, M, N, -8),
    (0, H, M, N, R), (O, 0, M, N, R), (O, 32, M, N, R), (96, H, M, N, R), (-64, H, M, N, R), (O, 1 << 31, M, N, R)])
def test_workspace_query_of_sizes_that_are_not_taken(L, bad):
    assert L.qlora_multi_linear_fwd_workspace_size(*bad) == 0
    assert L.qlora_multi_linear_bwd_workspace_size(*bad) == 0


def test_layer_refusals(L):
    plan = L.qlora_adapter_plan_size(M, N)
    wf = L.qlora_multi_linear_fwd_workspace_size(O, H, M, N, R)
    wb = L.qlora_multi_linear_bwd_workspace_size(O, H, M, N, R)
    n0 = L.qlora_launch_count()

    def fwd(X=FAKE, Y=FAKE, T=FAKE, dt=0, ws=FAKE, wsb=wf, pl=FAKE, plb=plan, tokens=M, **ad):
        b = qlora_adapters_t(FAKE, FAKE, FAKE, N, R)
        for k, v in ad.items():
            setattr(b, k, v)
        return L.qlora_multi_linear_fwd(ctypes.byref(_wq()), P(X), tokens, ctypes.byref(b), P(pl), plb, P(Y), dt, P(T),
                                        P(ws), wsb, None)

    def bwd(dY=FAKE, dX=FAKE, d1=FAKE, d2=FAKE, T=None, dt=0, ws=FAKE, wsb=wb):
        b = qlora_adapters_t(FAKE, FAKE, FAKE, N, R)
        return L.qlora_multi_linear_bwd(ctypes.byref(_wq()), P(FAKE), P(dY), M, ctypes.byref(b), P(FAKE), plan, P(T),
                                        P(dX), dt, P(d1), P(d2), P(ws), wsb, None)
    for r in (0, 4, 12, 264):
        assert fwd(r=r) == ERR_UNSUP
    assert fwd(n=0) == ERR_UNSUP and fwd(dt=2) == ERR_UNSUP
    assert fwd(tokens=0) == ERR_SHAPE
    for bad in ({"X": None}, {"Y": None}, {"pl": None}, {"L1": None}, {"L2": None}, {"s": None}):
        assert fwd(**bad) == ERR_NULL
    for bad in ({"X": FAKE + 2}, {"Y": FAKE + 4}, {"T": FAKE + 8}, {"L1": FAKE + 2}, {"s": FAKE + 2}, {"pl": FAKE + 4},
                {"ws": FAKE + 8}):
        assert fwd(**bad) == ERR_ALIGN
    assert fwd(wsb=wf - 1) == ERR_WS and fwd(ws=None) == ERR_WS and fwd(plb=plan - 1) == ERR_WS
    for bad in ({"dY": None}, {"dX": None}, {"d1": None}, {"d2": None}):
        assert bwd(**bad) == ERR_NULL
    for bad in ({"dY": FAKE + 2}, {"d1": FAKE + 4}, {"d2": FAKE + 4}, {"T": FAKE + 4}):
        assert bwd(**bad) == ERR_ALIGN
    assert bwd(dt=5) == ERR_UNSUP and bwd(wsb=wb - 1) == ERR_WS
    assert L.qlora_multi_linear_fwd(ctypes.byref(_wq()), P(FAKE), M, None, P(FAKE), plan, P(FAKE), 0, None, P(FAKE), wf,
                                    None) == ERR_NULL
    assert L.qlora_launch_count() == n0


def _weight():
    n = O * H
    return NF4Weight(torch.zeros(n // 2, dtype=torch.uint8), torch.zeros(n // 64, dtype=torch.uint8),
                     torch.zeros(n // 16384), torch.zeros(1), O, H, tuple(float(v) for v in range(-7, 9)))


def _raises(fn, *args, match, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def test_binding_refusals(L):
    bank = q.AdapterBank(torch.zeros(N, H, R, dtype=BF), torch.zeros(N, R, O, dtype=BF), torch.zeros(N))
    _raises(q.AdapterBank, bank.L1[0], bank.L2, bank.s, match="L1 must be")
    _raises(q.AdapterBank, bank.L1, bank.L2[:2], bank.s, match="L2 has shape")
    _raises(q.AdapterBank, bank.L1.float(), bank.L2, bank.s, match="L1 has dtype")
    _raises(q.AdapterBank, bank.L1, bank.L2, bank.s[:2], match="s has shape")
    _raises(q.AdapterBank, bank.L1, bank.L2.transpose(1, 2).contiguous().transpose(1, 2), bank.s, match="contiguous")
    _raises(q.qlora_adapter_plan, torch.zeros(M), N, match="int32")
    _raises(q.qlora_adapter_plan, torch.zeros(M, dtype=torch.int64), N, match="int32")
    _raises(q.qlora_adapter_plan, torch.zeros(0, dtype=torch.int32), N, match="empty")
    _raises(q.qlora_adapter_plan, torch.zeros(M, dtype=torch.int32), 0, match="not supported")
    plan = AdapterPlan(torch.zeros(L.qlora_adapter_plan_size(M, N), dtype=torch.uint8), M, N)
    _raises(q.qlora_adapter_plan, torch.zeros(M + 1, dtype=torch.int32), N, plan=plan, match="plan is for")
    _raises(q.qlora_adapter_plan, torch.zeros(M, dtype=torch.int32), N, match="CUDA")
    X, dY = torch.zeros(M, H, dtype=BF), torch.zeros(M, O, dtype=BF)
    n0 = q.qlora_launch_count()
    f, b = q.qlora_multi_linear_fwd, q.qlora_multi_linear_bwd
    _raises(f, _weight(), X[:, :H - 64], bank, plan, match="X has shape")
    _raises(f, _weight(), X[:M - 1], bank, plan, match="plan is for")
    _raises(f, _weight(), X, bank, AdapterPlan(plan.buffer, M, N + 1), match="plan is for")
    _raises(f, _weight(), X.float(), bank, plan, match="X has dtype")
    _raises(f, _weight(), X, q.AdapterBank(bank.L1, bank.L2[:, :, :O - 64].contiguous(), bank.s), plan, match="bank is for")
    _raises(f, _weight(), X, bank, plan, Y=torch.zeros(M, O - 64), match="Y has shape")
    _raises(f, _weight(), X, bank, plan, Y=torch.zeros(M, O, dtype=torch.float16), match="Y has dtype")
    _raises(f, _weight(), X, bank, plan, T_save=torch.zeros(M, R + 1), match="T has shape")
    _raises(f, _weight(), X, bank, plan, match="CUDA")
    _raises(b, _weight(), X, dY[:, :O - 64], bank, plan, match="dY has shape")
    _raises(b, _weight(), X, dY, bank, plan, dX=torch.zeros(M, H - 64), match="dX has shape")
    _raises(b, _weight(), X, dY, bank, plan, dL1=torch.zeros(N, H, R + 8), match="dL1 has shape")
    _raises(b, _weight(), X, dY, bank, plan, dL2=torch.zeros(N, R, O, dtype=BF), match="dL2 has dtype")
    _raises(b, _weight(), X, dY, bank, plan, T_saved=torch.zeros(M + 1, R), match="T has shape")
    _raises(b, _weight(), X, dY, bank, plan, match="CUDA")
    from bit_nf4_quantized_blockwise_b200._lib import _workspace
    with pytest.raises(ValueError, match="ws must be"):
        _workspace(torch.zeros(64, dtype=torch.uint8), 64, torch.device("cuda", 0))
    assert q.qlora_launch_count() == n0
