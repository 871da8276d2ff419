"""GPU tests of how many bits the many-adapter layer keeps: sums of long products and the adapters'
term, against 64 bits.

u = 2^-24.  The tensor core cuts its running sum by up to a step of fp32, 2 u of it, at every 16
products.  Above 32 tokens an accumulator ends after 1024 products (fp32 results: 512, and 256 where
there are 2048 or fewer) and is added in fp32, up to 8 tokens after 512."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_blockwise_b200 as q
from oracle import nf4

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _weight(o, h, codes):
    """Single-level constants of 1 and the given codes (uint8 [o*h/2])."""
    return q.NF4Weight(codes, None, None, None, o, h, tuple(float(v) for v in nf4.nf4_codebook()),
                       absmax=torch.ones(o * h // 64, device="cuda"))


def _all_positive(rows, o, h, k):
    """Positive weights and positive rows, so that a cut of the running sum does not average out."""
    g = torch.Generator(device="cuda").manual_seed(3)
    code = lambda: torch.randint(8, 16, (o * h // 2,), device="cuda", generator=g, dtype=torch.uint8)  # noqa: E731
    w = _weight(o, h, (code() << 4) | code())
    x = torch.rand(rows, k, device="cuda", generator=g) + 0.5
    x *= 1 + torch.rand(rows, 1, device="cuda", generator=g)
    return w, x.bfloat16()


def _base(w, x, bwd, dtype):
    """X W' (or dY W'^T) of tokens without adapter, by the many-adapter layer, and in 64 bits."""
    M, o, h = x.shape[0], w.o, w.h
    bank = q.AdapterBank(torch.zeros(1, h, 8, device="cuda", dtype=torch.bfloat16),
                         torch.zeros(1, 8, o, device="cuda", dtype=torch.bfloat16), torch.ones(1, device="cuda"))
    plan = q.qlora_adapter_plan(torch.full((M,), -1, device="cuda", dtype=torch.int32), 1)
    W = q.qlora_dequant(w).view(o, h)
    if bwd:
        X = torch.zeros(M, h, device="cuda", dtype=torch.bfloat16)
        return q.qlora_multi_linear_bwd(w, X, x, bank, plan, dx_dtype=dtype)[0], x.double() @ W.double()
    return q.qlora_multi_linear_fwd(w, x, bank, plan, y_dtype=dtype)[0], x.double() @ W.double().t()


@pytest.mark.parametrize("bwd", [False, True])
def test_bf16_results_are_the_fp32_sum_rounded_once(bwd):
    """8192 positive products in 8 accumulators A = S / 8 of 64 steps: at step i the running sum is
    i/64 A and is cut by at most 2 u of that, 64 u A in all: 64 u S; the 8 additions, below 8 u S.
    A result rounds to another value than the exact sum does only if a border lies between the two:
    for a share of 72 u S over the distance of the borders, 2^-8 S at least, that is 0.0011; 3
    standard deviations of a count over 757760 elements are 0.0001 more.  (In one accumulator of 512
    steps the cut may be 512 u S, and half of that on average.)"""
    n, k = 74 * 256, 8192  # as many 256-wide tiles as there are SM pairs: none is split along K
    w, x = _all_positive(40, *((k, n) if bwd else (n, k)), k)
    got, want = _base(w, x, bwd, torch.bfloat16)
    share = float((got != want.float().bfloat16()).double().mean())
    assert share <= 0.0012, share
    assert float(((got.double() - want).abs() / want).max()) <= 2.0 ** -8 + 72 * U


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("k,steps", [(1024, 16), (8192, 32)])
def test_fp32_results_are_as_exact_as_fp32_sums(k, steps, bwd):
    """Accumulators of `steps` steps: the running sums 1/steps A ... A are cut by at most 2 u of them,
    (steps + 1) u A, and each of their k / (16 steps) additions rounds by u S at most.  (In accumulators of
    64 steps the cut may be 65 u.)"""
    n = 74 * 256
    w, x = _all_positive(40, *((k, n) if bwd else (n, k)), k)
    got, want = _base(w, x, bwd, torch.float32)
    off = float(((got.double() - want).abs() / want).max()) / U
    assert off <= steps + 1 + k // (16 * steps), off


@pytest.mark.parametrize("M", [1, 8, 16])
def test_decode_results_are_as_exact_as_fp32_sums(M):
    """Up to 8 tokens accumulators of 512 products, 33 u S, up to 16 of 1024, 65 u S; they are added to sums
    in registers, 4 at most for K = 8192 and a warp, or to the result, fewer than 12 for all warps: 16 u S
    at most.  (In accumulators of 2048 products the cut may be 129 u.)"""
    w, x = _all_positive(M, 74 * 256, 8192, 8192)
    got, want = _base(w, x, False, torch.float32)
    assert float(((got.double() - want).abs() / want).max()) / U <= (33 if M <= 8 else 65) + 16


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("r", [8, 64, 72, 200, 256])
def test_fp32_results_keep_24_bits_of_the_rank_r_product(r, bwd):
    """W' = 0; T (or U) = 1 + 2^-9 + 2^-18 in every rank, which two bf16 parts of 8 bits cannot hold,
    times a factor of 1 in the last 8 ranks and 0 in the others: the result 8 (1 + 2^-9 + 2^-18) and
    every partial sum of it are fp32 values, and no product lies below the last bit of such a sum, so it
    has to come out exactly."""
    M, o, h = 40, 192, 128
    w = _weight(o, h, torch.full((o * h // 2,), 0x77, device="cuda", dtype=torch.uint8))  # the code of 0
    assert float(q.qlora_dequant(w).abs().max()) == 0.0
    L1, L2 = torch.ones(2, h, r), torch.ones(2, r, o)
    wide, last = (L2.transpose(1, 2), L1) if bwd else (L1, L2.transpose(1, 2))  # [n][o or h][r]
    wide[:, :3] = torch.tensor([1.0, 2.0 ** -9, 2.0 ** -18])[None, :, None]
    last[:, :, :r - 8] = 0
    bank = q.AdapterBank(L1.bfloat16().cuda(), L2.bfloat16().cuda(), torch.ones(2, device="cuda"))
    plan = q.qlora_adapter_plan(torch.arange(M, device="cuda", dtype=torch.int32) % 2, 2)
    x = torch.zeros(M, o if bwd else h, device="cuda", dtype=torch.bfloat16)
    x[:, :3] = 1
    if bwd:
        X = torch.zeros(M, h, device="cuda", dtype=torch.bfloat16)
        y = q.qlora_multi_linear_bwd(w, X, x, bank, plan)[0]
    else:
        y = q.qlora_multi_linear_fwd(w, x, bank, plan)[0]
    want = 8 * (1 + 2.0 ** -9 + 2.0 ** -18)
    assert float(np.float32(want)) == want
    assert bool((y == want).all()), (y.min().item(), y.max().item(), want)
