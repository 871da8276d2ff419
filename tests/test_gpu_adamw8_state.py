"""GPU tests of the many-tensor AdamW step at its edges: an eps at either end of fp32."""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_blockwise_b200 import MultiAdamW
from bit_nf4_quantized_blockwise_b200.paged import AdamWConfig

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
f32 = lambda x: float(np.float32(x))  # noqa: E731


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1.2e-38, 1e-30, 1e-8, 1e30, 3e38])
def test_every_eps_above_zero(bits, eps):
    """One step from zero state.  The quotient is m / (r / q + eps): 4 ulp, 8 u, for it, and the 12 u
    that the rest of the update rounds by (the 32-bit tests have the list), with m's own error of 8 u
    |m|.  Gradients: 0 (m = v = 0, the update 0 / eps = 0); normal ones; one whose square is below
    every fp32 value (v = 0, m / eps where that is an fp32 value)."""
    g = torch.zeros(512, device="cuda")
    g[1::4] = torch.randn(128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    tiny = 1e-26 if eps > 1e-20 else 1e-41  # m = a tenth of it
    g[258] = tiny                           # a block with normal gradients too
    p = torch.zeros(512, device="cuda")
    opt = MultiAdamW([p], AdamWConfig(lr=1e-3, eps=eps, weight_decay=0.0, max_grad_norm=None), state_bits=bits)
    opt.step([g])
    g, got = g.double().cpu().numpy(), p.double().cpu().numpy()
    b1, b2, lr, e = f32(0.9), f32(0.999), f32(1e-3), f32(eps)
    m = (1 - b1) * g
    v = np.float32((1 - b2) * np.float32(g) ** 2).astype(np.float64)
    q = np.sqrt(1 - b2)
    want = -lr / (1 - b1) * m / (np.sqrt(v) / q + e)
    step = 2.0 ** -149  # values below the normal numbers are multiples of it
    # m of the tiny gradient is itself such a multiple, and so may be the result
    tol = 40 * U * np.abs(want) + 2 * step + lr / (1 - b1) * step / (np.sqrt(v) / q + e) * (np.abs(m) < 2.0 ** -126)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= tol), (got[258], want[258], np.abs(got - want).max())
    assert np.all(got[g == 0] == 0)
