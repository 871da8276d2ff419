"""GPU test of factor gradients whose tokens are dealt to several CTAs (fewer tiles than SMs): the
parts are added in order, by each epilogue warp for its own rows."""
import pytest
import torch

import bit_nf4_quantized_blockwise_b200 as q
from test_gpu_multi_linear import Case, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,n,h,o,r", [(1100, 1, 128, 128, 8), (1500, 3, 192, 320, 72), (256, 2, 1024, 64, 64),
                                       (4000, 5, 64, 64, 16)])
def test_gradients_in_parts(M, n, h, o, r):
    c = Case(M, h, o, n, r, kind="mixed", none=0.05, seed=M, dq=False)
    bank, plan = c.device()
    X, dY = c.X.cuda(), c.dY.cuda()
    outs = [q.qlora_multi_linear_bwd(c.Wq, X, dY, bank, plan) for _ in range(4)]
    torch.cuda.synchronize()
    q.qlora_check_status()
    _, _, w1, b1, w2, b2 = c.backward()
    near(outs[0][1], w1, b1)
    near(outs[0][2], w2, b2)
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))
