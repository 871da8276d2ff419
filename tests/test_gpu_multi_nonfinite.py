"""GPU tests of infinities and NaN in the many-adapter layer: every element is what its formula gives
from its own token and adapter, +inf, -inf and NaN told apart, whatever else is in the batch.

The formulas are evaluated in 64 bits, where the finite numbers of these cases neither overflow nor
vanish, so a result is infinite or NaN for the infinities and NaN in its own terms alone.  Finite
elements have the bounds of the layer's other tests."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_blockwise_b200 as q
from test_gpu_multi_linear import Case, rounded

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def _mm(a, b):
    """a b by plain products and sums (a library product may add zeros times what is not asked for)."""
    with np.errstate(invalid="ignore"):
        return np.stack([(row[:, None] * b).sum(0) for row in a]) if len(a) else np.zeros((0, b.shape[1]))


def _formulas(c):
    X, dY, L1, L2, s = c.f64()
    with np.errstate(invalid="ignore"):
        Y, dX = _mm(X, c.W.T), _mm(dY, c.W)
        d1, d2 = np.zeros(L1.shape), np.zeros(L2.shape)
        for a in range(c.n):
            at = np.nonzero(c.ids == a)[0]
            if not at.size:
                continue
            T, U = s[a] * _mm(X[at], L1[a]), s[a] * _mm(dY[at], L2[a].T)
            Y[at] += _mm(T, L2[a])
            dX[at] += _mm(U, L1[a].T)
            d1[a], d2[a] = _mm(X[at].T, U), _mm(T.T, dY[at])
    return Y, dX, d1, d2


def _same(got, want, bound, what):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)), (what, "NaN", int(np.isnan(got).sum()), int(np.isnan(want).sum()))
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], want[inf]), (what, "inf")
    fine = np.isfinite(want)
    assert np.all(np.abs(got[fine] - want[fine]) <= bound[fine] + 1e-30), what


def _check(c, spoil, dtype=torch.float32, grads=True):
    _, bY, _, _ = c.forward()
    _, bX, _, b1, _, b2 = c.backward()
    spoil(c)
    Y, dX, d1, d2 = _formulas(c)
    bank, plan = c.device()
    x, dy = c.X.cuda(), c.dY.cuda()
    y, T = q.qlora_multi_linear_fwd(c.Wq, x, bank, plan, y_dtype=dtype)
    dx, g1, g2 = q.qlora_multi_linear_bwd(c.Wq, x, dy, bank, plan, T_saved=T, dx_dtype=dtype)
    torch.cuda.synchronize()
    q.qlora_check_status()
    fin = lambda v: np.where(np.isfinite(v), v, 0.0)  # noqa: E731
    _same(y, Y, rounded(fin(Y), bY, dtype), "Y")
    _same(dx, dX, rounded(fin(dX), bX, dtype), "dX")
    if grads:
        _same(g1, d1, b1, "dL1")
        _same(g2, d2, b2, "dL2")


def _one(c):
    return int(np.nonzero(c.ids == 1)[0][0])


def _others(c):
    """Infinities and NaN in an adapter that those rows do not use."""
    c.L2[2, 2, 9], c.L2[2, 3, 10] = INF, NAN
    c.L1[2, 7, 2], c.L1[2, 8, 3] = -INF, NAN


def _rows(c, value):
    none = np.nonzero(c.ids < 0)[0]
    rows = ([int(none[0])] if none.size else []) + [_one(c)]
    for i in rows:
        c.X[i, 3] = c.dY[i, 5] = value


SPOILS = {
    # an infinite activation and gradient of a token without adapter and of one with, beside an
    # adapter of infinities and NaN
    "rows": lambda c: (_rows(c, INF), _others(c)),
    "rows -inf": lambda c: (_rows(c, -INF), _others(c)),
    "two infinities": lambda c: (_rows(c, INF), c.X.__setitem__((_one(c), 4), INF), c.dY.__setitem__((_one(c), 6), -INF)),
    # one infinite element of the tokens' own factors
    "own L2": lambda c: c.L2.__setitem__((1, 2, 9), INF),
    "own L1": lambda c: c.L1.__setitem__((1, 7, 2), -INF),
    "own L1 and L2": lambda c: (c.L1.__setitem__((1, 7, 2), INF), c.L2.__setitem__((1, 3, 9), -INF)),
}


@pytest.mark.parametrize("M,kind", [(20, "mixed"), (150, "mixed"), (300, "runs"), (600, "mixed")])
@pytest.mark.parametrize("what", list(SPOILS))
def test_mixed_batches(M, kind, what):
    _check(Case(M, 256, 320, 3, 16, kind=kind, none=0.1, seed=M), SPOILS[what])


@pytest.mark.parametrize("what", list(SPOILS)[2:])
@pytest.mark.parametrize("M", [20, 256, 300])
def test_one_adapter_alone(M, what):
    """Tiles that no other adapter's tokens share."""
    c = Case(M, 256, 320, 2, 16, kind="runs", seed=M)
    c.ids[:] = 1
    _check(c, SPOILS[what])


@pytest.mark.parametrize("what", ["rows", "own L2", "own L1"])
def test_bf16_results(what):
    _check(Case(300, 256, 320, 3, 72, kind="mixed", none=0.1, seed=5), SPOILS[what], dtype=torch.bfloat16)


@pytest.mark.parametrize("what", ["rows", "own L2"])
def test_more_tiles_than_pairs(what):
    """Tiles of whole rounds and of the split last one."""
    _check(Case(2100, 512, 2368, 3, 8, kind="mixed", none=0.1, seed=6), SPOILS[what], grads=False)
