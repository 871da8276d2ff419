"""GPU tests of the 8-bit AdamW state at its edges: an eps below the normal numbers, and the moments
over thousands of steps."""
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


def _two_optimizers(scale_of, steps, **kw):
    """sqrt(v) of an 8-bit optimizer over that of a 32-bit one, after `steps` steps of the same
    gradients: normal ones times scale_of(t), 64 blocks."""
    cfg = AdamWConfig(lr=1e-4, max_grad_norm=None)
    params = [torch.zeros(64, 256, device="cuda") for _ in range(2)]
    a, b = MultiAdamW(params[:1], cfg, state_bits=8, **kw), MultiAdamW(params[1:], cfg)
    g = torch.Generator(device="cuda").manual_seed(4)
    for t in range(steps):
        x = [torch.randn(64, 256, device="cuda", generator=g) * scale_of(t)]
        a.step(x)
        b.step(x)
    return (a.moments(0)[1] / b.moments(0)[1]).sqrt(), params


def _change(factor):
    def scale_of(t):
        s = torch.ones(256, device="cuda")
        s[128:] = factor if t >= 300 else 1.0
        return s
    return scale_of


@pytest.mark.parametrize("factor", [1.0, 0.1, 4.0])
def test_the_second_moment_follows_its_average(factor):
    """3000 steps at beta2 = 0.999, the gradients of half of each block changing by `factor` at step 300.
    Codes rounded without bias: each step moves r by a share d of about 0.0008 (0.0005 of decay, as much
    of the gradients), and rounding to codes a step of h = 0.06 to 0.125 apart gives a variance of d h at
    most, which the average forgets at 0.0005 a step for r: a standard deviation of sqrt(0.0008 0.125 /
    (2 0.0005)) = 0.32 at most, and a mean of r that is high by half that variance, 0.05.  So the mean
    over 8192 elements lies within 0.06 (three standard deviations of it are 0.01), and 95 % of the
    elements within a factor of 2 (ln 2 is 2.1 standard deviations: 96 %).  A half that shrank tenfold is
    still above its new size after 2700 steps (e^-1.35 of the old r), which the 32-bit average has too."""
    ratio, params = _two_optimizers(_change(factor), 3000, rounding="stochastic")
    for half in (ratio[:, :128], ratio[:, 128:]):
        x = half.double().cpu().numpy().reshape(-1)
        assert abs(x.mean() - 1) <= 0.06, x.mean()
        assert np.mean((x > 0.5) & (x < 2.0)) >= 0.95
    assert all(torch.isfinite(p).all() for p in params)


def _stepped(steps, seed=7, opt=None, graph=False):
    cfg = AdamWConfig(lr=1e-3, max_grad_norm=0.3)
    g = torch.Generator(device="cuda").manual_seed(seed)
    shapes = [(1000, 256), (333,), (64, 257)]
    params = [torch.randn(s, device="cuda", generator=g) * 0.02 for s in shapes]
    grads = [torch.randn(s, device="cuda", generator=g) * 0.01 for s in shapes]
    opt = MultiAdamW(params, cfg, state_bits=8, rounding="stochastic")
    for k in range(steps):
        if graph and k == 1:
            cg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cg):
                opt.step(grads)
        if graph and k >= 1:
            cg.replay()
        else:
            opt.step(grads)
    torch.cuda.synchronize()
    return opt, grads


def _bits(opt):
    return [p.view(torch.int32) for p in opt.params] + [opt.m.view(torch.uint8), opt.v.view(torch.uint8), opt.m_scale,
                                                        opt.v_scale, opt.steps]


def test_stochastic_codes_are_neighbours_and_their_mean_is_the_value():
    """One step from zero state against the fp32 moments (of which 32-bit state tells).  A code is one of
    the two values around x, so off by less than their distance, 2^-3 of x at most (2^-9 units below 2^-6
    units).  The errors of n elements, each of at most that range and independent, have a mean within 6
    standard deviations, 6 / 2 of the rms distance over sqrt(n), of 0; plus 2^-16 of a distance for the
    random bits' number, 2^-22 of x for the scale and the factor."""
    params = [torch.zeros(4096, 256, device="cuda") for _ in range(2)]
    cfg = AdamWConfig(lr=1e-3, max_grad_norm=None)
    a, b = MultiAdamW(params[:1], cfg, state_bits=8, rounding="stochastic"), MultiAdamW(params[1:], cfg)
    g = torch.randn(4096, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    g *= torch.logspace(0, -7, 256, device="cuda")  # down into the smallest codes
    for o in (a, b):
        o.step([g])
    for x, code, scale, root in ((b.moments(0)[0], a.m, a.m_scale, False), (b.moments(0)[1].sqrt(), a.v, a.v_scale, True)):
        c = scale.double()[:, None]
        y = x.double() / c
        got = code.float().double().view(4096, 256)
        dist = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        err = got - y
        assert bool((err.abs() <= dist + 2.0 ** -20 * y.abs()).all())
        assert float((err != 0).double().mean()) > 0.9
        fine = y.abs() >= 2.0 ** -9 if root else y.abs() >= 0  # a positive root below the smallest code takes it
        e = (err * y.sign())[fine]  # away from 0 positive, so that a bias by size is seen
        d = dist[fine]
        tol = 3 * float((d ** 2).mean().sqrt()) / e.numel() ** 0.5 + float(d.mean()) * 2.0 ** -16 + \
            float(y.abs()[fine].mean()) * 2.0 ** -22
        assert abs(float(e.mean())) <= tol, (float(e.mean()), tol)
        # neighbours draw independently: the correlation of n pairs is within 5 / sqrt(n)
        u = (err / dist)[:, :128]
        u = (u - u.mean(0)) / u.std(0)
        assert abs(float((u[:, 1:] * u[:, :-1]).mean())) <= 5 / (4096 * 127) ** 0.5
        assert abs(float((u[1:] * u[:-1]).mean())) <= 5 / (4095 * 128) ** 0.5
    # the parameter's step does not see the codes
    n = torch.zeros(4096, 256, device="cuda")
    MultiAdamW([n], cfg, state_bits=8).step([g])
    assert torch.equal(n, params[0])


def test_stochastic_steps_repeat_replay_and_continue():
    a, grads = _stepped(6)
    for b in (_stepped(6)[0], _stepped(6, graph=True)[0]):
        for x, y in zip(_bits(a), _bits(b)):
            assert torch.equal(x, y)
    b, _ = _stepped(3)
    c = MultiAdamW([p.clone() for p in b.params], b.cfg, state_bits=8, rounding="stochastic")
    c.load_state(b.state_dict())
    for _ in range(3):
        c.step(grads)
    for x, y in zip(_bits(a), _bits(c)):
        assert torch.equal(x, y)
    d, _ = _stepped(3)
    assert not torch.equal(d.v.view(torch.uint8), a.v.view(torch.uint8))


def test_stochastic_codes_of_nan_and_of_blocks_of_zeros():
    p = torch.zeros(1024, device="cuda")
    opt = MultiAdamW([p], AdamWConfig(lr=1e-3, max_grad_norm=None), state_bits=8, rounding="stochastic")
    g = torch.randn(1024, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    g[:256] = 0
    g[300] = float("nan")
    for _ in range(3):
        opt.step([g])
        for x in opt.moments(0):
            assert torch.isnan(x).nonzero().view(-1).tolist() == [300]
            assert bool((x[:256] == 0).all())
        g[300] = 0
    assert torch.isnan(p).nonzero().view(-1).tolist() == [300] and bool((p[:256] == 0).all())
