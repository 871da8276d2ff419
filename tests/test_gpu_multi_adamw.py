"""GPU tests of the many-tensor AdamW step (states in 32 and in 8 bits) against
the formulas in fp64, one step at a time from the state the kernel left.

Tolerances, with u = 2^-24 (half a step of fp32, relative):
  m' = m + (1 - b1)(g c - m): the clipped gradient, the difference, its product
    and the sum round once each: |err| <= u (|m'| + 3 (1 - b1)(|g| + |m|)), under
    4 u (|m| + |g|).
  v' = b2 v + (1 - b2)(g c)^2: all terms positive, five roundings in a chain: 8 u v'.
  p' = p d - s m'/(sqrt(v')/q + e): two roundings on p; on the quotient those of
    v' (half, by the root), the root, its division, the sum, the division, the
    product and s, q and d themselves: 16 u on |upd|, and m's own error:
    |err| <= 3 u |p| + 16 u |upd| + s / den 4 u (|m| + |g|); each is doubled below
    for the clipping factor's own rounding.
  A code of 8 bits is off by half a step: 2^-4 of the value, or half the smallest
    code (2^-10 of 448 / max) below the normal range; a positive root is at least
    2^-9 units.  2^-20 more covers the fp32 rounding of the scale and the factor.
    v itself is an fp32 value: below 2^-126 its two products and their sum round to
    multiples of 2^-149, off by 3/2 of one, so the root is off by at most
    sqrt(2^-148) = 2^-74, and is 0 where v is under half of 2^-149."""
import math

import numpy as np
import pytest
import torch

from bit_nf4_quantized_blockwise_b200 import MultiAdamW
from bit_nf4_quantized_blockwise_b200.paged import AdamWConfig

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CFG = AdamWConfig(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, max_grad_norm=0.3)
SHAPES = [(1,), (255,), (256,), (257,), (33, 17), (1024, 16), (16, 1000), (4099,), (3,)]
f32 = lambda x: float(np.float32(x))  # noqa: E731


def _tensors(shapes, seed=0, shift=0, std=0.02):
    """Tensors of the given shapes, each `shift` elements into its own buffer."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for sh in shapes:
        n = math.prod(sh)
        buf = torch.zeros(n + shift + 8, device="cuda")
        buf[shift:shift + n] = torch.randn(n, generator=g).cuda() * std
        out.append(buf[shift:shift + n].view(sh))
    return out


def _grads(shapes, step, dtype=torch.float32, shift=0, scale=None):
    s = (0.002 if step % 2 else 0.05) if scale is None else scale
    out = []
    for t in _tensors(shapes, seed=1000 + step, std=s):
        buf = torch.zeros(t.numel() + shift, device="cuda", dtype=dtype)
        buf[shift:] = t.reshape(-1).to(dtype)
        out.append(buf[shift:].view(t.shape))
    return out


def _d(t):
    return t.detach().double().cpu().numpy()


def _check_step(opt, grads, cfg=CFG):
    """One step of opt, checked against fp64 from the state it starts with."""
    p0 = [_d(p) for p in opt.params]
    mv0 = [tuple(_d(x) for x in opt.moments(i)) for i in range(len(p0))]
    before = opt.state_dict()
    t0 = opt.steps.tolist()
    g = [None if x is None else _d(x) for x in grads]
    opt.step(grads)
    torch.cuda.synchronize()
    norm = math.sqrt(sum(float((x ** 2).sum()) for x in g if x is not None))
    clip = 1.0 if not cfg.max_grad_norm else min(1.0, f32(cfg.max_grad_norm) / (norm + 1e-6))
    b1, b2, lr, wd, eps = (f32(x) for x in (cfg.beta1, cfg.beta2, cfg.lr, cfg.weight_decay, cfg.eps))
    for i, gi in enumerate(g):
        p1 = _d(opt.params[i])
        a, n = opt.offsets[i], p1.size
        if gi is None:
            assert np.array_equal(p1, p0[i]) and int(opt.steps[i]) == t0[i]
            for k in ("m", "v"):
                assert torch.equal(before[k][a:a + n].view(torch.uint8), getattr(opt, k)[a:a + n].view(torch.uint8))
            continue
        t = t0[i] + 1
        assert int(opt.steps[i]) == t
        gc = gi * clip
        m = mv0[i][0] + (1 - b1) * (gc - mv0[i][0])
        v = b2 * mv0[i][1] + (1 - b2) * gc ** 2
        s, q = lr / (1 - b1 ** t), math.sqrt(1 - b2 ** t)
        den = np.sqrt(v) / q + eps
        upd = s * m / den
        p = p0[i] * (1 - lr * wd) - upd
        merr = 8 * U * (np.abs(mv0[i][0]) + np.abs(gc))
        assert np.all(np.abs(p1 - p) <= 2 * (3 * U * np.abs(p0[i]) + 16 * U * np.abs(upd) + s / den * merr) + 1e-45)
        if opt.copies[i] is not None:
            assert torch.equal(opt.copies[i], opt.params[i].to(torch.bfloat16))
        m1, v1 = (_d(x) for x in opt.moments(i))
        if opt.state_bits == 32:
            assert np.all(np.abs(m1 - m) <= merr + 1e-45) and np.all(np.abs(v1 - v) <= 16 * U * v + 1e-45)
            continue
        nb = -(-n // 256)
        for x, code, scale, root in ((m, opt.m, opt.m_scale, False), (np.sqrt(v), opt.v, opt.v_scale, True)):
            x = np.concatenate([x.reshape(-1), np.zeros(nb * 256 - n)]).reshape(nb, 256)
            c = _d(scale[a // 256:a // 256 + nb])
            top = np.abs(x).max(1)
            assert np.all(np.abs(c - top / 448) <= 2.0 ** -20 * top / 448 + merr.max() / 448)
            got = _d(code[a:a + nb * 256].float()).reshape(nb, 256) * c[:, None]
            unit = c[:, None] * 2.0 ** -9
            tol = np.maximum(np.abs(x) * (2.0 ** -4 + 2.0 ** -20), unit * 0.5001) + 2 * merr.max()
            if root:
                tol = tol + 2.0 ** -74
                assert np.all(got[x > 2.0 ** -74] > 0)
                tol = np.where((x > 0) & (x < unit), unit * 1.0001 + 2 * merr.max() + 2.0 ** -74, tol)
            live = np.arange(nb * 256).reshape(nb, 256) < n
            assert np.all((np.abs(got - x) <= tol)[live])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1])
def test_steps_match_formulas(bits, dtype, shift):
    params = _tensors(SHAPES, shift=shift)
    copies = [torch.zeros(p.shape, dtype=torch.bfloat16, device="cuda") if i % 3 else None for i, p in enumerate(params)]
    opt = MultiAdamW(params, CFG, copies=copies, state_bits=bits)
    for t in range(1, 6):
        _check_step(opt, _grads(SHAPES, t, dtype, shift))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("norm", [None, 0.3])
def test_tensors_without_gradient_stand_still(bits, norm):
    cfg = AdamWConfig(lr=1e-3, max_grad_norm=norm)
    opt = MultiAdamW(_tensors(SHAPES), cfg, state_bits=bits)
    for t in range(1, 5):
        g = _grads(SHAPES, t)
        for i in range(len(g)):
            if (i + t) % 3 == 0:
                g[i] = None
        _check_step(opt, g, cfg)
    assert len(set(opt.steps.tolist())) > 1
    n = opt.steps.clone()
    opt.step([None] * len(SHAPES))
    assert torch.equal(n, opt.steps)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_and_tiny_gradients(bits):
    opt = MultiAdamW(_tensors(SHAPES), CFG, state_bits=bits)
    _check_step(opt, _grads(SHAPES, 1, scale=0.0))
    _check_step(opt, _grads(SHAPES, 2, scale=1e-18))
    _check_step(opt, _grads(SHAPES, 3, scale=0.0))
    assert all(torch.isfinite(p).all() for p in opt.params)


def test_wide_range_in_a_block_keeps_the_denominator():
    # Gradients from 1 down to 1e-9 in one block: sqrt(v) of the small ones is below the
    # smallest code; it must not become 0, or a later step without gradient would divide by eps.
    p = torch.zeros(256, device="cuda")
    g = torch.logspace(0, -9, 256, device="cuda")
    opt = MultiAdamW([p], AdamWConfig(lr=1e-3, max_grad_norm=None), state_bits=8)
    for _ in range(3):
        opt.step([g])
    opt.step([torch.zeros_like(g)])
    assert float(p.abs().max()) <= 5e-3


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_and_parameter_lists_past_one_launch(bits):
    shapes = [(1 + 7 * (i % 61),) for i in range(1100)]
    opt = MultiAdamW(_tensors(shapes), CFG, state_bits=bits)
    for t in (1, 2):
        g = _grads(shapes, t)
        g[497] = g[1099] = None
        _check_step(opt, g)


@pytest.mark.parametrize("bits", [32, 8])
def test_large_tensors_are_deterministic_and_equal_small_lists(bits):
    # the same tensors alone or in a list: identical when nothing is clipped; and run to run
    cfg = AdamWConfig(lr=1e-3, max_grad_norm=None)
    shapes = [(2048, 1024), (1000, 333), (5,)]
    runs = []
    for split in (False, True, False):
        params = _tensors(shapes)
        opts = [MultiAdamW([p], cfg, state_bits=bits) for p in params] if split else [MultiAdamW(params, cfg, state_bits=bits)]
        for t in (1, 2, 3):
            g = _grads(shapes, t)
            if split:
                for o, x in zip(opts, g):
                    o.step([x])
            else:
                opts[0].step(g)
        runs.append(params)
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


def test_clipped_steps_repeat_bit_for_bit():
    outs = []
    for _ in range(2):
        params = _tensors([(3000, 1000), (77,)])
        opt = MultiAdamW(params, CFG, state_bits=8)
        for t in (2, 4):
            opt.step(_grads([(3000, 1000), (77,)], t))
        outs.append(params + [opt.m.view(torch.uint8), opt.v.view(torch.uint8)])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_replays_as_the_next_steps(bits):
    def fresh():
        return MultiAdamW(_tensors(SHAPES), CFG, state_bits=bits)
    eager, graphed = fresh(), fresh()
    g = _grads(SHAPES, 2)
    for _ in range(4):
        eager.step(g)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graphed.step(g)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step(g)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert eager.steps.tolist() == graphed.steps.tolist() == [4] * len(SHAPES)
    for a, b in zip(eager.params, graphed.params):
        assert torch.equal(a, b)


def test_paged_state_gives_the_same_steps():
    outs = []
    for paged in (False, True):
        params = _tensors(SHAPES)
        opt = MultiAdamW(params, CFG, state_bits=8, paged=paged)
        for t in range(1, 5):
            if paged and t in (2, 4):
                opt.evict()
            opt.step(_grads(SHAPES, t))
        torch.cuda.synchronize()
        outs.append([p.clone() for p in params])
        opt.close()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_gradient_stays_in_its_element_or_block(bits, value):
    p = _tensors([(1024,)])
    opt = MultiAdamW(p, AdamWConfig(lr=1e-3, max_grad_norm=None), state_bits=bits)
    g = _grads([(1024,)], 1)
    g[0][300] = value
    opt.step(g)
    assert torch.isnan(p[0]).nonzero().view(-1).tolist() == [300]
    opt.step(_grads([(1024,)], 2))
    bad = torch.isnan(p[0]).nonzero().view(-1).tolist()
    assert bad == (list(range(256, 512)) if bits == 8 and value == float("inf") else [300])


def _encode(x, floor):
    """E4M3 codes and scales of blocks of 256 by fp32 operations on the CPU."""
    top = x.abs().amax(1)
    y = x * (torch.full_like(top, 448.0) / top)[:, None]
    if floor:
        y = torch.where((y > 0) & (y < 2.0 ** -9), torch.full_like(y, 2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn), top / torch.full_like(top, 448.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_codes_and_scales_are_those_of_ieee_arithmetic(dtype):
    """Bit for bit over several steps: a value on the other side of a rounding boundary would be a
    whole code off, and the next step's parameter with it.  400 thousand elements a step."""
    shapes = [(1000, 256), (600, 256)]
    opt = MultiAdamW(_tensors(shapes), CFG, state_bits=8)
    m = v = torch.zeros(1600, 256)
    b1, b2 = f32(CFG.beta1), f32(CFG.beta2)
    c1, c2 = float(np.float32(1) - np.float32(b1)), float(np.float32(1) - np.float32(b2))
    for t in range(1, 5):
        grads = _grads(shapes, t, dtype)
        opt.step(grads)
        g = torch.cat([x.float().cpu() for x in grads])
        norm = math.sqrt(float(g.double().square().sum()))
        g = g * torch.tensor(min(1.0, f32(CFG.max_grad_norm) / (norm + 1e-6)), dtype=torch.float32)
        m = m + (g - m) * c1
        r = torch.from_numpy(np.sqrt((v.square() * b2 + (g * g) * c2).numpy()))  # torch's own is not to nearest on the CPU
        (mc, ms), (rc, rs) = _encode(m, False), _encode(r, True)
        for got, want in ((opt.m, mc), (opt.v, rc)):
            assert torch.equal(got.cpu().view(torch.uint8), want.view(-1).view(torch.uint8))
        assert torch.equal(opt.m_scale.cpu(), ms) and torch.equal(opt.v_scale.cpu(), rs)
        m, v = mc.float() * ms[:, None], rc.float() * rs[:, None]


@pytest.mark.parametrize("bits", [32, 8])
def test_moments_of_a_nan_gradient_are_nan(bits):
    opt = MultiAdamW(_tensors([(1024,)]), AdamWConfig(lr=1e-3, max_grad_norm=None), state_bits=bits)
    g = _grads([(1024,)], 1)
    g[0][300] = float("nan")
    for t in (2, 3):
        opt.step(g)
        for x in opt.moments(0):
            assert torch.isnan(x).nonzero().view(-1).tolist() == [300]
        g = _grads([(1024,)], t)


def test_state_moves_between_optimizers():
    a = MultiAdamW(_tensors(SHAPES), CFG, state_bits=8)
    for t in (1, 2):
        a.step(_grads(SHAPES, t))
    b = MultiAdamW([p.clone() for p in a.params], CFG, state_bits=8)
    b.load_state(a.state_dict())
    for o in (a, b):
        o.step(_grads(SHAPES, 3))
    for x, y in zip(a.params, b.params):
        assert torch.equal(x, y)


def test_refusals_on_the_device():
    p = _tensors([(8, 4)])
    opt = MultiAdamW(p, CFG)
    good = torch.zeros(8, 4, device="cuda")
    for bad in ([], [good, good], [good[:4]], [good.half()], [good.cpu()], [good.t().contiguous().t()]):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(ValueError):
        opt.evict()
    buf = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        MultiAdamW([buf[:40], buf[39:]])
    with pytest.raises(ValueError, match="overlap"):
        MultiAdamW([buf, buf])
    with pytest.raises(ValueError):
        opt.load_state({"m": opt.m, "v": opt.v})
    assert opt.steps.tolist() == [0]
