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


def _state_of(sizes):
    """A MultiAdamW with 8-bit state on the CPU, not made by its constructor."""
    from bit_nf4_quantized_blockwise_b200.multi_adamw import STATE_BLOCK, MultiAdamW
    opt = MultiAdamW.__new__(MultiAdamW)
    opt.state_bits, opt._numel, opt._shapes, opt.offsets, total = 8, list(sizes), [(n,) for n in sizes], [], 0
    for n in sizes:
        opt.offsets.append(total)
        total += -(-n // STATE_BLOCK) * STATE_BLOCK
    g = torch.Generator().manual_seed(0)
    opt.m, opt.v = (torch.randn(total, generator=g).abs().to(torch.float8_e4m3fn) for _ in range(2))
    opt.m_scale, opt.v_scale = (torch.rand(total // STATE_BLOCK, generator=g) for _ in range(2))
    return opt


@pytest.mark.parametrize("sizes", [(1,), (256,), (5, 700, 256, 257), (1000, 1)])
def test_moments_decode_their_own_blocks(sizes):
    opt = _state_of(sizes)
    m = opt.m.float() * opt.m_scale.repeat_interleave(256)
    v = (opt.v.float() * opt.v_scale.repeat_interleave(256)).square()
    for i, n in enumerate(sizes):
        a = opt.offsets[i]
        got = opt.moments(i)
        assert torch.equal(got[0], m[a:a + n]) and torch.equal(got[1], v[a:a + n])


def test_moments_of_a_small_tensor_touch_nothing_else(monkeypatch):
    """The scales of the tensors behind it are not expanded (of a large model, 4 bytes a parameter)."""
    opt = _state_of((10, 1 << 20))
    sizes = []
    repeat = torch.Tensor.repeat_interleave

    def counted(self, *args, **kw):
        out = repeat(self, *args, **kw)
        sizes.append(out.numel())
        return out
    monkeypatch.setattr(torch.Tensor, "repeat_interleave", counted)
    opt.moments(0)
    assert sizes and max(sizes) <= 256


@pytest.mark.parametrize("which", ["params", "copies"])
def test_a_step_refuses_tensors_that_have_moved(which):
    """The plan holds the addresses of params and copies: a step after x.data = y would write to memory
    that x no longer owns."""
    opt = _state_of((5, 300))
    opt.params = [torch.zeros(5), torch.zeros(300)]
    opt.copies = [None, torch.zeros(300, dtype=torch.bfloat16)]
    opt._places = opt._addresses()
    tensor = getattr(opt, which)[1]
    tensor.data = tensor.data.clone()
    with pytest.raises(ValueError, match="moved"):
        opt.step([torch.zeros(5), torch.zeros(300)])


@pytest.mark.parametrize("steps", [-1, torch.tensor([3, -2], dtype=torch.int32)])
def test_loading_refuses_negative_step_counts(steps):
    """The first step after -1 would divide by 1 - beta^0 = 0 and make every parameter NaN."""
    opt = _state_of((5, 300))
    opt.steps = torch.tensor([7, 8], dtype=torch.int32)
    state = {k: getattr(opt, k).clone() for k in ("m", "v", "m_scale", "v_scale")}
    before = opt.m.clone()
    state["m"] = torch.zeros_like(before)
    with pytest.raises(ValueError, match="negative"):
        opt.load_state(state, steps=steps)
    assert opt.steps.tolist() == [7, 8] and torch.equal(opt.m.view(torch.uint8), before.view(torch.uint8))
    opt.load_state(state, steps=torch.tensor([0, 4], dtype=torch.int32))
    assert opt.steps.tolist() == [0, 4]
