"""AdamW over many tensors at once (the LoRA factors of every linear and
adapter), with the moments in 32 or in 8 bits, and in unified memory on demand.

The arithmetic runs in libqlora.so (qlora_multi_adamw_step: two launches for
all tensors, clipping by their global gradient norm included); the class holds
the flat state and the table of tensors.  PagedAdamW is the form for one flat
parameter buffer.
"""
from __future__ import annotations

import array
import ctypes
import operator
from typing import Callable, Dict, List, Optional, Sequence, Tuple, Union

import torch

from ._lib import (QLORA_DTYPE_BF16, QLORA_DTYPE_F32, _call, _check, _stream, lib, qlora_adamw_state_t, qlora_adamw_t,
                   qlora_adamw_tensor_t)
from .paged import AdamWConfig, ManagedBuffer, PagingPolicy

STATE_BLOCK = 256
ROUNDINGS = {"nearest": 0, "stochastic": 1}

_dtype, _shape = operator.attrgetter("dtype"), operator.attrgetter("shape")
_device, _contiguous, _data_ptr = torch.Tensor.get_device, torch.Tensor.is_contiguous, torch.Tensor.data_ptr


class MultiAdamW:
    """AdamW over a list of fp32 CUDA tensors, updated in place.

    params: contiguous fp32 tensors of one device, none of them empty and no two
    of them overlapping; their memory is used until the optimizer is dropped
    (a step after one of them moved, as by x.data = y, is refused);
    copies (optional): one bf16 tensor per parameter, or None, written with the
    rounded parameter after each step (the factors the layer reads).
    state_bits: 32, or 8 (E4M3 codes of m and of sqrt(v) with one fp32 scale per
    256 elements; include/qlora.h has the rule).  rounding of the 8-bit codes:
    "nearest", or "stochastic" (reproducible), which training over more than some
    hundred steps needs: nearest codes do not follow the slow average of v where
    the gradients' scale changes.  paged: state in unified memory, moved by the
    policy of PagedAdamW.

    State, flat over all tensors: ``m`` and ``v`` (fp32, or float8_e4m3fn codes;
    in 8 bits ``v`` holds sqrt(v)), ``m_scale`` and ``v_scale`` (8 bits only)
    and ``steps`` (int32, one per tensor).  Tensor i occupies the elements
    ``offsets[i] : offsets[i] + params[i].numel()``; each starts a new block of
    256."""

    def __init__(self, params: Sequence[torch.Tensor], cfg: AdamWConfig = AdamWConfig(),
                 copies: Optional[Sequence[Optional[torch.Tensor]]] = None, state_bits: int = 32, paged: bool = False,
                 watermark_bytes: int = 0, mem_info: Optional[Callable[[], Tuple[int, int]]] = None,
                 rounding: str = "nearest"):
        self.params: List[torch.Tensor] = list(params)
        self.copies = [None] * len(self.params) if copies is None else list(copies)
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if rounding not in ROUNDINGS or (rounding != "nearest" and state_bits != 8):
            raise ValueError(f"rounding must be one of {sorted(ROUNDINGS)}, and 'nearest' with 32-bit state")
        if not self.params:
            raise ValueError("params is empty")
        if len(self.copies) != len(self.params):
            raise ValueError(f"{len(self.copies)} copies for {len(self.params)} params")
        for i, (p, c) in enumerate(zip(self.params, self.copies)):
            if not (p.is_cuda and p.dtype == torch.float32 and p.is_contiguous() and p.numel() > 0):
                raise ValueError(f"params[{i}] must be a non-empty contiguous fp32 CUDA tensor")
            if p.device != self.params[0].device:
                raise ValueError(f"params[{i}] is on {p.device}, params[0] on {self.params[0].device}")
            if c is not None and (c.dtype != torch.bfloat16 or c.shape != p.shape or not c.is_contiguous() or
                                  c.device != p.device):
                raise ValueError(f"copies[{i}] must be a contiguous bf16 tensor shaped like its parameter")
        spans = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size())
                       for p in self.params + [c for c in self.copies if c is not None])
        for (_, end), (start, _) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError("params and copies overlap in memory")
        self.cfg, self.state_bits, self.rounding = cfg, state_bits, rounding
        self.device = self.params[0].device
        self._numel = [p.numel() for p in self.params]
        self._shapes = [p.shape for p in self.params]
        self.offsets: List[int] = []
        total = 0
        for n in self._numel:
            self.offsets.append(total)
            total += -(-n // STATE_BLOCK) * STATE_BLOCK
        self._elems = total
        self._buffers: List[ManagedBuffer] = []
        dt = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        self.m, self.v = (self._state(total, dt, paged) for _ in range(2))
        self.m_scale = self.v_scale = None
        if state_bits == 8:
            self.m_scale, self.v_scale = (self._state(total // STATE_BLOCK, torch.float32, paged) for _ in range(2))
        self.steps = torch.zeros(len(self.params), dtype=torch.int32, device=self.device)
        self.watermark = int(watermark_bytes)
        self.policy = PagingPolicy(sum(b.nbytes for b in self._buffers), self.watermark,
                                   mem_info or (lambda: torch.cuda.mem_get_info(self.device)), self._move)
        self._make_plan()

    def _state(self, numel: int, dtype: torch.dtype, paged: bool) -> torch.Tensor:
        if not paged:
            return torch.zeros(numel, dtype=torch.uint8 if dtype.itemsize == 1 else dtype,
                               device=self.device).view(dtype)
        buf = ManagedBuffer(-(-numel * dtype.itemsize // 4), self.device)
        buf.tensor.zero_()
        self._buffers.append(buf)
        return buf.tensor.view(dtype)[:numel]

    def _make_plan(self) -> None:
        n = len(self.params)
        self._places = self._addresses()
        table = (qlora_adamw_tensor_t * n)()
        for e, p, c in zip(table, self.params, self.copies):
            e.param, e.copy, e.n = p.data_ptr(), None if c is None else c.data_ptr(), p.numel()
        L = lib()
        size = L.qlora_multi_adamw_plan_size(n, self._elems)
        self._plan = torch.empty(size, dtype=torch.uint8, device=self.device)
        with torch.cuda.device(self.device):
            _check(L.qlora_multi_adamw_plan(ctypes.cast(table, ctypes.c_void_p), n,
                                            ctypes.c_void_p(self._plan.data_ptr()), size, _stream(self.device)),
                   "qlora_multi_adamw_plan")
        st = qlora_adamw_state_t()
        st.m, st.v = self.m.data_ptr(), self.v.data_ptr()
        if self.state_bits == 8:
            st.m_scale, st.v_scale = self.m_scale.data_ptr(), self.v_scale.data_ptr()
        st.steps, st.bits, st.rounding = self.steps.data_ptr(), self.state_bits, ROUNDINGS[self.rounding]
        self._struct = st

    def _addresses(self) -> List[int]:
        return list(map(_data_ptr, self.params)) + [c.data_ptr() for c in self.copies if c is not None]

    def _move(self, to_host: bool) -> None:
        for b in self._buffers:
            b.advise(prefer_host=to_host)
            b.prefetch(to_host=to_host)

    def evict(self) -> None:
        """Send the state to host RAM now (paged state only)."""
        if not self._buffers:
            raise ValueError("the state is not paged")
        if not self.policy.on_host:
            self._move(True)
            self.policy.on_host = True
            self.policy.moves.append("to_host")

    def step(self, grads: Sequence[Optional[torch.Tensor]]) -> None:
        """One step: grads[i] (fp32 or bf16, all the same type, shaped like
        params[i]) or None, which leaves parameter, state and step count i as
        they are.  The gradients are not modified.  May be captured into a CUDA
        graph: the step counts live on the device.  A captured step keeps what the
        call was given for good: the gradients' addresses, which of them are None,
        and the numbers of cfg (learning rate, clipping bound and the others), so a
        changed learning rate needs a new capture."""
        grads = list(grads)
        if len(grads) != len(self._numel):
            raise ValueError(f"{len(grads)} grads for {len(self._numel)} params")
        if self._addresses() != self._places:
            raise ValueError("params or copies have moved since the optimizer was made")
        at = [i for i, g in enumerate(grads) if g is not None]
        if not at:
            return
        given, shapes = grads, self._shapes
        if len(at) < len(grads):
            given, shapes = [grads[i] for i in at], [self._shapes[i] for i in at]
        # whole lists at once: a model has hundreds of tensors, and a step takes a few hundred microseconds
        dtypes = set(map(_dtype, given))
        if len(dtypes) != 1 or not dtypes <= {torch.float32, torch.bfloat16}:
            raise ValueError(f"grads must all be fp32 or all be bf16, not {sorted(map(str, dtypes))}")
        if list(map(_shape, given)) != shapes or set(map(_device, given)) != {self.device.index} or \
                not all(map(_contiguous, given)):
            for i, g, s in zip(at, given, shapes):
                if g.shape != s or g.device != self.device or not g.is_contiguous():
                    raise ValueError(f"grads[{i}] must be a contiguous tensor of shape {tuple(s)} on {self.device}")
        found = list(map(_data_ptr, given))
        if len(at) < len(grads):
            ptrs = [0] * len(grads)
            for i, x in zip(at, found):
                ptrs[i] = x
            found = ptrs
        ptrs = (ctypes.c_uint64 * len(found)).from_buffer(array.array("Q", found))
        if self._buffers and (self.watermark > 0 or self.policy.on_host):
            self.policy.on_step()
        c = self.cfg
        hp = qlora_adamw_t(c.lr, c.beta1, c.beta2, c.eps, c.weight_decay, float(c.max_grad_norm or 0.0), 0)
        _call(lib().qlora_multi_adamw_step, "qlora_multi_adamw_step", self.device, self._plan.data_ptr(),
              self._plan.numel(), len(found), self._elems, ptrs,
              QLORA_DTYPE_F32 if torch.float32 in dtypes else QLORA_DTYPE_BF16, ctypes.byref(self._struct),
              ctypes.byref(hp))

    def moments(self, i: int) -> Tuple[torch.Tensor, torch.Tensor]:
        """m and v of tensor i in fp32, shaped like it, decoded from 8 bits where they are held so."""
        a, n = self.offsets[i], self._numel[i]
        out = []
        for x, scale in ((self.m, self.m_scale), (self.v, self.v_scale)):
            y = x[a:a + n].float()
            if scale is not None:
                first = a // STATE_BLOCK
                y = y * scale[first:first - (-n // STATE_BLOCK)].repeat_interleave(STATE_BLOCK)[:n]
            out.append(y.view(self._shapes[i]))
        return out[0], out[1] if self.state_bits == 32 else out[1].square()

    def state_dict(self) -> Dict[str, torch.Tensor]:
        """Copies of the flat state and the step counts."""
        names = ("m", "v", "m_scale", "v_scale", "steps")
        return {k: getattr(self, k).clone() for k in names if getattr(self, k) is not None}

    def load_state(self, state: Dict[str, torch.Tensor], steps: Union[int, torch.Tensor, None] = None) -> None:
        """Takes state as state_dict gives it; ``steps`` (one number for all
        tensors, or one each) replaces its step counts."""
        want = ("m", "v") + (("m_scale", "v_scale") if self.state_bits == 8 else ())
        for k in want:
            mine = getattr(self, k)
            if k not in state or state[k].shape != mine.shape or state[k].dtype != mine.dtype:
                raise ValueError(f"state[{k!r}] must be a {mine.dtype} tensor of {mine.numel()} elements")
        if steps is None:
            if "steps" not in state:
                raise ValueError("state has no 'steps'")
            steps = state["steps"]
        if isinstance(steps, torch.Tensor) and steps.shape != self.steps.shape:
            raise ValueError(f"steps must have {self.steps.numel()} entries")
        if (int(steps.min()) if isinstance(steps, torch.Tensor) else int(steps)) < 0:
            raise ValueError("steps holds a negative count")
        for k in want:
            getattr(self, k).copy_(state[k])
        if isinstance(steps, torch.Tensor):
            self.steps.copy_(steps)
        else:
            self.steps.fill_(int(steps))

    def close(self) -> None:
        """Frees paged state; the optimizer cannot step afterwards."""
        if self._buffers:
            self.m = self.v = self.m_scale = self.v_scale = None
            self._struct = qlora_adamw_state_t()
        for b in self._buffers:
            b.free()
        self._buffers = []
