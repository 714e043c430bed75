"""AdamW over all adapters at once (qlora_adamw_step): the step that follows the linears' backward.
Takes their fp32 dA and dB (or bf16 gradients) and leaves the bf16 A and B that the next forward
reads, with moments in 32 or 8 bits and the clip of the global norm, in one or two launches
however many tensors there are.
"""

import ctypes

import torch

from . import abi
from .block import _bind
from .linear import _ptr

_BLOCK = 256


class AdamW:
    """AdamW on a fixed list of tensors.

    params: contiguous bf16 or fp32 CUDA tensors; grads: as many, bf16 or fp32, in which the
    backward leaves the gradients before each step (``linear.backward(..., dA=, dB=)`` writes
    them).  Both are bound at construction: the memory they have then is what every step reads
    and writes (a step can so be captured into a CUDA graph, and each replay takes the next one).
    masters: fp32 copies of the parameters that the step is taken on, None entries (or no list)
    where there are none; a bf16 parameter without one is rounded stochastically.  All of them start
    at multiples of 16 bytes (step raises QLoraError otherwise, and for numbers out of range).

    bits: 32 or 8 for the moments.  lr: a float, which a captured step keeps, or a CUDA fp32 tensor of
    one element that is read at every step.  lr_scales, weight_decays: one value a tensor (default
    1 and weight_decay).  max_grad_norm: clips the norm over all gradients (None or 0: not);
    grad_scale multiplies them first.  check_finite: computes the norm without a clip too.  Where
    the norm is computed and is not finite (as the fp32 number that step() returns) the step
    changes nothing but that and ``skipped``.  seed: of the stochastic rounding, which is
    reproducible.  step: steps taken before.

    State: m, v: flat over the list, tensor i from offsets[i] on (every tensor starts a block of
    256 elements): fp32, or uint8 codes with the blocks' fp32 m_scale, v_scale.  It is zeroed on the
    stream current at construction; the caller orders steps on other streams after that, and
    one step after another.
    """

    def __init__(self, params, grads, masters=None, bits=32, lr=1e-4, betas=(0.9, 0.999), eps=1e-8,
                 weight_decay=0.0, lr_scales=None, weight_decays=None, max_grad_norm=None,
                 grad_scale=1.0, check_finite=False, seed=0, step=0):
        params, grads = list(params), list(grads)
        count = len(params)
        masters = [None] * count if masters is None else list(masters)
        lr_scales = [1.0] * count if lr_scales is None else list(lr_scales)
        weight_decays = [weight_decay] * count if weight_decays is None else list(weight_decays)
        if count < 1 or not all(len(x) == count for x in (grads, masters, lr_scales,
                                                          weight_decays)):
            raise ValueError("AdamW: params, grads, masters, lr_scales and weight_decays are "
                             "lists of one length, at least one")
        if bits not in (8, 32):
            raise ValueError(f"AdamW: bits {bits} is neither 8 nor 32")
        if step < 0:
            raise ValueError(f"AdamW: step {step} is negative")
        self.device = params[0].device
        # Aliases that keep the bound memory alive whatever becomes of the caller's tensors.
        self._bound = [[None if t is None else t.detach() for t in ts]
                       for ts in (params, masters, grads)]
        self._tensors = (abi.AdamWTensor * count)()
        self._count = count
        self.offsets = []
        at = 0
        for i, (p, w, g) in enumerate(zip(*self._bound)):
            self._check(p, (torch.bfloat16, torch.float32), p.shape, f"params[{i}]")
            self._check(g, (torch.bfloat16, torch.float32), p.shape, f"grads[{i}]")
            if w is not None:
                if p.dtype is torch.float32:
                    raise ValueError(f"masters[{i}]: an fp32 parameter takes no master copy")
                self._check(w, (torch.float32,), p.shape, f"masters[{i}]")
            self._tensors[i] = abi.AdamWTensor(p.data_ptr(), _ptr(w), g.data_ptr(), p.numel(),
                                               lr_scales[i], weight_decays[i],
                                               p.dtype is torch.float32,
                                               g.dtype is torch.float32)
            self.offsets.append(at)
            at += -(-p.numel() // _BLOCK) * _BLOCK
        self._lr = lr.detach() if isinstance(lr, torch.Tensor) else None
        if self._lr is not None:
            if self._lr.numel() != 1:
                raise ValueError("lr: expected one element")
            self._check(self._lr, (torch.float32,), self._lr.shape, "lr")
        self._no_overlap()
        blocks = at // _BLOCK
        kind = torch.uint8 if bits == 8 else torch.float32
        zeros = lambda n, dtype: torch.zeros(n, dtype=dtype, device=self.device)  # noqa: E731
        # One element where there is none, so that every buffer has an address.
        self.m, self.v = zeros(max(at, 1), kind)[:at], zeros(max(at, 1), kind)[:at]
        self.m_scale = self.v_scale = None
        if bits == 8:
            self.m_scale = zeros(max(blocks, 1), torch.float32)[:blocks]
            self.v_scale = zeros(max(blocks, 1), torch.float32)[:blocks]
        self._state = zeros(16, torch.int32)
        if step:
            self._state.view(torch.int64)[0] = step
        self._norm = self._state.view(torch.float32)[2:3]
        self._config = abi.AdamWConfig(0.0 if self._lr is not None else lr, betas[0], betas[1],
                                       eps, grad_scale, max_grad_norm or 0.0, _ptr(self._lr),
                                       seed & 0xFFFFFFFF, bits, bool(check_finite))
        self._has_norm = self._config.max_norm > 0 or bool(check_finite)
        self._stream = _bind().current_stream
        self._ws = zeros(abi.qlora_adamw_workspace_bytes(count), torch.uint8)
        # What a step passes, marshalled once.
        buffer = lambda t: None if t is None else t.untyped_storage().data_ptr()  # noqa: E731
        self._args = (self._tensors, count, ctypes.byref(self._config), buffer(self.m),
                      buffer(self.v), buffer(self.m_scale), buffer(self.v_scale),
                      self._state.data_ptr(), self._ws.data_ptr(), self._ws.numel())

    def _check(self, t, dtypes, shape, name):
        if not (t.is_cuda and t.device == self.device and t.dtype in dtypes and t.shape == shape
                and t.is_contiguous()):
            raise ValueError(f"{name}: expected contiguous {' or '.join(map(str, dtypes))} "
                             f"{tuple(shape)} on {self.device}, got {t.dtype} {tuple(t.shape)} "
                             f"(strides {t.stride()}) on {t.device}")

    def _no_overlap(self):
        """Parameters and masters are written: no two of them, nor one and a gradient or the
        learning rate, may share memory."""
        spans = []
        for kind, ts in zip(("params", "masters", "grads", "lr"), (*self._bound, [self._lr])):
            spans += [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), kind, i)
                      for i, t in enumerate(ts) if t is not None and t.numel()]
        end, written_end = (0, None, None), (0, None, None)
        for a, b, kind, i in sorted(spans):
            written = kind in ("params", "masters")
            hit = end if written else written_end
            if a < hit[0]:
                raise ValueError(f"AdamW: {kind}[{i}] shares memory with {hit[1]}[{hit[2]}]")
            end = max(end, (b, kind, i), key=lambda e: e[0])
            if written:
                written_end = max(written_end, (b, kind, i), key=lambda e: e[0])

    def step(self):
        """One step on the current stream.  Returns the gradients' norm (a one-element fp32 tensor
        that the next step overwrites), or None where it is not computed."""
        stream = self._stream(self.device.index)
        if stream is None:
            raise ValueError(f"AdamW.step: the tensors are on {self.device}, the current device "
                             f"is {torch.cuda.current_device()}")
        abi.qlora_adamw_step(*self._args, stream)
        return self._norm if self._has_norm else None

    @property
    def lr(self):
        """The learning rate; assign to change it from the next step on (a tensor given as lr is
        changed in place instead)."""
        return self._lr if self._lr is not None else self._config.lr

    @lr.setter
    def lr(self, value):
        if self._lr is not None:
            self._lr.fill_(value)
        else:
            self._config.lr = value

    @property
    def steps(self):
        """Steps taken (synchronises)."""
        return int(self._state.view(torch.int64)[0])

    @property
    def skipped(self):
        """Steps left out for a norm that was not finite (synchronises)."""
        return int(self._state[4])

    def moments(self, dtype=torch.float32):
        """(m, v) flat over the list, as values: the fp32 state itself with 32 bits (for fp32), or
        what the 8-bit codes stand for, in fp32 or bf16."""
        if dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"moments: expected fp32 or bf16, got {dtype}")
        if self.m_scale is None:
            return self.m.to(dtype), self.v.to(dtype)
        return _bind().adamw_moments(self.m, self.v, self.m_scale, self.v_scale,
                                     dtype is torch.float32)

    def state_dict(self):
        """Copies of the moments and the step count."""
        d = {"bits": self._config.bits, "offsets": list(self.offsets),
             "state": self._state.clone(), "m": self.m.clone(), "v": self.v.clone()}
        if self.m_scale is not None:
            d["m_scale"], d["v_scale"] = self.m_scale.clone(), self.v_scale.clone()
        return d

    def load_state_dict(self, d):
        """Takes over what state_dict gave for a list of the same sizes."""
        if d["bits"] != self._config.bits or list(d["offsets"]) != self.offsets or \
                d["m"].shape != self.m.shape:
            raise ValueError("load_state_dict: a state of other tensors or bits")
        for name in ("m", "v") + (("m_scale", "v_scale") if self.m_scale is not None else ()):
            getattr(self, name).copy_(d[name])
        self._state.copy_(d["state"])
