"""What stands between the linears of a block: residual updates with their RMS norms, and rotary
positions on the heads of q and k.  Tensor-level API over the C ABI, as in ``linear``: torch
tensors in, torch tensors out, on the current stream of the current device; every step of the
computation runs in libqlora_nf4.so, and the checks of the arguments in _torch_bind.so.

The buffers are those of the linears: ``linear.grouped_forward``'s packed q/k/v output goes to
``rope`` as it is, a layer's output h is the ``y`` of ``residual_norm_forward``, and its ``n`` the
next layer's X.
"""

from dataclasses import dataclass

import torch

from . import abi

_BIND = None


def _bind():
    """The binding's module, loaded on first use; raises if it has not been built."""
    global _BIND
    if _BIND is None:
        abi.loaded_path()
        try:
            from . import _torch_bind
        except ImportError as e:
            raise RuntimeError("_torch_bind.so is missing: build it with "
                               "`python -m nf4_base_lora_blockwise_b200.build`") from e
        _torch_bind.set_error(abi.QLoraError)
        _BIND = _torch_bind
    return _BIND


def residual_norm_forward(h, y=None, w_pre=None, w_post=None, gate=None, eps=1e-5, res_scale=1.0,
                          branch_scale=1.0, weight_offset=0.0, h_out=None, n=None, rstd_pre=None,
                          rstd_post=None, save_rstd=True):
    """The residual update of a block with the norms before and after it
    (qlora_residual_norm_fwd)::

        a     = rms(y) * (w_post + weight_offset)          (a = y without w_post)
        h_out = res_scale * h + branch_scale * gate * a
        n     = rms(h_out) * (w_pre + weight_offset)       (bf16; w_pre: the next block's norm)

    with rms(x) = x / sqrt(mean(x^2) + eps).  h [M, D] bf16 or fp32, y [M, D] bf16, weights [D]
    bf16 or fp32, gate None, [D], [M, 1] or [M, D] bf16 or fp32.  Without y only the norm of h is
    taken (h_out is h); without w_pre only the update.  h_out may be h: the stream is then updated
    in place; n may be y.  Other given outputs share no memory with the inputs or each other
    (ValueError).  Returns (h_out, n or None, rstd_pre or None, rstd_post or None); the fp32 [M] rstd
    are what residual_norm_backward needs (save_rstd=False: not kept)."""
    return (_BIND or _bind()).residual_norm_forward(
        h, y, w_pre, w_post, gate, eps, res_scale, branch_scale, weight_offset, h_out, n, rstd_pre,
        rstd_post, save_rstd)


def residual_norm_backward(dn, dh_out, h_out, y=None, rstd_pre=None, rstd_post=None, w_pre=None,
                           w_post=None, gate=None, res_scale=1.0, branch_scale=1.0,
                           weight_offset=0.0, need_dw=True, need_dgate=True, branch=None, dh=None,
                           dy=None, dw_pre=None, dw_post=None, dgate=None, ws=None):
    """Backward of residual_norm_forward (qlora_residual_norm_bwd).  dn [M, D] bf16: gradient of n
    (with w_pre); dh_out [M, D] in the residual's type: gradient of h_out from the blocks after it
    (None: zero); h_out, rstd_pre, rstd_post: the forward's.  y may be None where neither w_post
    nor a gate's gradient needs it; `branch` then says whether the forward had one (default: y, a
    gate or w_post was given).
    Returns (dh [M, D] in the residual's type, dy [M, D] bf16 or None, dw_pre and dw_post fp32 [D]
    or None, dgate or None: fp32 [D], fp32 [M, 1], or [M, D] in the gate's type).  dh may be
    dh_out, dy may be y or dn, else given outputs share no memory with the inputs or each other
    (ValueError); frozen norm weights take need_dw=False."""
    return (_BIND or _bind()).residual_norm_backward(
        dn, dh_out, h_out, y, rstd_pre, rstd_post, w_pre, w_post, gate, res_scale, branch_scale,
        weight_offset, need_dw, need_dgate, branch, dh, dy, dw_pre, dw_post, dgate, ws)


@dataclass
class RopePlan:
    """Rotary positions of one head layout (device tensor owned by this object)."""
    phase: torch.Tensor      # [rotary_dim / 2] int64: turns per position times 2^64
    scale: float             # on the rotated elements (1 but for "ramp")
    head_dim: int
    rotary_dim: int
    interleaved: bool = False


_ROPE_KINDS = {"linear": (1, ()), "base": (2, ()), "bands": (3, ("low", "high", "original")),
               "ramp": (4, ("slow", "fast", "original"))}


def rope_plan(head_dim, rotary_dim=None, base=10000.0, scaling=None, interleaved=False, scale=None,
              device=None):
    """Plan of rotary positions (qlora_rope_phase): pair i turns by position x f_i, with
    f_i = base^(-2i / rotary_dim) (default: the whole head), scaled for contexts longer than the
    trained one by ``scaling``::

        None                                              not scaled
        {"kind": "linear", "factor"}                      f / factor
        {"kind": "base", "factor"}                        base grown until the slowest pair is f / factor
        {"kind": "bands", "factor", "low", "high", "original"}
                 pairs under `low` turns in `original` tokens slowed by factor, over `high` kept,
                 a blend in the frequency between
        {"kind": "ramp", "factor", "slow", "fast", "original"}
                 the same with a blend in the pair's index, and values scaled by
                 0.1 ln(factor) + 1

    interleaved: pairs (2i, 2i + 1) instead of (i, i + rotary_dim / 2).  scale: factor on the
    rotated elements in place of the kind's own."""
    rotary_dim = head_dim if rotary_dim is None else rotary_dim
    kind, args = 0, {"factor": 1.0}
    if scaling is not None:
        args = dict(scaling)
        name = args.pop("kind", None)
        if name not in _ROPE_KINDS:
            raise ValueError(f"rope_plan: scaling kind {name!r} is none of {sorted(_ROPE_KINDS)}")
        kind, needs = _ROPE_KINDS[name]
        if set(args) != {"factor", *needs}:
            raise ValueError(f"rope_plan: scaling {name!r} takes {('factor', *needs)}, got "
                             f"{tuple(sorted(args))}")
    if not 2 <= rotary_dim <= head_dim:
        raise ValueError(f"rope_plan: rotary_dim {rotary_dim} of a head of {head_dim}")
    phase, own = abi.qlora_rope_phase(rotary_dim, base, kind, args["factor"],
                                      args.get("low", args.get("slow", 1.0)),
                                      args.get("high", args.get("fast", 2.0)),
                                      args.get("original", 1.0))
    phase = torch.tensor(list(phase), dtype=torch.int64)
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return RopePlan(phase.to(device), own if scale is None else float(scale), head_dim, rotary_dim,
                    bool(interleaved))


def rope(x, positions, plan, n_heads=None, k=None, n_heads_k=None, inverse=False, inplace=True,
         out=None, out_k=None):
    """Rotary positions on the heads of x, and of k in the same launch (qlora_rope).

    x, k: bf16 or fp32, [M, n * head_dim] (such as the packed q/k/v output of
    linear.grouped_forward, of which the first n_heads heads are turned), [M, n, head_dim] or
    [B, S, n, head_dim] views of any strides but 1 in the head.  positions: int32 or int64 tensor,
    one a token, or an int: the first token's, counting up along S (M).  inverse: the backward
    pass, on the gradients.  inplace=False (or out / out_k): to a contiguous tensor of the turned
    heads, [M, n_heads * head_dim] or x's shape with n_heads.  What is written shares no element
    with another argument (ValueError): x and k may be parts of one packed row, not overlap.
    Returns the turned x, or (x, k)."""
    return (_BIND or _bind()).rope(
        x, positions, plan.phase, plan.scale, plan.head_dim, plan.rotary_dim, plan.interleaved,
        n_heads, k, n_heads_k, inverse, inplace, out, out_k)
