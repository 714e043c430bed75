"""What stands between the linears of a block: residual updates with their RMS norms, and rotary
positions on the heads of q and k.  Tensor-level API over the C ABI, as in ``linear``: torch
tensors in, torch tensors out, on the current stream of the current device; every step of the
computation runs in libqlora_nf4.so.

The buffers are those of the linears: ``linear.grouped_forward``'s packed q/k/v output goes to
``rope`` as it is, a layer's output h is the ``y`` of ``residual_norm_forward``, and its ``n`` the
next layer's X.
"""

from dataclasses import dataclass

import torch

from . import abi
from .linear import _ptr

_BF16, _F32 = torch.bfloat16, torch.float32


def _here(t, name):
    """The current device's index; raises unless the CUDA tensor t is on it."""
    dev = torch.cuda.current_device()
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on the current CUDA device {dev}, got "
                         f"{t.device}")
    return dev


def _stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


def _want(t, dtypes, shape, name, dev):
    if not (t.dtype in dtypes and t.shape == shape and t.is_contiguous()
            and t.is_cuda and t.get_device() == dev):
        raise ValueError(f"{name}: expected contiguous {' or '.join(map(str, dtypes))} "
                         f"{tuple(shape)} on the current CUDA device {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} (strides {t.stride()}) on {t.device}")


_ONE16 = (_BF16,)
_ONE32 = (_F32,)
_EITHER = (_BF16, _F32)


def _norm_types(R, w_pre, w_post, gate, M, D, dev):
    """(types mask, gate kind) of the shared arguments, checked."""
    types = abi.F32_RESIDUAL if R is _F32 else 0
    w = w_pre if w_pre is not None else w_post
    if w is not None:
        if w_pre is not None:
            _want(w_pre, _EITHER, (D,), "w_pre", dev)
        if w_post is not None:
            _want(w_post, (w.dtype,), (D,), "w_post", dev)
            if w_post.dtype not in _EITHER:
                raise ValueError(f"w_post: expected bf16 or fp32, got {w_post.dtype}")
        if w.dtype is _F32:
            types |= abi.F32_WEIGHTS
    kind = abi.GATE_NONE
    if gate is not None:
        if gate.dim() == 1:
            kind = abi.GATE_CHANNEL
            _want(gate, _EITHER, (D,), "gate", dev)
        elif gate.dim() == 2 and gate.shape[1] == 1 and D > 1:
            kind = abi.GATE_TOKEN
            _want(gate, _EITHER, (M, 1), "gate", dev)
        else:
            kind = abi.GATE_FULL
            _want(gate, _EITHER, (M, D), "gate", dev)
        if gate.dtype is _F32:
            types |= abi.F32_GATE
    return types, kind


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
    in place.  Returns (h_out, n or None, rstd_pre or None, rstd_post or None); the fp32 [M] rstd
    are what residual_norm_backward needs (save_rstd=False: not kept)."""
    M, D = h.shape
    dev = _here(h, "h")
    _want(h, _EITHER, (M, D), "h", dev)
    types, kind = _norm_types(h.dtype, w_pre, w_post, gate, M, D, dev)
    if y is None:
        if w_pre is None:
            raise ValueError("residual_norm_forward: nothing to do without y and w_pre")
        if w_post is not None or gate is not None or h_out is not None:
            raise ValueError("residual_norm_forward: w_post, gate and h_out need y")
        if res_scale != 1.0 or branch_scale != 1.0:
            raise ValueError("residual_norm_forward: the scales need y")
    else:
        _want(y, _ONE16, (M, D), "y", dev)
        if h_out is None:
            h_out = torch.empty_like(h)
        else:
            _want(h_out, (h.dtype,), (M, D), "h_out", dev)
    if w_pre is not None:
        if n is None:
            n = torch.empty((M, D), dtype=_BF16, device=h.device)
        else:
            _want(n, _ONE16, (M, D), "n", dev)
        if rstd_pre is not None:
            _want(rstd_pre, _ONE32, (M,), "rstd_pre", dev)
        elif save_rstd:
            rstd_pre = torch.empty(M, dtype=_F32, device=h.device)
    elif n is not None or rstd_pre is not None:
        raise ValueError("residual_norm_forward: n and rstd_pre need w_pre")
    if w_post is not None:
        if rstd_post is not None:
            _want(rstd_post, _ONE32, (M,), "rstd_post", dev)
        elif save_rstd:
            rstd_post = torch.empty(M, dtype=_F32, device=h.device)
    elif rstd_post is not None:
        raise ValueError("residual_norm_forward: rstd_post needs w_post")
    if M:
        abi.qlora_residual_norm_fwd(h.data_ptr(), _ptr(y), _ptr(w_pre), _ptr(w_post), _ptr(gate),
                                    kind, M, D, types, eps, res_scale, branch_scale, weight_offset,
                                    _ptr(h_out), _ptr(n), _ptr(rstd_pre), _ptr(rstd_post),
                                    _stream(dev))
    return (h if y is None else h_out), n, rstd_pre, rstd_post


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
    dh_out; frozen norm weights take need_dw=False."""
    lead = dh_out if dh_out is not None else h_out
    if lead is None:
        raise ValueError("residual_norm_backward: one of dh_out and h_out gives the residual")
    M, D = lead.shape
    R = lead.dtype
    dev = _here(lead, "dh_out" if dh_out is not None else "h_out")
    _want(lead, _EITHER, (M, D), "dh_out" if dh_out is not None else "h_out", dev)
    types, kind = _norm_types(R, w_pre, w_post, gate, M, D, dev)
    if w_pre is not None:
        if dn is None or h_out is None or rstd_pre is None:
            raise ValueError("residual_norm_backward: w_pre needs dn, h_out and rstd_pre")
        _want(dn, _ONE16, (M, D), "dn", dev)
        _want(h_out, (R,), (M, D), "h_out", dev)
        _want(rstd_pre, _ONE32, (M,), "rstd_pre", dev)
    elif dn is not None:
        raise ValueError("residual_norm_backward: dn needs w_pre")
    elif dh_out is None:
        raise ValueError("residual_norm_backward: no gradient comes in")
    branch = (y is not None or gate is not None or w_post is not None) if branch is None else branch
    need_dgate = need_dgate and gate is not None
    if y is not None:
        _want(y, _ONE16, (M, D), "y", dev)
    elif w_post is not None or need_dgate:
        raise ValueError("residual_norm_backward: w_post and the gate's gradient need y")
    if not branch and (gate is not None or w_post is not None or y is not None):
        raise ValueError("residual_norm_backward: y, gate and w_post belong to a branch")
    if w_post is not None:
        if rstd_post is None:
            raise ValueError("residual_norm_backward: w_post needs rstd_post")
        _want(rstd_post, _ONE32, (M,), "rstd_post", dev)
    device = lead.device

    def out(t, dtype, shape, name):
        if t is None:
            return torch.empty(shape, dtype=dtype, device=device)
        _want(t, (dtype,), shape, name, dev)
        return t

    dh = out(dh, R, (M, D), "dh")
    dy = out(dy, _BF16, (M, D), "dy") if branch else None
    dw_pre = out(dw_pre, _F32, (D,), "dw_pre") if need_dw and w_pre is not None else None
    dw_post = out(dw_post, _F32, (D,), "dw_post") if need_dw and w_post is not None else None
    if need_dgate:
        shape = {abi.GATE_CHANNEL: (D,), abi.GATE_TOKEN: (M, 1), abi.GATE_FULL: (M, D)}[kind]
        dgate = out(dgate, gate.dtype if kind == abi.GATE_FULL else _F32, shape, "dgate")
    else:
        dgate = None
    if dw_pre is not None or dw_post is not None or (dgate is not None
                                                     and kind == abi.GATE_CHANNEL):
        if ws is None and M:
            ws = torch.empty(abi.qlora_residual_norm_workspace_bytes(M, D), dtype=torch.uint8,
                             device=device)
    else:
        ws = None
    # An empty tensor has no address: with no tokens only the sums over them are written.
    at = _ptr if M else (lambda t: 16 if t is not None and t.numel() == 0 else _ptr(t))
    abi.qlora_residual_norm_bwd(
        at(dn), at(dh_out), at(h_out) if w_pre is not None else None, at(y),
        at(rstd_pre) if w_pre is not None else None,
        at(rstd_post) if w_post is not None else None, _ptr(w_pre), _ptr(w_post), at(gate), kind,
        M, D, types, res_scale, branch_scale, weight_offset, at(dh), at(dy), _ptr(dw_pre),
        _ptr(dw_post), at(dgate), _ptr(ws), ws.numel() if ws is not None else 0, _stream(dev))
    return dh, dy, dw_pre, dw_post, dgate


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


def _heads(x, n_heads, hd, name, dev):
    """(B, S, heads, strides) of x as [B, S, heads, hd]."""
    if not x.is_cuda or x.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on the current CUDA device {dev}, got "
                         f"{x.device}")
    shape, st = x.shape, x.stride()
    if len(shape) == 2:
        heads = shape[1] // hd if n_heads is None else n_heads
        ok = heads * hd <= shape[1] and (n_heads is not None or shape[1] % hd == 0)
        B, S, strides = 1, shape[0], (0, st[0], hd)
    elif len(shape) == 3:
        heads, ok = shape[1] if n_heads is None else n_heads, shape[2] == hd
        ok = ok and heads <= shape[1]
        B, S, strides = 1, shape[0], (0, st[0], st[1])
    elif len(shape) == 4:
        heads, ok = shape[2] if n_heads is None else n_heads, shape[3] == hd
        ok = ok and heads <= shape[2]
        B, S, strides = shape[0], shape[1], (st[0], st[1], st[2])
    else:
        heads, ok, B, S, strides = 0, False, 0, 0, ()
    if not ok or heads < 1 or (st[-1] != 1 and x.numel()):
        raise ValueError(f"{name}: expected [M, n * {hd}], [M, n, {hd}] or [B, S, n, {hd}] with "
                         f"unit stride in the head and n >= {n_heads or 1}, got {tuple(shape)} "
                         f"(strides {st})")
    return B, S, heads, strides


def _distinct(sizes, strides, hd):
    """Whether no two elements of [B, S, heads, hd] (unit stride in the head) share an address, as
    far as sorted strides tell."""
    reach = hd
    for stride, size in sorted((a, b) for a, b in zip(strides, sizes) if b > 1):
        if stride < reach:
            return False
        reach = stride * (size - 1) + reach
    return True


def rope(x, positions, plan, n_heads=None, k=None, n_heads_k=None, inverse=False, inplace=True,
         out=None, out_k=None):
    """Rotary positions on the heads of x, and of k in the same launch (qlora_rope).

    x, k: bf16 or fp32, [M, n * head_dim] (such as the packed q/k/v output of
    linear.grouped_forward, of which the first n_heads heads are turned), [M, n, head_dim] or
    [B, S, n, head_dim] views of any strides but 1 in the head.  positions: int32 or int64 tensor,
    one a token, or an int: the first token's, counting up along S (M).  inverse: the backward
    pass, on the gradients.  inplace=False (or out / out_k): to a contiguous tensor of the turned
    heads, [M, n_heads * head_dim] or x's shape with n_heads.
    Returns the turned x, or (x, k)."""
    hd = plan.head_dim
    dev = _here(x, "x")
    dtype = x.dtype
    if dtype not in _EITHER:
        raise ValueError(f"x: expected bf16 or fp32, got {dtype}")
    B, S, heads, strides = _heads(x, n_heads, hd, "x", dev)
    tensors = [(x, heads, strides, out, "out")]
    if k is not None:
        if k.dtype is not dtype:
            raise ValueError(f"k: expected {dtype} as x, got {k.dtype}")
        Bk, Sk, heads_k, strides_k = _heads(k, n_heads_k, hd, "k", dev)
        if Bk != B or Sk != S:
            raise ValueError(f"k: expected {B} x {S} tokens as x, got {Bk} x {Sk}")
        tensors.append((k, heads_k, strides_k, out_k, "out_k"))
    elif out_k is not None or n_heads_k is not None:
        raise ValueError("rope: out_k and n_heads_k need k")
    if plan.phase.get_device() != dev:
        raise ValueError(f"plan: expected on the current CUDA device {dev}, got "
                         f"{plan.phase.device}")
    inplace = inplace and out is None and out_k is None
    results, structs = [], []
    for t, n, st, o, name in tensors:
        if inplace:
            o, ost = t, st
        else:
            shape = (S, n * hd) if t.dim() == 2 else (*t.shape[:-2], n, hd)
            if o is None:
                o = torch.empty(shape, dtype=dtype, device=t.device)
                ost = (S * n * hd, n * hd, hd)
            else:
                if o.dtype is not dtype or tuple(o.shape) != shape:
                    raise ValueError(f"{name}: expected {dtype} {shape}, got {o.dtype} "
                                     f"{tuple(o.shape)}")
                _, _, _, ost = _heads(o, n, hd, name, dev)
        if not _distinct((B, S, n), ost, hd):
            raise ValueError(f"rope: elements of {name if not inplace else 'x or k'} share an "
                             f"address (strides {ost})")
        results.append(o)
        structs.append(abi.RopeHeads(t.data_ptr(), o.data_ptr(), *st, *ost, n))
    if isinstance(positions, int):
        pos, pos64, start = None, 0, positions
    else:
        _want(positions, (torch.int32, torch.int64),
              (B, S) if positions.dim() == 2 else (B * S,), "positions", dev)
        pos, pos64, start = positions.data_ptr(), positions.dtype is torch.int64, 0
    if B and S:
        abi.qlora_rope(structs[0], structs[1] if k is not None else None, B, S, hd,
                       plan.rotary_dim, dtype is _F32, pos, pos64, start, plan.phase.data_ptr(),
                       plan.scale, plan.interleaved, inverse, _stream(dev))
    return results[0] if k is None else (results[0], results[1])
