"""The C ABI of the residual norm, rotary positions and AdamW on the CPU: refusals before any device
work, host-only results, struct layouts."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from nf4_base_lora_blockwise_b200 import abi, block, optim
from oracle import block as oracle_block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20   # an aligned, non-null address: never dereferenced on these paths
NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from nf4_base_lora_blockwise_b200 import build
        build.build()
    return abi._lib()


def _fwd(lib, **c):
    a = dict(h=FAKE, y=FAKE, w_pre=FAKE, w_post=FAKE, gate=FAKE, kind=1, M=4, D=64, types=0,
             h_out=FAKE, n=FAKE, r_pre=FAKE, r_post=FAKE)
    assert set(c) <= set(a)
    a.update(c)
    return lib.qlora_residual_norm_fwd(a["h"], a["y"], a["w_pre"], a["w_post"], a["gate"],
                                       a["kind"], a["M"], a["D"], a["types"], 1e-5, 1.0, 1.0, 0.0,
                                       a["h_out"], a["n"], a["r_pre"], a["r_post"], None)


def test_norm_forward_refusals(lib):
    for name in ("h", "h_out", "n", "gate"):
        assert _fwd(lib, **{name: None}) == NULL, name
    assert _fwd(lib, y=None, w_pre=None) == NULL
    for c in ({"M": -1}, {"D": 0}, {"D": 16385}, {"kind": 4}, {"kind": -1}, {"types": 8},
              {"y": None}, {"w_pre": None}, {"w_post": None}, {"kind": 0}):
        assert _fwd(lib, **c) == SHAPE, c
    for name in ("h", "y", "w_pre", "w_post", "gate", "h_out", "n", "r_pre", "r_post"):
        assert _fwd(lib, **{name: FAKE + 8}) == ALIGN, name
    assert _fwd(lib, M=0) == 0


def _bwd(lib, **c):
    a = dict(dn=FAKE, dh_out=FAKE, h_out=FAKE, y=FAKE, r_pre=FAKE, r_post=FAKE, w_pre=FAKE,
             w_post=FAKE, gate=FAKE, kind=1, M=4, D=64, types=0, dh=FAKE, dy=FAKE, dw_pre=FAKE,
             dw_post=FAKE, dgate=FAKE, ws=FAKE, ws_bytes=1 << 30)
    assert set(c) <= set(a)
    a.update(c)
    return lib.qlora_residual_norm_bwd(
        a["dn"], a["dh_out"], a["h_out"], a["y"], a["r_pre"], a["r_post"], a["w_pre"], a["w_post"],
        a["gate"], a["kind"], a["M"], a["D"], a["types"], 1.0, 1.0, 0.0, a["dh"], a["dy"],
        a["dw_pre"], a["dw_post"], a["dgate"], a["ws"], a["ws_bytes"], None)


def test_norm_backward_refusals(lib):
    for name in ("dn", "h_out", "y", "r_pre", "r_post", "w_pre", "w_post", "gate", "dh", "dy"):
        assert _bwd(lib, **{name: None}) == NULL, name
    assert _bwd(lib, dn=None, dh_out=None, w_pre=None, dw_pre=None) == NULL
    for c in ({"M": -1}, {"D": 0}, {"D": 16385}, {"kind": 4}, {"kind": 0}, {"types": 16}):
        assert _bwd(lib, **c) == SHAPE, c
    for name in ("dn", "dh_out", "h_out", "y", "r_pre", "dh", "dy", "dw_pre", "dgate", "ws"):
        assert _bwd(lib, **{name: FAKE + 4}) == ALIGN, name
    assert _bwd(lib, ws=None) == WORKSPACE
    assert _bwd(lib, ws_bytes=lib.qlora_residual_norm_workspace_bytes(4, 64) - 1) == WORKSPACE
    assert lib.qlora_residual_norm_workspace_bytes(0, 64) == 0
    assert lib.qlora_residual_norm_workspace_bytes(4, 16385) == 0


def _heads(x=FAKE, out=FAKE, st=(0, 512, 64), ost=(0, 512, 64), heads=8):
    return abi.RopeHeads(x, out, *st, *ost, heads)


def _rope(lib, q=None, k=None, B=1, S=4, hd=64, rd=64, pos=FAKE, pos64=0, phase=FAKE):
    q = _heads() if q is None else q
    return lib.qlora_rope(ctypes.byref(q), ctypes.byref(k) if k is not None else None, B, S, hd,
                          rd, 0, pos, pos64, 0, phase, 1.0, 0, 0, None)


def test_rope_refusals(lib):
    assert lib.qlora_rope(None, None, 1, 4, 64, 64, 0, FAKE, 0, 0, FAKE, 1.0, 0, 0, None) == NULL
    assert _rope(lib, phase=None) == NULL
    assert _rope(lib, q=_heads(x=None)) == NULL and _rope(lib, q=_heads(out=None)) == NULL
    for c in ({"B": -1}, {"S": -1}, {"B": 1 << 20, "S": 1 << 20}, {"hd": 2050, "rd": 64},
              {"rd": 63}, {"rd": 66}, {"rd": 0}):
        assert _rope(lib, **c) == SHAPE, c
    assert _rope(lib, q=_heads(heads=0)) == SHAPE and _rope(lib, q=_heads(heads=4097)) == SHAPE
    assert _rope(lib, q=_heads(heads=4000), k=_heads(x=2 * FAKE, out=2 * FAKE, heads=97)) == SHAPE
    assert _rope(lib, q=_heads(st=(0, -512, 64))) == SHAPE
    assert _rope(lib, q=_heads(ost=(0, 1024, 64))) == SHAPE          # in place, other strides
    assert _rope(lib, k=_heads(x=2 * FAKE, out=4 * FAKE)) == SHAPE   # one in place, one not
    assert _rope(lib, q=_heads(x=FAKE + 1, out=FAKE + 1)) == ALIGN
    assert _rope(lib, pos=FAKE + 4, pos64=1) == ALIGN and _rope(lib, pos=FAKE + 2) == ALIGN
    assert _rope(lib, S=0) == 0


def test_rope_phase_refusals(lib):
    ph, sc = (ctypes.c_int64 * 64)(), ctypes.c_float()
    call = lambda rd=64, base=1e4, kind=0, factor=2.0, low=1.0, high=4.0, n=4096.0, p=ph: (  # noqa: E731
        lib.qlora_rope_phase(rd, base, kind, factor, low, high, n, p, ctypes.byref(sc)))
    assert call() == 0 and call(kind=4) == 0
    assert call(p=None) == NULL
    inf, nan = float("inf"), float("nan")
    for c in ({"rd": 0}, {"rd": 3}, {"rd": 2050}, {"base": 1.0}, {"base": nan}, {"base": inf},
              {"kind": 5}, {"kind": -1}, {"kind": 1, "factor": 0.5}, {"kind": 1, "factor": nan},
              {"kind": 2, "rd": 2}, {"kind": 3, "low": 4.0}, {"kind": 3, "low": 0.0},
              {"kind": 4, "high": inf}, {"kind": 4, "n": 0.0}):
        assert call(**c) == SHAPE, c


@pytest.mark.parametrize("rd", [2, 6, 64, 128, 2048])
@pytest.mark.parametrize("scaling", [
    None, {"kind": "linear", "factor": 4.0}, {"kind": "base", "factor": 8.0},
    {"kind": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "original": 8192},
    {"kind": "ramp", "factor": 16.0, "slow": 1.0, "fast": 32.0, "original": 4096}])
def test_rope_phase_matches_oracle(lib, rd, scaling):
    """Phases are turns per position to 2^-64, from two derivations in extended precision: 2^-62
    holds both roundings of a value below 1/6 with a few operations on it.  The ramp's blend is a
    quotient in 64 bits (relative 2^-52 of a frequency)."""
    if scaling and scaling["kind"] == "base" and rd == 2:
        pytest.skip("refused: one pair is the fastest and the slowest")
    plan = block.rope_plan(2048, rotary_dim=rd, base=500000.0, scaling=scaling, device="cpu")
    f, scale = oracle_block.frequencies(rd, 500000.0, scaling)
    want = f / np.longdouble("6.283185307179586476925286766559")
    got = np.array([int(p) for p in plan.phase], dtype=np.longdouble) / np.longdouble(2) ** 64
    tol = 2.0 ** -62 if not scaling or scaling["kind"] != "ramp" else 2.0 ** -53
    assert np.max(np.abs(got - want)) <= tol
    assert abs(plan.scale - scale) <= 2.0 ** -24 * scale


def test_rope_plan_refusals():
    for kw in ({"rotary_dim": 130}, {"rotary_dim": 0}, {"scaling": {"kind": "other"}},
               {"scaling": {"kind": "linear"}}, {"scaling": {"factor": 2.0}},
               {"scaling": {"kind": "linear", "factor": 2.0, "low": 1.0}}):
        with pytest.raises(ValueError):
            block.rope_plan(128, device="cpu", **kw)
    with pytest.raises(abi.QLoraError):
        block.rope_plan(128, rotary_dim=3, device="cpu")


def _adam(lib, t=None, count=1, m=FAKE, ms=FAKE, state=FAKE, ws=FAKE, ws_bytes=1 << 20, **c):
    t = abi.AdamWTensor(FAKE, FAKE, FAKE, 100, 1.0, 0.0, 0, 1) if t is None else t
    f = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, max_norm=1.0, bits=8,
             lr_device=None, seed=0, check_finite=0)
    f.update(c)
    cfg = abi.AdamWConfig(**f)
    return lib.qlora_adamw_step(ctypes.byref(t), count, ctypes.byref(cfg), m, FAKE, ms, ms, state,
                                ws, ws_bytes, None)


def test_adamw_refusals(lib):
    T = abi.AdamWTensor
    assert _adam(lib, m=None) == NULL and _adam(lib, state=None) == NULL
    assert _adam(lib, ms=None) == NULL                      # 8 bits need scales
    assert _adam(lib, bits=32) == NULL                      # 32 bits have none
    nan, inf = float("nan"), float("inf")
    for c in ({"bits": 16}, {"lr": nan}, {"beta1": 1.0}, {"beta2": -0.1}, {"eps": -1e-8},
              {"eps": inf}, {"max_norm": -1.0}, {"max_norm": nan}, {"grad_scale": inf},
              {"count": 0}):
        assert _adam(lib, **c) == SHAPE, c
    assert _adam(lib, t=T(FAKE, FAKE, FAKE, -1, 1, 0, 0, 0)) == SHAPE
    assert _adam(lib, t=T(FAKE, FAKE, FAKE, 8, 1, 0, 1, 0)) == SHAPE   # fp32 with a master
    assert _adam(lib, t=T(None, None, FAKE, 8, 1, 0, 0, 0)) == NULL
    assert _adam(lib, t=T(FAKE, None, None, 8, 1, 0, 0, 0)) == NULL
    for t in (T(FAKE + 2, None, FAKE, 8, 1, 0, 0, 0), T(FAKE, FAKE + 4, FAKE, 8, 1, 0, 0, 0),
              T(FAKE, None, FAKE + 8, 8, 1, 0, 0, 0)):
        assert _adam(lib, t=t) == ALIGN
    assert _adam(lib, m=FAKE + 8) == ALIGN and _adam(lib, state=FAKE + 8) == ALIGN
    assert _adam(lib, lr_device=FAKE + 2) == ALIGN
    assert _adam(lib, ws=None) == WORKSPACE and _adam(lib, ws_bytes=8) == WORKSPACE
    ts = (T * 3)(T(FAKE, None, FAKE, 1, 1, 0, 0, 0), T(FAKE, None, FAKE, 0, 1, 0, 0, 0),
                 T(FAKE, None, FAKE, 257, 1, 0, 0, 0))
    assert lib.qlora_adamw_blocks(ts, 3) == 3
    # One double for each of up to 8 CTAs an SM (148) that sum a launch of up to 512 tensors.
    assert lib.qlora_adamw_workspace_bytes(0) == 0
    assert lib.qlora_adamw_workspace_bytes(1) >= 148 * 8 * 8
    assert lib.qlora_adamw_workspace_bytes(513) >= 2 * 148 * 8 * 8
    assert lib.qlora_adamw_moments(FAKE, FAKE, FAKE, None, 1, 0, FAKE, FAKE, None) == NULL
    assert lib.qlora_adamw_moments(FAKE, FAKE, FAKE, FAKE, -1, 0, FAKE, FAKE, None) == SHAPE
    assert lib.qlora_adamw_moments(FAKE + 8, FAKE, FAKE, FAKE, 1, 0, FAKE, FAKE, None) == ALIGN


def test_adamw_lists_refused_before_any_device():
    p, g = torch.zeros(8), torch.zeros(8)
    for args in (([], []), ([p], []), ([p], [g], [])):
        with pytest.raises(ValueError):
            optim.AdamW(*args)
    with pytest.raises(ValueError, match="CUDA|on cpu"):
        optim.AdamW([p], [g])
    with pytest.raises(ValueError):
        optim.AdamW([p], [g], bits=16)


def test_struct_layouts(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    src = tmp_path / "sizes.c"
    src.write_text('#include "qlora_nf4.h"\n#include <stdio.h>\nint main(void) {\n'
                   '  printf("%zu %zu %zu %zu %zu\\n", sizeof(qlora_rope_heads),\n'
                   '         sizeof(qlora_adamw_tensor), sizeof(qlora_adamw_config),\n'
                   '         offsetof(qlora_adamw_config, seed), offsetof(qlora_rope_heads, heads));\n'
                   '  return 0;\n}\n')
    exe = tmp_path / "sizes"
    subprocess.run([gcc, "-std=c11", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [ctypes.sizeof(abi.RopeHeads), ctypes.sizeof(abi.AdamWTensor),
                   ctypes.sizeof(abi.AdamWConfig), abi.AdamWConfig.seed.offset,
                   abi.RopeHeads.heads.offset]


def test_binding_raises():
    """The torch binding's errors reach Python as exceptions (it shares torch's C++ runtime)."""
    b = block._bind()
    for f in (b.residual_norm_forward, b.residual_norm_backward, b.rope, b.adamw_moments):
        with pytest.raises(TypeError, match="arguments, got 1"):
            f(None)
    with pytest.raises(TypeError):
        b.current_stream("x")


def test_divisions_of_rope_are_exact(tmp_path):
    """csrc/divide.cuh, compiled for the host: for every number of items that a head can have, below
    and at every multiple, as far as the 4096 heads of a call reach or the heads of one launch do.
    Past these the quotient is wrong for some divisor (2046: from head 1028 on)."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src = tmp_path / "divide.cpp"
    src.write_text('#include "divide.cuh"\n#include <cstdio>\n'
                   'int main() {\n'
                   '  unsigned long long wrong = 0, split = 0;\n'
                   '  for (uint32_t d = 1; d <= 2048; ++d) {\n'
                   '    const qlora::Divide v = qlora::divide_by(d);\n'
                   '    const uint32_t most = qlora::exact_heads(d);\n'
                   '    const uint32_t heads = most < 4096 ? most : 4096;\n'
                   '    split += most < 4096;\n'
                   '    for (uint32_t h = 0; h < heads; ++h)\n'
                   '      wrong += qlora::quotient(h * d, v) != h || qlora::quotient(h * d + d - 1, v) != h;\n'
                   '  }\n'
                   '  const qlora::Divide v = qlora::divide_by(2046);\n'
                   '  std::printf("%llu %llu %u %d", wrong, split, qlora::quotient(2105333, v), qlora::exact_heads(0));\n'
                   '}\n')
    exe = tmp_path / "divide"
    inc = os.path.join(ROOT, "nf4_base_lora_blockwise_b200", "csrc")
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-I" + inc, str(src), "-o",
                    str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    # 4096 d^2 > 2^32 for d > 1024.
    assert got == [0, 2048 - 1024, 2105333 // 2046 + 1, 2 ** 31 - 1]


def test_norm_refuses_numbers_out_of_range(lib):
    """eps is not negative, the scales and the offset are finite (as fp32 numbers)."""
    fwd = lambda eps, res=1.0, br=1.0, o=0.0, M=4: lib.qlora_residual_norm_fwd(  # noqa: E731
        FAKE, FAKE, FAKE, None, None, 0, M, 64, 0, eps, res, br, o, FAKE, FAKE, None, None, None)
    bwd = lambda res, br, o: lib.qlora_residual_norm_bwd(  # noqa: E731
        FAKE, FAKE, FAKE, None, FAKE, None, FAKE, None, None, 0, 4, 64, 0, res, br, o, FAKE, FAKE,
        None, None, None, None, 0, None)
    inf, nan = float("inf"), float("nan")
    assert fwd(0.0, M=0) == 0
    for eps in (-1e-5, nan, inf, -inf, 1e39):
        assert fwd(eps) == fwd(eps, M=0) == SHAPE, eps
    for x in (nan, inf, -inf):
        for at in range(3):
            args = [1.0, 1.0, 0.0]
            args[at] = x
            assert fwd(1e-5, *args) == SHAPE and bwd(*args) == SHAPE, args


def test_adamw_refuses_rates_that_are_not_finite(lib):
    T = abi.AdamWTensor
    for x in (float("nan"), float("inf"), -float("inf")):
        for n in (8, 0):
            assert _adam(lib, t=T(FAKE, FAKE, FAKE, n, x, 0, 0, 0)) == SHAPE
            assert _adam(lib, t=T(FAKE, FAKE, FAKE, n, 1, x, 0, 0)) == SHAPE
