"""GPU parity of the residual norm (qlora_residual_norm_fwd / _bwd) with the fp64 oracle.

Tolerances, elementwise, with u = 2^-24: an output is rounded once to its type (half a step: 2^-8
of the value for bf16, 2^-24 for fp32), and the fp32 arithmetic before it adds at most C u of the
magnitude that the oracle gives (the sum of the absolute values added).  A row's sum of squares or
products passes at most 16 sequential additions in a thread, 5 + 32 over the row's threads, and
mean, rsqrt (2 ulp) and scaling about 10 more: 64 u for a sum, 80 u for one norm, so C = 128
forward.  Backward, two nested sums and the products around them: C = 256.  Column sums over M
tokens add at most M sequential additions: C = 256 + M.  n is checked against the norm of h' as the
library stored it, which is its definition.
"""

import ctypes
import itertools
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from nf4_base_lora_blockwise_b200 import abi, block
from oracle import block as oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _close(got, want, mag, c, name):
    half = 2.0 ** -8 if got.dtype is BF16 else U
    err = np.abs(_np(got) - want)
    tol = half * np.abs(want) * (1 + 2.0 ** -8) + c * U * mag + 1e-37
    assert np.all(err <= tol), (name, float(np.max(err / tol)), np.argwhere(err > tol)[:4].tolist())


def _inputs(M, D, R, W, post, gate, pre, seed, gate_type=None, y=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g) * std  # noqa: E731
    G = gate_type or W
    d = {"h": rnd(M, D).to(R), "y": rnd(M, D, std=0.7).to(BF16) if y else None,
         "w_pre": rnd(D).to(W) if pre else None, "w_post": rnd(D).to(W) if post else None,
         "gate": {"none": None, "channel": rnd(D).to(G), "token": rnd(M, 1).to(G),
                  "full": rnd(M, D).to(G)}[gate],
         "dn": rnd(M, D).to(BF16) if pre else None, "dh": rnd(M, D).to(R)}
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def _check(M, D, R=BF16, W=BF16, post=True, gate="channel", pre=True, res=0.5, br=1.25, o=1.0,
           seed=0, gate_type=None, eps=1e-5, change=None):
    i = _inputs(M, D, R, W, post, gate, pre, seed, gate_type)
    if change:
        change(i)
    h, n, r_pre, r_post = block.residual_norm_forward(
        i["h"], i["y"], i["w_pre"], i["w_post"], i["gate"], eps=eps, res_scale=res,
        branch_scale=br, weight_offset=o)
    want, mag, want_r = oracle.update(_np(i["h"]), _np(i["y"]), _np(i["w_post"]), _np(i["gate"]),
                                      eps, res, br, o)
    assert h.dtype is R and h.shape == (M, D)
    _close(h, want, mag, 128, "h")
    if post:
        _close(r_post, want_r, want_r, 128, "rstd_post")
    else:
        assert r_post is None
    if pre:
        want, want_r = oracle.norm(_np(h), _np(i["w_pre"]), eps, o)
        assert n.dtype is BF16
        _close(n, want, np.abs(want), 128, "n")
        _close(r_pre, want_r, want_r, 128, "rstd_pre")
    else:
        assert n is None and r_pre is None
    got = dict(zip(("dh", "dy", "dw_pre", "dw_post", "dgate"), block.residual_norm_backward(
        i["dn"], i["dh"], h, i["y"], r_pre, r_post, i["w_pre"], i["w_post"], i["gate"],
        res_scale=res, branch_scale=br, weight_offset=o)))
    ref = oracle.backward(_np(i["dn"]), _np(i["dh"]), _np(h), _np(i["y"]), _np(r_pre),
                          _np(r_post), _np(i["w_pre"]), _np(i["w_post"]), _np(i["gate"]), res, br,
                          o)
    for name, t in got.items():
        if name not in ref:
            assert t is None, name
            continue
        want, mag = ref[name]
        c = 256
        if name.startswith("dw"):
            c += M
        if name == "dgate" and gate == "channel":
            want, mag, c = want.sum(0), mag.sum(0), c + M
        if name == "dgate" and gate == "token":
            want, mag = want.sum(1, keepdims=True), mag.sum(1, keepdims=True)
        assert t.shape == want.shape, name
        _close(t, want, mag, c, name)
    return i, (h, n, r_pre, r_post), got


# Widths on both sides of every change of layout: one element; slices of a warp; whole warps; even
# and odd rows; the widest.
@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 24, 31, 64, 127, 128, 250, 256, 257, 264, 511, 1000,
                               2040, 2048, 2050, 2051, 2056, 4096, 4104, 8183, 8185, 8186, 8192,
                               8200, 12243, 16376, 16373, 16374, 16384])
def test_widths(D):
    _check(5, D, seed=D)
    _check(3, D, R=F32, W=F32, gate="full", seed=D + 1, gate_type=BF16)


@pytest.mark.parametrize("M", [1, 2, 7, 33, 148, 149, 600, 1185])
def test_token_counts(M):
    for D in (72, 1024, 37, 333, 1030):
        _check(M, D, seed=M)


@pytest.mark.parametrize("M,D,R", [(901, 8192, BF16), (1900, 4096, BF16), (3601, 2040, F32)])
def test_more_rows_than_are_on_their_way(M, D, R):
    i, (h, _, r, _), got = _check(M, D, R=R, post=False, gate="none", seed=M)
    args = dict(rstd_pre=r, w_pre=i["w_pre"], res_scale=0.5, branch_scale=1.25, weight_offset=1.0)
    frozen = block.residual_norm_backward(i["dn"], i["dh"], h, need_dw=False, branch=True, **args)
    assert torch.equal(frozen[0], got["dh"]) and torch.equal(frozen[1], got["dy"])
    # Only as many rows as the others see of theirs: bits do not depend on the batch.
    few = block.residual_norm_backward(i["dn"][:9], i["dh"][:9], h[:9], need_dw=False, branch=True,
                                       **{**args, "rstd_pre": r[:9]})
    assert torch.equal(few[0], got["dh"][:9]) and torch.equal(few[1], got["dy"][:9])


@pytest.mark.parametrize("post,gate,pre", list(itertools.product(
    (True, False), ("none", "channel", "token", "full"), (True, False))))
@pytest.mark.parametrize("R,W,G", [(BF16, BF16, F32), (F32, BF16, BF16), (BF16, F32, BF16),
                                   (F32, F32, F32)])
def test_forms_and_types(post, gate, pre, R, W, G):
    _check(9, 136, R=R, W=W, post=post, gate=gate, pre=pre, gate_type=G)
    _check(4, 35, R=R, W=W, post=post, gate=gate, pre=pre, gate_type=G, o=0.0)


def test_norm_alone():
    for M, D in ((6, 4096), (300, 128), (4, 33)):
        i = _inputs(M, D, BF16, BF16, False, "none", True, 5, y=False)
        h, n, r, none = block.residual_norm_forward(i["h"], w_pre=i["w_pre"])
        assert h is i["h"] and none is None
        want, want_r = oracle.norm(_np(h), _np(i["w_pre"]), 1e-5, 0.0)
        _close(n, want, np.abs(want), 128, "n")
        dh, dy, dw, a, b = block.residual_norm_backward(i["dn"], None, h, rstd_pre=r,
                                                        w_pre=i["w_pre"])
        assert dy is None and a is None and b is None
        ref = oracle.backward(_np(i["dn"]), None, _np(h), None, _np(r), None, _np(i["w_pre"]), None,
                              None, 1.0, 1.0, 0.0)
        _close(dh, *ref["dh"], 256, "dh")
        _close(dw, *ref["dw_pre"], 256 + M, "dw_pre")


def test_rows_of_zeros_and_extremes():
    """A row of zeros has n = 0 and finite gradients (eps holds the root); a row with an infinity or
    NaN touches no other row; large and tiny rows keep their precision."""
    def change(i):
        i["h"][0] = 0
        i["y"][0] = 0
        i["h"][1] *= 2.0 ** 40
        i["y"][2] *= 2.0 ** -30
    _check(6, 264, R=F32, change=change, eps=1e-6)
    i = _inputs(6, 264, BF16, BF16, True, "channel", True, 9)
    clean = block.residual_norm_forward(i["h"], i["y"], i["w_pre"], i["w_post"], i["gate"])
    i["h"][2, 5], i["y"][4, 200] = float("inf"), float("nan")
    dirty = block.residual_norm_forward(i["h"], i["y"], i["w_pre"], i["w_post"], i["gate"])
    keep = torch.tensor([0, 1, 3, 5], device="cuda")
    for a, b in zip(clean, dirty):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(dirty[1][4].float()).all()


def test_in_place_and_given_outputs():
    i = _inputs(70, 520, BF16, BF16, True, "channel", True, 3)
    want = block.residual_norm_forward(i["h"], i["y"], i["w_pre"], i["w_post"], i["gate"])
    back = block.residual_norm_backward(i["dn"], i["dh"], want[0], i["y"], want[2], want[3],
                                        i["w_pre"], i["w_post"], i["gate"])
    h, y = i["h"].clone(), i["y"].clone()
    got = block.residual_norm_forward(h, y, i["w_pre"], i["w_post"], i["gate"], h_out=h, n=y)
    assert got[0] is h and got[1] is y
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    dh, y = i["dh"].clone(), i["y"].clone()
    outs = block.residual_norm_backward(i["dn"], dh, want[0], y, want[2], want[3], i["w_pre"],
                                        i["w_post"], i["gate"], dh=dh, dy=y)
    assert outs[0] is dh and outs[1] is y
    for a, b in zip(back, outs):
        assert torch.equal(a, b)
    frozen = block.residual_norm_backward(i["dn"], i["dh"], want[0], i["y"], want[2], want[3],
                                          i["w_pre"], i["w_post"], i["gate"], need_dw=False,
                                          need_dgate=False)
    assert torch.equal(frozen[0], back[0]) and torch.equal(frozen[1], back[1])
    assert frozen[2] is frozen[3] is frozen[4] is None
    gone = block.residual_norm_forward(i["h"], i["y"], i["w_pre"], i["w_post"], i["gate"],
                                       save_rstd=False)
    assert gone[2] is gone[3] is None and torch.equal(gone[1], want[1])
    # A plain residual has dy = branch_scale dh_out without reading y.
    dh, dy, *_ = block.residual_norm_backward(None, i["dh"], None, branch=True, branch_scale=0.5)
    assert torch.equal(dh, i["dh"]) and torch.equal(dy, (i["dh"].float() * 0.5).to(BF16))


def test_no_tokens():
    i = _inputs(0, 64, BF16, BF16, True, "channel", True, 3)
    h, n, a, b = block.residual_norm_forward(i["h"], i["y"], i["w_pre"], i["w_post"], i["gate"])
    assert h.shape == n.shape == (0, 64)
    outs = block.residual_norm_backward(i["dn"], i["dh"], h, i["y"], a, b, i["w_pre"],
                                        i["w_post"], i["gate"])
    assert outs[0].shape == (0, 64) and all(torch.count_nonzero(t) == 0 for t in outs[2:])


def test_same_bits_again_and_in_a_graph():
    """Column sums are added in a fixed order; replays see new inputs."""
    i = _inputs(1000, 512, BF16, BF16, True, "channel", True, 4)

    def both():
        f = block.residual_norm_forward(i["h"], i["y"], i["w_pre"], i["w_post"], i["gate"])
        return (*f, *block.residual_norm_backward(i["dn"], i["dh"], f[0], i["y"], f[2], f[3],
                                                  i["w_pre"], i["w_post"], i["gate"]))
    first = both()
    for a, b in zip(first, both()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        outs = both()
    for t in (i["h"], i["y"], i["dn"]):
        t.copy_(t.flip(0))
    want = both()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert torch.equal(a, b)
    assert not torch.equal(first[1], outs[1])


def test_long_rows_offset_past_32_bits():
    """Row offsets are 64-bit: 2^31 elements and a few rows (fp32 residual of 8.6 GB)."""
    M, D = 131074, 16384
    h = torch.zeros(M, D, dtype=BF16, device="cuda")
    h[-2:] = torch.randn(2, D, device="cuda").to(BF16)
    w = torch.ones(D, dtype=BF16, device="cuda")
    _, n, r, _ = block.residual_norm_forward(h, w_pre=w)
    want, want_r = oracle.norm(_np(h[-2:]), _np(w), 1e-5, 0.0)
    _close(n[-2:], want, np.abs(want), 128, "n")
    assert torch.count_nonzero(n[:-2]) == 0
    del n
    dn = h
    dh, *_ = block.residual_norm_backward(dn, None, h, rstd_pre=r, w_pre=w, need_dw=False)
    ref = oracle.backward(_np(dn[-2:]), None, _np(h[-2:]), None, _np(r[-2:]), None, _np(w), None,
                          None, 1.0, 1.0, 0.0)
    _close(dh[-2:], *ref["dh"], 256, "dh")


def test_refusals():
    i = _inputs(8, 64, BF16, BF16, True, "channel", True, 1)
    f = lambda **kw: block.residual_norm_forward(**{**dict(  # noqa: E731
        h=i["h"], y=i["y"], w_pre=i["w_pre"], w_post=i["w_post"], gate=i["gate"]), **kw})
    bad = [dict(h=i["h"].half()), dict(h=i["h"].cpu()), dict(y=i["y"].float()),
           dict(y=i["y"][:4]), dict(y=torch.empty(64, 8, dtype=BF16, device="cuda").t()),
           dict(w_pre=i["w_pre"][:32]), dict(w_post=i["w_post"].float()),
           dict(gate=i["gate"][:8]), dict(gate=i["h"].half()), dict(h_out=i["h"].float()),
           dict(y=None), dict(n=i["h"][:2]), dict(w_pre=None, n=i["h"]),
           dict(y=None, w_post=None, gate=None, res_scale=0.5),
           dict(y=None, w_post=None, gate=None, w_pre=None)]
    for kw in bad:
        with pytest.raises(ValueError):
            f(**kw)
    with pytest.raises(RuntimeError, match="ALIGN"):
        wide = torch.zeros(8 * 64 + 1, dtype=BF16, device="cuda")
        f(h=wide[1:].view(8, 64))
    with pytest.raises(RuntimeError, match="SHAPE"):
        block.residual_norm_forward(torch.zeros(1, 16392, dtype=BF16, device="cuda"),
                                    w_pre=torch.zeros(16392, dtype=BF16, device="cuda"))
    with pytest.raises(RuntimeError, match="SHAPE"):
        block.residual_norm_forward(torch.zeros(1, 16377, dtype=BF16, device="cuda"),
                                    w_pre=torch.zeros(16377, dtype=BF16, device="cuda"))
    h, n, a, b = f()
    g = lambda **kw: block.residual_norm_backward(**{**dict(  # noqa: E731
        dn=i["dn"], dh_out=i["dh"], h_out=h, y=i["y"], rstd_pre=a, rstd_post=b, w_pre=i["w_pre"],
        w_post=i["w_post"], gate=i["gate"]), **kw})
    for kw in (dict(dn=None), dict(rstd_pre=None), dict(rstd_post=None), dict(y=None),
               dict(w_pre=None), dict(dh_out=i["dh"].float()), dict(dh=i["dh"].float()),
               dict(dw_pre=i["w_pre"]), dict(branch=False), dict(dn=None, w_pre=None, dh_out=None),
               dict(ws=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, RuntimeError)):
            g(**kw)


@pytest.mark.parametrize("M", [1, 2, 149, 300, 1500])
@pytest.mark.parametrize("D", [64, 250, 2048])
def test_an_infinity_stays_where_it_is(M, D):
    """dn of one element infinite: its column's sum is, the others' are finite, also where rows do not
    fill the last round."""
    g = torch.Generator().manual_seed(1)
    h = torch.randn(M, D, generator=g).abs().add(0.5).to(BF16).cuda()
    w = torch.ones(D, dtype=BF16, device="cuda")
    _, _, r, _ = block.residual_norm_forward(h, w_pre=w)
    for row in {0, M // 2, M - 1}:
        dn = torch.randn(M, D, generator=g).to(BF16).cuda()
        dn[row, 5] = float("inf")
        dh, _, dw, _, _ = block.residual_norm_backward(dn, None, h, rstd_pre=r, w_pre=w)
        assert dw[5] == float("inf") and torch.isfinite(dw).sum() == D - 1
        assert torch.isfinite(dh).all(1).sum() == M - 1


def test_given_outputs_are_apart():
    i = _inputs(8, 64, BF16, BF16, True, "channel", True, 1)
    buf = torch.empty(3, 8, 64, dtype=BF16, device="cuda")
    f = lambda **kw: block.residual_norm_forward(**{**dict(  # noqa: E731
        h=i["h"], y=i["y"], w_pre=i["w_pre"], w_post=i["w_post"], gate=i["gate"]), **kw})
    half = torch.empty(12, 64, dtype=BF16, device="cuda")
    for kw in (dict(h_out=i["y"]), dict(n=i["h"]), dict(h_out=buf[0], n=buf[0]),
               dict(h=half[:8], h_out=half[4:]), dict(n=half[:8], y=half[4:])):
        with pytest.raises(ValueError, match="shares memory"):
            f(**kw)
    h, n, a, b = f()
    g = lambda **kw: block.residual_norm_backward(**{**dict(  # noqa: E731
        dn=i["dn"], dh_out=i["dh"], h_out=h, y=i["y"], rstd_pre=a, rstd_post=b, w_pre=i["w_pre"],
        w_post=i["w_post"], gate=i["gate"]), **kw})
    col = torch.empty(64, device="cuda")
    for kw in (dict(dh=h), dict(dy=h), dict(dh=i["dn"]), dict(dh=buf[0], dy=buf[0]),
               dict(dw_pre=col, dw_post=col), dict(dw_pre=col, dgate=col)):
        with pytest.raises(ValueError, match="shares memory"):
            g(**kw)


CALLER = r"""
#include <pthread.h>
#include <stdint.h>
#include "qlora_nf4.h"
typedef qlora_status (*call_t)(const void*, const void*, const void*, const void*, const void*, int,
                               int64_t, int, int, float, float, float, float, void*, void*, float*,
                               float*, qlora_stream_t);
typedef struct { call_t call; const void *h, *w; void* n; int D, calls; qlora_stream_t s; int status; } job;
static void* work(void* p) {
  job* j = (job*)p;
  for (int i = 0; i < j->calls && j->status == QLORA_OK; ++i)
    j->status = j->call(j->h, 0, j->w, 0, 0, 0, 1, j->D, 0, 1e-5f, 1.f, 1.f, 0.f, 0, j->n, 0, 0, j->s);
  return 0;
}
int two(job* a, job* b) {
  pthread_t t;
  if (pthread_create(&t, 0, work, a)) return -1;
  work(b);
  return pthread_join(t, 0);
}
"""


def test_host_threads_at_once(tmp_path):
    """Calls of one kernel that take little and much shared memory, from two host threads on two
    streams: neither changes what the other's launch may take."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    (tmp_path / "caller.c").write_text(CALLER)
    lib = tmp_path / "caller.so"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([gcc, "-shared", "-fPIC", "-O1", "-pthread", "-I" + include,
                    str(tmp_path / "caller.c"), "-o", str(lib)], check=True)

    class Job(ctypes.Structure):
        _fields_ = [("call", ctypes.c_void_p), ("h", ctypes.c_void_p), ("w", ctypes.c_void_p),
                    ("n", ctypes.c_void_p), ("D", ctypes.c_int), ("calls", ctypes.c_int),
                    ("s", ctypes.c_void_p), ("status", ctypes.c_int)]

    call = ctypes.cast(abi._lib().qlora_residual_norm_fwd, ctypes.c_void_p).value
    keep, jobs = [], []
    for D in (33, 16375):
        s = torch.cuda.Stream()
        h, w = (torch.ones(*shape, dtype=BF16, device="cuda") for shape in ((1, D), (D,)))
        n = torch.empty_like(h)
        keep.append((s, h, w, n))
        jobs.append(Job(call, h.data_ptr(), w.data_ptr(), n.data_ptr(), D, 20000, s.cuda_stream, 0))
    torch.cuda.synchronize()
    assert ctypes.CDLL(str(lib)).two(ctypes.byref(jobs[0]), ctypes.byref(jobs[1])) == 0
    torch.cuda.synchronize()
    assert [j.status for j in jobs] == [0, 0]
    for _, h, _, n in keep:
        assert torch.allclose(n.float(), h.float(), rtol=2.0 ** -8)


@pytest.mark.parametrize("size", [2.0 ** -44, 2.0 ** 50])
@pytest.mark.parametrize("D", [264, 37, 8200])
def test_branches_of_any_size(size, D):
    """The branch's norm takes any size out of y: cubes of its 1 / rms, past both ends of fp32 here,
    do not enter the gradients."""
    def change(i):
        i["y"] *= size
    _check(6, D, change=change, eps=0.0, seed=D)
    _check(6, D, R=F32, W=F32, gate="token", change=change, eps=0.0, seed=D)


# Wide rows by one CTA of 1024 threads (whole granules) and by a pair of CTAs, without sums of columns;
# a whole gate of an fp32 residual is read from global memory there.
@pytest.mark.parametrize("D", [8186, 8200, 12243, 16376, 16384])
@pytest.mark.parametrize("R,W,G", [(BF16, BF16, BF16), (F32, F32, F32), (F32, BF16, BF16),
                                   (BF16, F32, F32)])
@pytest.mark.parametrize("post,gate,pre", [(True, "channel", True), (True, "full", True),
                                           (False, "full", True), (False, "token", True),
                                           (True, "none", False), (True, "token", True),
                                           (False, "none", True), (True, "full", False)])
def test_wide_rows_without_column_sums(D, R, W, G, post, gate, pre):
    # More rows than two rounds of every SM have their weights staged, where those fit.
    staged = D == 8200 and R is BF16 and gate in ("none", "token")
    for M in (4, 301) if staged else (4,):
        i = _inputs(M, D, R, W, post, gate, pre, D, G)
        h, _, r_pre, r_post = block.residual_norm_forward(
            i["h"], i["y"], i["w_pre"], i["w_post"], i["gate"], res_scale=0.5, branch_scale=1.25,
            weight_offset=1.0)
        got = dict(zip(("dh", "dy", "dw_pre", "dw_post", "dgate"), block.residual_norm_backward(
            i["dn"], i["dh"], h, i["y"], r_pre, r_post, i["w_pre"], i["w_post"], i["gate"],
            res_scale=0.5, branch_scale=1.25, weight_offset=1.0, need_dw=False,
            need_dgate=gate in ("token", "full"))))
        ref = oracle.backward(_np(i["dn"]), _np(i["dh"]), _np(h), _np(i["y"]), _np(r_pre),
                              _np(r_post), _np(i["w_pre"]), _np(i["w_post"]), _np(i["gate"]), 0.5,
                              1.25, 1.0)
        assert got["dw_pre"] is got["dw_post"] is None
        assert (got["dgate"] is not None) == (gate in ("token", "full"))
        for name, t in got.items():
            if t is None:
                continue
            want, mag = ref[name]
            if name == "dgate" and gate == "token":
                want, mag = want.sum(1, keepdims=True), mag.sum(1, keepdims=True)
            assert t.shape == want.shape, name
            _close(t, want, mag, 256, name)


@pytest.mark.parametrize("D", [136, 35, 2056, 8192, 8200, 8191])
def test_each_gradient_by_itself(D):
    """What is not asked for changes nothing of what is."""
    for gate in ("channel", "token", "full"):
        i, (h, _, r_pre, r_post), whole = _check(7, D, gate=gate, seed=D)
        f = lambda **kw: block.residual_norm_backward(  # noqa: E731
            i["dn"], i["dh"], h, i["y"], r_pre, r_post, i["w_pre"], i["w_post"], i["gate"],
            res_scale=0.5, branch_scale=1.25, weight_offset=1.0, **kw)
        names = ("dh", "dy", "dw_pre", "dw_post", "dgate")
        for kw in (dict(need_dw=False), dict(need_dgate=False), dict(need_dw=False, need_dgate=False)):
            for name, t in zip(names, f(**kw)):
                asked = kw.get("need_dgate", True) if name == "dgate" else \
                    kw.get("need_dw", True) or not name.startswith("dw")
                assert (t is not None) == asked, (name, kw)
                if t is not None:
                    # The sums of wide rows are split otherwise without columns to add up.
                    same = torch.equal(t, whole[name])
                    assert same or (D > 8185 and torch.allclose(t.float(), whole[name].float(),
                                                                rtol=2 ** -7, atol=1e-3)), (name, kw)
