"""The operators between the linears together with them: one training step of a decoder block (norms
with gate and residual scale, packed q/k/v, rotary positions, SwiGLU MLP, AdamW on the adapters),
its gradients against float64 autograd of the same block, the step captured into a CUDA graph, and
a token by itself.

Tolerance of the gradients: every stored bf16 tensor is off by up to 2^-8 of its values, and the
longest path from the input to a gradient passes about 20 of them, forward and back.  Independent
roundings add as the root of their number: sqrt(20) 2^-8 = 1.7 % of the largest value for factors
of about one a stage; 5 % leaves room for three times that.
"""

import numpy as np
import pytest
import torch

from nf4_base_lora_blockwise_b200 import block, linear, optim

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
B, S, D, HQ, HK, HD, I, R = 2, 48, 256, 4, 2, 64, 384, 8
M, ALPHA, RES, BR = B * S, 16.0, 0.9, 0.5
ROWS = [HQ * HD, HK * HD, HK * HD]
TOL = 5e-2


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


class Block:
    """Weights, adapters (with fp32 masters) and the gradients' buffers of one block."""

    def __init__(self, seed, bits=8):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).cuda()  # noqa: E731
        self.base, self.A, self.B = {}, {}, {}
        shapes = {"qkv": (sum(ROWS), D, 3), "o": (D, HQ * HD, 1), "gu": (2 * I, D, 2),
                  "down": (D, I, 1)}
        masters = []
        for name, (n, k, groups) in shapes.items():
            self.base[name] = linear.nf4_pack(rnd(n, k, std=k ** -0.5).to(BF16))
            for store, shape in ((self.A, (groups * R, k)), (self.B, (n, R))):
                masters.append(rnd(*shape, std=0.05))
                store[name] = masters[-1].to(BF16)
        self.w = {k: (1 + rnd(D, std=0.1)).to(BF16) for k in ("in", "post", "mid", "out")}
        self.gate = rnd(D, std=0.5).to(BF16)
        self.plan = block.rope_plan(HD, base=10000.0)
        self.pos = torch.arange(S, dtype=torch.int32).repeat(B).cuda()
        self.params = [t for n in shapes for t in (self.A[n], self.B[n])]
        self.grads = [torch.zeros(p.shape, device="cuda") for p in self.params]
        self.of = {n: (self.grads[2 * i], self.grads[2 * i + 1]) for i, n in enumerate(shapes)}
        self.masters = masters
        self.opt = optim.AdamW(self.params, self.grads, masters, bits=bits, lr=1e-3,
                               max_grad_norm=0.3, weight_decay=0.01, seed=seed)


def _attention(q, k, v):
    """Causal attention of [B, S, heads, HD] in the type of q (a stand-in for the user's own)."""
    k, v = (t.repeat_interleave(HQ // HK, dim=2) for t in (k, v))
    z = torch.einsum("bihd,bjhd->bhij", q, k) * HD ** -0.5
    z = z.masked_fill(torch.ones(S, S, device=q.device).triu(1).bool(), float("-inf"))
    return torch.einsum("bhij,bjhd->bihd", z.softmax(-1), v).reshape(M, HQ * HD)


def _split(qkv, dtype):
    heads = qkv.view(B, S, -1, HD).to(dtype)
    return heads[:, :, :HQ], heads[:, :, HQ:HQ + HK], heads[:, :, HQ + HK:]


def _step(b, h0, dn, update=True):
    """Forward, backward for the upstream gradient dn of the last norm, and AdamW."""
    _, n1, r1, _ = block.residual_norm_forward(h0, w_pre=b.w["in"])
    qkv, xa_qkv = linear.grouped_forward(n1, b.base["qkv"], b.A["qkv"], b.B["qkv"], ROWS, ALPHA)
    block.rope(qkv, b.pos, b.plan, n_heads=HQ + HK)
    parts = [t.requires_grad_() for t in _split(qkv, F32)]
    with torch.enable_grad():
        att32 = _attention(*parts)
    att = att32.detach().to(BF16)
    o, xa_o = linear.forward(att, b.base["o"], b.A["o"], b.B["o"], ALPHA)
    h1, n2, r2, rp = block.residual_norm_forward(h0, o, b.w["mid"], b.w["post"], b.gate,
                                                 res_scale=RES, branch_scale=BR)
    gu, xa_gu = linear.grouped_forward(n2, b.base["gu"], b.A["gu"], b.B["gu"], [I, I], ALPHA)
    act = linear.swiglu_packed_forward(gu)
    down, xa_d = linear.forward(act, b.base["down"], b.A["down"], b.B["down"], ALPHA)
    h2, n3, r3, _ = block.residual_norm_forward(h1, down, b.w["out"])

    dh1, ddown, dw_out, _, _ = block.residual_norm_backward(dn, None, h2, rstd_pre=r3,
                                                            w_pre=b.w["out"], branch=True)
    dact, *_ = linear.backward(ddown, act, b.base["down"], b.A["down"], b.B["down"], xa_d, ALPHA,
                               dA=b.of["down"][0], dB=b.of["down"][1])
    dgu = linear.swiglu_packed_backward(gu, dact)
    dn2, *_ = linear.grouped_backward(dgu, n2, b.base["gu"], b.A["gu"], b.B["gu"], xa_gu, [I, I],
                                      ALPHA, dA=b.of["gu"][0], dB=b.of["gu"][1])
    dh0, do, dw_mid, dw_post, dgate = block.residual_norm_backward(
        dn2, dh1, h1, o, r2, rp, b.w["mid"], b.w["post"], b.gate, res_scale=RES, branch_scale=BR)
    datt, *_ = linear.backward(do, att, b.base["o"], b.A["o"], b.B["o"], xa_o, ALPHA,
                               dA=b.of["o"][0], dB=b.of["o"][1])
    dparts = torch.autograd.grad(att32, parts, datt.float())
    dqkv = torch.cat([t.reshape(M, -1) for t in dparts], 1).to(BF16)
    block.rope(dqkv, b.pos, b.plan, n_heads=HQ + HK, inverse=True)
    dn1, *_ = linear.grouped_backward(dqkv, n1, b.base["qkv"], b.A["qkv"], b.B["qkv"], xa_qkv,
                                      ROWS, ALPHA, dA=b.of["qkv"][0], dB=b.of["qkv"][1])
    dh, _, dw_in, _, _ = block.residual_norm_backward(dn1, dh0, h0, rstd_pre=r1, w_pre=b.w["in"])
    norm = b.opt.step() if update else None
    return n3, dh, {"in": dw_in, "mid": dw_mid, "post": dw_post, "out": dw_out}, dgate, norm


def _reference(b, h0, dn):
    """The same block in float64, by autograd."""
    leaf = lambda t: t.detach().to(F64).requires_grad_()  # noqa: E731
    A = {k: leaf(v) for k, v in b.A.items()}
    Bm = {k: leaf(v) for k, v in b.B.items()}
    w, gate, h = {k: leaf(v) for k, v in b.w.items()}, leaf(b.gate), leaf(h0)
    W = {k: linear.nf4_dequant(v).to(F64) for k, v in b.base.items()}
    rms = lambda x, g: x * (x.square().mean(1, keepdim=True) + 1e-5).rsqrt() * g  # noqa: E731

    def layer(name, x, rows):
        y, at = [], 0
        for i, n in enumerate(rows):
            a = A[name][i * R:(i + 1) * R]
            y.append(x @ W[name][at:at + n].T + ALPHA / R * (x @ a.T) @ Bm[name][at:at + n].T)
            at += n
        return torch.cat(y, 1)

    def turn(x):  # [B, S, heads, HD]
        f = 10000.0 ** (-torch.arange(0, HD, 2, dtype=F64, device="cuda") / HD)
        a = b.pos.view(B, S, 1, 1).to(F64) * f
        p, q = x.chunk(2, -1)
        return torch.cat([p * a.cos() - q * a.sin(), q * a.cos() + p * a.sin()], -1)

    q, k, v = _split(layer("qkv", rms(h, w["in"]), ROWS), F64)
    o = layer("o", _attention(turn(q), turn(k), v), [D])
    h1 = RES * h + BR * gate * rms(o, w["post"])
    g, u = layer("gu", rms(h1, w["mid"]), [I, I]).chunk(2, 1)
    h2 = h1 + layer("down", torch.nn.functional.silu(g) * u, [D])
    n3 = rms(h2, w["out"])
    leaves = [h, gate, *w.values(), *(t for n in A for t in (A[n], Bm[n]))]
    grads = torch.autograd.grad(n3, leaves, dn.to(F64))
    return n3, grads[0], dict(zip(w, grads[2:6])), grads[1], list(grads[6:])


def _inputs(seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, D, generator=g).to(BF16).cuda(),
            (torch.randn(M, D, generator=g) * 1e-2).to(BF16).cuda())


def test_gradients_of_a_training_step():
    b = Block(1)
    h0, dn = _inputs(2)
    n3, dh, dw, dgate, _ = _step(b, h0, dn, update=False)
    want = _reference(b, h0, dn)
    pairs = [("n3", n3, want[0]), ("dh", dh, want[1]), ("dgate", dgate, want[3])]
    pairs += [("dw " + k, dw[k], want[2][k]) for k in dw]
    pairs += [(f"adapter {i}", g, r) for i, (g, r) in enumerate(zip(b.grads, want[4]))]
    for name, got, ref in pairs:
        err = ((got.to(F64) - ref).abs().max() / ref.abs().max()).item()
        assert err <= TOL, (name, err)
    assert linear.device_error() == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_captured_and_replayed(bits):
    """Three replays of a captured step leave the bits that three eager steps leave."""
    h0, dn = _inputs(3)
    eager = Block(4, bits)
    for _ in range(3):
        out = _step(eager, h0, dn)
    assert torch.isfinite(out[4]).all() and eager.opt.steps == 3
    for p, m in zip(eager.params, eager.masters):
        assert torch.equal(p, m.to(BF16))
    again = Block(4, bits)
    start = [t.clone() for t in (*again.params, *again.masters)]
    saved = again.opt.state_dict()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(again, h0, dn)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(again, h0, dn)
    again.opt.load_state_dict(saved)
    for t, s in zip((*again.params, *again.masters), start):
        t.copy_(s)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert again.opt.steps == 3
    for a, c in zip((*eager.params, *eager.masters, *eager.grads, eager.opt.m, eager.opt.v),
                    (*again.params, *again.masters, *again.grads, again.opt.m, again.opt.v)):
        assert torch.equal(a, c)


def test_two_models_step_on_two_streams():
    """Handles, workspaces and outputs of two blocks at once do not meet."""
    h0, dn = _inputs(5)
    alone = [Block(6), Block(7)]
    for b in alone:
        for _ in range(3):
            _step(b, h0, dn)
    torch.cuda.synchronize()
    both = [Block(6), Block(7)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for b, s in zip(both, streams):
            with torch.cuda.stream(s):
                _step(b, h0, dn)
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        for p, q in zip((*x.params, x.opt.m), (*y.params, y.opt.m)):
            assert torch.equal(p, q)


def test_a_token_by_itself():
    """Norms and rotations of a row do not depend on the batch it is in."""
    b = Block(8)
    h0, y = _inputs(9)
    args = dict(w_pre=b.w["mid"], w_post=b.w["post"], gate=b.gate, res_scale=RES, branch_scale=BR)
    whole = block.residual_norm_forward(h0, y, **args)
    qkv = torch.randn(M, sum(ROWS), device="cuda").to(BF16)
    turned = block.rope(qkv, b.pos, b.plan, n_heads=HQ + HK, inplace=False)
    for i in (0, 17, M - 1):
        one = block.residual_norm_forward(h0[i:i + 1], y[i:i + 1], **args)
        for a, c in zip(whole, one):
            assert torch.equal(a[i:i + 1], c)
        t = block.rope(qkv[i:i + 1], int(b.pos[i]), b.plan, n_heads=HQ + HK, inplace=False)
        assert torch.equal(t[0], turned[i])


def test_other_streams_wait_for_nothing_else():
    """A call runs on the current stream: work queued before it on that stream is seen."""
    s = torch.cuda.Stream()
    h = torch.zeros(512, 4096, dtype=BF16, device="cuda")
    w = torch.ones(4096, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        h.fill_(3.0)
        _, n, _, _ = block.residual_norm_forward(h, w_pre=w)
        block.rope(n, 0, block.rope_plan(128), inplace=True)
    s.synchronize()
    # rms 1 rows of ones, turned: every pair keeps its length sqrt(2)
    length = n.float().view(512, 32, 2, 64).square().sum(2).sqrt()
    assert np.allclose(length.cpu().numpy(), 2 ** 0.5, rtol=2 ** -6)
