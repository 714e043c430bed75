"""GPU parity of rotary positions (qlora_rope) with the extended-precision oracle.

Tolerance, elementwise: one rounding to the output's type (2^-8 of the value for bf16, 2^-24 for
fp32) and 16 x 2^-24 of scale (|a| + |b|): the fp32 angle is off by at most 2^-25 half turns
(2^-23.3 radians: 2 units), sincospif by 2 ulp (2 units), its product with scale, the two products
and the sum by half an ulp each.
"""

import numpy as np
import pytest
import torch

from nf4_base_lora_blockwise_b200 import block
from oracle import block as oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
RAMP = {"kind": "ramp", "factor": 16.0, "slow": 1.0, "fast": 32.0, "original": 4096}
BANDS = {"kind": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "original": 8192}


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _np(t):
    return t.detach().double().cpu().numpy()


def _agree(got, x, positions, plan, base, scaling, inverse, what=""):
    """got, x: [M, heads, hd] (any strides) on the GPU."""
    f, scale = oracle.frequencies(plan.rotary_dim, base, scaling)
    want, mag = oracle.rope(_np(x), positions, f, scale, plan.rotary_dim, plan.interleaved, inverse)
    rd = plan.rotary_dim
    half = 2.0 ** -8 if got.dtype is BF16 else U
    err = np.abs(_np(got) - want)[..., :rd]
    tol = (half * np.abs(want) * (1 + 2.0 ** -8) + 16 * U * mag)[..., :rd] + 1e-37
    assert np.all(err <= tol), (what, float(np.max(err / tol)))
    assert torch.equal(got[..., rd:], x[..., rd:]), what


def _rnd(*shape, dtype=BF16, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("hd,rd", [(128, 128), (128, 64), (64, 64), (80, 80), (80, 40), (96, 24),
                                   (192, 128), (256, 256), (36, 36), (36, 18), (72, 24), (40, 8),
                                   (10, 6), (7, 2),
                                   (2, 2), (33, 32), (512, 510), (2048, 2048)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_layouts(hd, rd, interleaved):
    """In place and out of place, both directions, both types; q and k of different head counts."""
    plan = block.rope_plan(hd, rotary_dim=rd, scaling=RAMP, interleaved=interleaved)
    pos = torch.tensor([0, 1, 5, 4095, 70000], dtype=torch.int32, device="cuda")
    for dtype in (BF16, F32):
        for inverse in (False, True):
            q, k = _rnd(5, 3 * hd, dtype=dtype, seed=hd), _rnd(5, 2 * hd, dtype=dtype, seed=rd)
            q0, k0 = q.clone(), k.clone()
            oq, ok = block.rope(q, pos, plan, k=k, inverse=inverse, inplace=False)
            assert torch.equal(q, q0) and torch.equal(k, k0)
            for got, x, n in ((oq, q0, 3), (ok, k0, 2)):
                _agree(got.view(5, n, hd), x.view(5, n, hd), pos.tolist(), plan, 10000.0, RAMP,
                       inverse)
            a, b = block.rope(q, pos, plan, k=k, inverse=inverse)
            assert a is q and b is k
            assert torch.equal(q, oq) and torch.equal(k, ok)


@pytest.mark.parametrize("M", [1, 2, 16, 147, 591, 593, 2048])
def test_packed_rows_and_token_counts(M):
    """q and k heads of packed q/k/v rows are turned in place; v and the rows' ends stay."""
    hd, hq, hk = 128, 4, 2
    plan = block.rope_plan(hd, base=500000.0, scaling=BANDS)
    qkv = _rnd(M, (hq + 2 * hk) * hd, seed=M)
    before = qkv.clone()
    pos = torch.randint(0, 1 << 20, (M,), generator=torch.Generator().manual_seed(M)).cuda()
    assert block.rope(qkv, pos, plan, n_heads=hq + hk) is qkv
    v = qkv.view(M, -1, hd)
    _agree(v[:, :hq + hk], before.view(M, -1, hd)[:, :hq + hk], pos.tolist(), plan, 500000.0, BANDS,
           False)
    assert torch.equal(v[:, hq + hk:], before.view(M, -1, hd)[:, hq + hk:])


def test_positions_of_any_sign_and_size():
    plan = block.rope_plan(64)
    far = [0, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 12345678]
    for dtype, pos in ((torch.int32, far), (torch.int64, far + [2 ** 40 + 3, -2 ** 40])):
        x = _rnd(len(pos), 2, 64, dtype=F32)
        out = block.rope(x, torch.tensor(pos, dtype=dtype, device="cuda"), plan, inplace=False)
        _agree(out, x, pos, plan, 10000.0, None, False)
    x = _rnd(6, 2, 64)
    counted = block.rope(x, 131070, plan, inplace=False)
    given = block.rope(x, torch.arange(131070, 131076, device="cuda"), plan, inplace=False)
    assert torch.equal(counted, given)


def test_strided_views_and_batches():
    """[B, S, n, hd] of token-major and head-major memory, rows with gaps, odd alignment."""
    B, S, n, hd = 3, 5, 4, 64
    plan = block.rope_plan(hd, rotary_dim=48, interleaved=True)
    pos = torch.randint(0, 9999, (B, S), generator=torch.Generator().manual_seed(1)).cuda()
    x = _rnd(B, S, n, hd)
    want = block.rope(x.clone(), pos, plan)
    _agree(want.view(B * S, n, hd), x.view(B * S, n, hd), pos.flatten().tolist(), plan, 10000.0,
           None, False)
    heads = x.transpose(1, 2).contiguous()                  # [B, n, S, hd]
    block.rope(heads.transpose(1, 2), pos, plan)
    assert torch.equal(heads.transpose(1, 2), want)
    wide = torch.zeros(B, S, n + 2, hd + 3, dtype=BF16, device="cuda")   # gaps, odd strides
    view = wide[:, :, 1:n + 1, 1:hd + 1]
    view.copy_(x)
    block.rope(view, pos, plan)
    assert torch.equal(view, want)
    wide[:, :, 1:n + 1, 1:hd + 1] = 0
    assert torch.count_nonzero(wide) == 0
    out = torch.empty(B, n, S, hd, dtype=BF16, device="cuda").transpose(1, 2)
    assert block.rope(x, pos, plan, out=out) is out and torch.equal(out, want)
    one = block.rope(x, 7, plan, inplace=False)             # counts along S in every batch
    same = block.rope(x, (7 + torch.arange(S)).repeat(B, 1).cuda(), plan, inplace=False)
    assert torch.equal(one, same)
    part = block.rope(x, pos, plan, n_heads=2, inplace=False)
    assert part.shape == (B, S, 2, hd) and torch.equal(part, want[:, :, :2])


def test_backward_is_the_transpose():
    """The gradient of <rope(x), d>: rope's transpose, against central differences of the fp32 form
    (linear in x, so a difference of step 1 is exact up to rounding)."""
    plan = block.rope_plan(16, rotary_dim=12, scaling=RAMP)
    x, d = _rnd(3, 2, 16, dtype=F32, seed=1), _rnd(3, 2, 16, dtype=F32, seed=2)
    pos = torch.tensor([3, 100, 2000], device="cuda")
    grad = block.rope(d, pos, plan, inverse=True, inplace=False)
    eye = torch.eye(96, device="cuda").view(96, 3, 2, 16)
    for j in range(96):
        hi = block.rope(x + eye[j], pos, plan, inplace=False)
        lo = block.rope(x - eye[j], pos, plan, inplace=False)
        diff = (((hi.double() - lo.double()) * d.double()).sum() / 2).item()
        # up to 32 products of values below 5 by 5, each off by a few 2^-24 of it
        assert abs(diff - grad.flatten()[j].item()) <= 32 * 25 * 8 * U


def test_no_tokens_and_graph():
    plan = block.rope_plan(64)
    empty = torch.empty(0, 128, dtype=BF16, device="cuda")
    assert block.rope(empty, torch.empty(0, dtype=torch.int32, device="cuda"), plan) is empty
    x = _rnd(40, 128)
    pos = torch.arange(40, device="cuda", dtype=torch.int32)
    block.rope(x, pos, plan, inplace=False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.rope(x, pos, plan, inplace=False)
    pos += 1000
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, block.rope(x, pos, plan, inplace=False))


def test_offsets_past_32_bits():
    M, hd, n = 33000, 2048, 32                               # 2^31 and more elements
    x = torch.zeros(M, n * hd, dtype=BF16, device="cuda")
    x[-2:] = _rnd(2, n * hd)
    last = x[-2:].clone()
    plan = block.rope_plan(hd)
    block.rope(x, 5, plan)
    _agree(x[-2:].view(2, n, hd), last.view(2, n, hd), [5 + M - 2, 5 + M - 1], plan, 10000.0, None,
           False)
    assert torch.count_nonzero(x[:-2]) == 0


def test_refusals():
    plan = block.rope_plan(64)
    x = _rnd(4, 256)
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    bad = [dict(x=x.half()), dict(x=x.cpu()), dict(x=_rnd(4, 100)), dict(x=_rnd(4, 4, 32)),
           dict(n_heads=5), dict(n_heads=0), dict(positions=pos[:3]), dict(positions=pos.float()),
           dict(positions=pos.cpu()), dict(k=x.float()), dict(k=_rnd(5, 64)), dict(n_heads_k=1),
           dict(out=x.float()), dict(out=_rnd(4, 128)), dict(x=_rnd(64, 4).t().reshape(4, 64)[:, ::2]),
           dict(x=_rnd(4, 1, 64).expand(4, 4, 64)),
           dict(x=_rnd(1, 256).expand(4, 256))]
    for kw in bad:
        with pytest.raises(ValueError):
            block.rope(**{**dict(x=x, positions=pos, plan=plan), **kw})
    with pytest.raises(ValueError):
        block.rope(x, pos, block.rope_plan(64, device="cpu"))
    # An input may repeat (one row for every token) when the output is another tensor.
    row = _rnd(1, 256)
    out = block.rope(row.expand(4, 256), pos, plan, inplace=False)
    _agree(out.view(4, 4, 64), row.expand(4, 256).view(4, 4, 64), pos.tolist(), plan, 10000.0, None,
           False)


def test_what_is_written_is_apart():
    """q and k of one packed row or cache are; the same heads twice, or an output over its input, not."""
    plan = block.rope_plan(64)
    row = _rnd(2, 6, 8 * 64)
    want = block.rope(row.view(12, 512), 3, plan, n_heads=6, inplace=False)
    for parts in (lambda t: (t[..., :256], t[..., 256:384]), lambda t: (t[..., 256:384], t[..., :256])):
        r = row.clone().view(12, 512)
        q, k = parts(r)
        block.rope(q, 3, plan, k=k)
        assert torch.equal(r[:, :384], want) and torch.equal(r[:, 384:], row.view(12, 512)[:, 384:])
    cache = _rnd(2, 5, 6, 64)                                # [B, heads, S, 64]: heads further apart
    c = cache.clone().transpose(1, 2)
    block.rope(c[:, :, :3], 0, plan, k=c[:, :, 3:])
    assert torch.equal(c, block.rope(cache.transpose(1, 2), 0, plan, inplace=False))
    x, wide = _rnd(4, 256), _rnd(4, 320)
    same = x.clone()
    block.rope(same, 0, plan, out=same)                      # in place by name
    assert torch.equal(same, block.rope(x, 0, plan, inplace=False))
    y = _rnd(4, 256)
    for kw in (dict(k=x), dict(k=x[:, 64:]), dict(k=x[1:2].expand(4, 256)), dict(x=wide[:, :256], out=wide[:, 64:]),
               dict(k=y, out=y), dict(k=y, out=torch.empty_like(x), out_k=x),
               dict(k=y, out=wide[:, :256], out_k=wide[:, 64:])):
        with pytest.raises(ValueError, match="share"):
            block.rope(**{**dict(x=x, positions=0, plan=plan), **kw})
    for hd, rd in ((0, 0), (64, 0), (32, 64)):
        with pytest.raises(ValueError):
            block.rope(x, 0, block.RopePlan(plan.phase[:rd // 2], 1.0, hd, rd))


@pytest.mark.parametrize("heads,heads_k,rd", [(4096, None, 2), (1100, 1029, 2), (2049, 2047, 4),
                                              (1200, None, 1024), (4096, None, 2048)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_the_most_and_widest_heads(heads, heads_k, rd, interleaved):
    """Up to 4096 heads of 2048, few of whose elements are turned: every copied element of every head
    is written once, from its own place."""
    plan = block.rope_plan(2048, rotary_dim=rd, interleaved=interleaved)
    x = _rnd(1, heads, 2048, seed=rd)
    k = None if heads_k is None else _rnd(1, heads_k, 2048, seed=rd + 1)
    outs = block.rope(x, 777, plan, k=k, out=torch.zeros_like(x),
                      out_k=None if k is None else torch.zeros_like(k))
    for got, of in zip([outs] if k is None else outs, (x, k)):
        _agree(got, of, [777], plan, 10000.0, None, False)
