"""GPU parity of the AdamW step (qlora_adamw_step) with the fp64 oracle.

Tolerances, elementwise, u = 2^-24.  m: two products and a sum, the factor and the coefficients
rounded: 6 u of |b1 m| + |(1 - b1) g|; v: one product more: 8 u.  Parameters: 4 u of |p| and 16 u of
the move (6 u from m, root, quotient to 2 ulp, four products), taken with |b1 m| + |(1 - b1) g| for
m: the error that m's two terms bring stays when they cancel and m itself is small.
8-bit codes: a block's scale is off by its largest element's tolerance, x = |m| / scale by its own
and that and 4 u; the decision between two grid values is the oracle's unless the place is within
that of the threshold (and 2^-17, the grain of 16 random bits), and codes are then one apart.
Stochastically rounded bf16: the same with bf16's grid (fp32's own grain is 2^-16 of its step).
"""

import numpy as np
import pytest
import torch

from nf4_base_lora_blockwise_b200 import optim
from oracle import optim as oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _np(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def _lists(sizes, param, grad, seed, scale=1e-2):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda n, s: torch.randn(n, generator=g) * s  # noqa: E731
    full = [rnd(n, 0.05).cuda() for n in sizes]
    grads = [(rnd(n, 1.0) * torch.exp(rnd(n, 1.5)) * scale).to(grad).cuda() for n in sizes]
    if param == "f32":
        return full, grads, None
    return [p.to(BF16) for p in full], grads, full if param == "master" else None


def _run(sizes, param="master", grad=F32, bits=32, steps=3, max_norm=None, seed=0, grad_scale=1.0,
         wd=0.1, lr=1e-2, start=0, betas=(0.9, 0.99), **kw):
    params, grads, masters = _lists(sizes, param, grad, seed)
    lrs = [1.0 + 0.5 * (i % 3) for i in range(len(sizes))]
    wds = [wd * (i % 2) for i in range(len(sizes))]
    opt = optim.AdamW(params, grads, masters, bits=bits, lr=lr, betas=betas, eps=1e-8,
                      lr_scales=lrs, weight_decays=wds, max_grad_norm=max_norm,
                      grad_scale=grad_scale, seed=77, step=start, **kw)
    g = torch.Generator().manual_seed(seed + 1)
    for t in range(start + 1, start + steps + 1):
        for x in grads:
            x.copy_((torch.randn(x.shape, generator=g) * 1e-2).to(x.dtype))
        p0 = [_np(p) for p in (masters or params)]
        m0, v0 = (_np(x) for x in opt.moments())
        norm = opt.step()
        want_norm, factor = oracle.clip_factor([_np(x) for x in grads], grad_scale, max_norm or 0)
        if norm is not None:
            assert abs(float(norm) - want_norm) <= 2 * U * want_norm
        factor = float(np.float32(factor))
        m1, v1 = (_np(x) for x in opt.moments())
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            at = slice(opt.offsets[i], opt.offsets[i] + n)
            gi = _np(grads[i])
            p, m, v, m_mag, move = oracle.step(p0[i], gi, m0[at], v0[at], t, lr * lrs[i], *betas, 1e-8,
                                        wds[i], factor)
            tol = 4 * U * np.abs(p0[i]) + 16 * U * move + 1e-30
            lead = _np((masters or params)[i])
            if param == "bf16":
                # between the bf16 neighbours of p, the upper one by 16 random bits
                rand = (oracle.element_bits(77 ^ 0x55555555, t, opt.offsets[i] + np.arange(n))
                        & np.uint64(0xFFFF)).astype(np.float64)
                step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(p), 1e-30))) - 7)
                place = np.abs(p) / step
                lo = np.floor(place)
                near = np.abs(place - lo + rand / 65536 - 1) < 2.0 ** -15 + tol / step
                want = np.sign(p) * (lo + (place - lo + rand / 65536 >= 1)) * step
                assert np.all((lead == want) | (near & (np.abs(lead - p) <= step + tol)))
                assert np.mean(near) < 0.02 or n < 1000
            else:
                assert np.all(np.abs(lead - p) <= tol), (i, n, t)
                if masters:
                    assert torch.equal(params[i], masters[i].to(BF16))
            m_tol = 6 * U * m_mag
            if bits == 32:
                assert np.all(np.abs(m1[at] - m) <= m_tol + 1e-37)
                assert np.all(np.abs(v1[at] - v) <= 8 * U * v + 1e-37)
            else:
                _codes(opt, i, n, t, m, v, m_tol, m1[at], v1[at])
        # The padding between tensors stays zero.
        for i, n in enumerate(sizes):
            end = opt.offsets[i + 1] if i + 1 < len(sizes) else opt.m.numel()
            assert torch.count_nonzero(opt.m[opt.offsets[i] + n:end]) == 0
            assert torch.count_nonzero(opt.v[opt.offsets[i] + n:end]) == 0
    assert opt.steps == start + steps and opt.skipped == 0
    return opt, params


def _codes(opt, i, n, t, m, v, m_tol, m1, v1):
    first = opt.offsets[i] // 256
    bits = oracle.element_bits(77, t, opt.offsets[i] + np.arange(n)).astype(np.int64)
    codes = {"m": opt.m, "v": opt.v}
    for name, x, tol, values, r16, never in (
            ("m", np.abs(m), m_tol, oracle.M_GRID, bits & 0xFFFF, False),
            ("v", np.sqrt(v), 5 * U * np.sqrt(v), oracle.V_GRID, bits >> 16, True)):
        scale = getattr(opt, name + "_scale")[first:first + -(-n // 256)].double().cpu().numpy()
        tops = np.array([x[b * 256:(b + 1) * 256].max() for b in range(len(scale))])
        off = np.array([tol[b * 256:(b + 1) * 256].max() for b in range(len(scale))])
        assert np.all(np.abs(scale - tops) <= off)
        each, off = np.repeat(tops, 256)[:n], np.repeat(off, 256)[:n]
        x = x / each
        want, distance, step = oracle.encode(np.minimum(x, 1.0), values, r16, never)
        near = distance < ((tol + x * off) / each + 4 * U * x) / step + 2.0 ** -17
        got = codes[name][opt.offsets[i]:opt.offsets[i] + n].cpu().numpy().astype(np.int64)
        if name == "m":
            assert np.all((((got & 128) != 0) == (m < 0)) | (np.abs(m) <= m_tol))
            got = got & 127
        assert np.all((got == want) | (near & (np.abs(got - want) <= 1))), name
        assert np.mean(near) < 0.01 or n < 1000
        # The values are those of the codes.
        scale32 = np.repeat(scale, 256)[:n]
        val = values[got] * scale32
        val = val if name == "m" else val * val
        assert np.all(np.abs((np.abs(m1) if name == "m" else v1) - val) <= 4 * U * np.abs(val))


SIZES = [1, 7, 255, 256, 257, 0, 4096, 4099, 70001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param", ["master", "f32", "bf16"])
@pytest.mark.parametrize("grad", [F32, BF16])
def test_types_and_sizes(bits, param, grad):
    _run(SIZES, param, grad, bits)
    _run(SIZES, param, grad, bits, max_norm=0.1, grad_scale=0.25, seed=5, start=12345)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch(bits):
    sizes = [1 + (37 * i) % 700 for i in range(1100)]
    _run(sizes, bits=bits, steps=2, max_norm=0.5)


@pytest.mark.parametrize("bits,clip", [(8, None), (32, None), (8, 1e9)])
def test_one_large_tensor_and_its_slices(bits, clip):
    """The numbering of elements is all that a step depends on: one tensor whose chunks are drawn, and
    the same memory as 4096 tensors in launches that draw none, leave the same bits."""
    n, part = 4096 * 2048 - 77, 2048
    g = torch.Generator().manual_seed(5)
    p0 = torch.randn(n, generator=g).to(BF16).cuda()
    grads = [(torch.randn(n, generator=g) * 1e-2).cuda() for _ in range(3)]
    left = []
    for split in (False, True):
        p, grad = p0.clone(), torch.zeros(n, device="cuda")
        cut = (lambda t: list(t.split(part))) if split else (lambda t: [t])
        opt = optim.AdamW(cut(p), cut(grad), bits=bits, lr=1e-2, max_grad_norm=clip, seed=3)
        for d in grads:
            grad.copy_(d)
            opt.step()
        assert opt.steps == 3 and opt.skipped == 0
        assert int(opt._state[5]) == int(opt._state[6]) == 0        # tickets and chunks drawn
        left.append([p, opt.m, opt.v] + ([opt.m_scale, opt.v_scale] if bits == 8 else []))
    for a, b in zip(*left):
        assert torch.equal(a, b)


def test_nothing_beyond_the_workspace_and_state():
    """Guards around the workspace and the state of a list that fills the card stay as they are."""
    n = 40_000_000
    p, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    opt = optim.AdamW([p], [g], max_grad_norm=1.0)
    size = opt._ws.numel()
    guarded = torch.full((size + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    state = torch.full((64 + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    state[256:320] = 0
    args = list(opt._args)
    args[7], args[8] = state[256:].data_ptr(), guarded[4096:].data_ptr()
    opt._args = tuple(args)
    opt.step()
    for t, a, b in ((guarded, 4096, 4096 + size), (state, 256, 320)):
        assert torch.all(t[:a] == 0xA5) and torch.all(t[b:] == 0xA5)
    assert torch.any(guarded[4096:4096 + size] != 0xA5)
    assert abs(state[264:268].view(torch.float32).item() - n ** 0.5) <= 2 * U * n ** 0.5


def test_clip_far_away_and_close():
    for max_norm in (1e-6, 1e6):
        _run([5000, 300], max_norm=max_norm, steps=2)
    _run([300], max_norm=None, steps=1, check_finite=True)


def test_scalings_reach_their_tensors():
    """A zero rate leaves a tensor but for nothing else; rates scale the move."""
    params, grads, _ = _lists([1000, 1000], "f32", F32, 3)
    before = [p.clone() for p in params]
    optim.AdamW(params, grads, lr_scales=[0.0, 2.0], lr=1e-3).step()
    assert torch.equal(params[0], before[0])
    # first step: |move| = lr_scale lr |g| / (|g| + eps')
    move = (params[1] - before[1]).abs()
    assert torch.all(move <= 2e-3 * (1 + 1e-4)) and move.median() > 1.9e-3


@pytest.mark.parametrize("bits", [32, 8])
def test_norm_not_finite_changes_nothing(bits):
    for bad in (float("inf"), float("nan")):
        params, grads, masters = _lists([300, 5000], "master", F32, 4)
        opt = optim.AdamW(params, grads, masters, bits=bits, max_grad_norm=1.0)
        opt.step()
        state = [x.clone() for x in (*params, *masters, opt.m, opt.v)]
        keep = grads[1][77].item()
        grads[1][77] = bad
        norm = opt.step()
        assert not torch.isfinite(norm).item()
        for a, b in zip(state, (*params, *masters, opt.m, opt.v)):
            assert torch.equal(a, b)
        assert opt.steps == 1 and opt.skipped == 1
        grads[1][77] = keep
        opt.step()
        assert opt.steps == 2 and opt.skipped == 1
        assert not torch.equal(state[3], masters[1])
    # Without the norm a NaN reaches its block of 8-bit moments and its parameters, and no other.
    params, grads, masters = _lists([300, 5000], "master", F32, 4)
    opt = optim.AdamW(params, grads, masters, bits=8)
    grads[1][700] = float("nan")
    opt.step()
    m, v = opt.moments()
    at = opt.offsets[1] + 512
    assert torch.isnan(m[at:at + 256]).all() and torch.isnan(v[at:at + 256]).all()
    m[at:at + 256] = v[at:at + 256] = 0
    assert torch.isfinite(m).all() and torch.isfinite(v).all()
    bad = torch.isnan(masters[1])
    assert bad[700] and bad.sum() == 1 and not torch.isnan(masters[0]).any()


def test_zero_gradients_and_huge_ones():
    params, grads, _ = _lists([600], "f32", F32, 4)
    before = params[0].clone()
    grads[0].zero_()
    opt = optim.AdamW(params, grads, bits=8, max_grad_norm=1.0, weight_decay=0.0)
    assert float(opt.step()) == 0.0
    assert torch.equal(params[0], before) and torch.count_nonzero(opt.v) == 0
    grads[0].fill_(3e38)     # squares overflow fp32; the norm is a sum in 64 bits
    opt = optim.AdamW(params, grads, max_grad_norm=1.0)
    norm = opt.step()
    assert torch.isinf(norm) or abs(float(norm) - 3e38 * 600 ** 0.5) < 1e34
    grads[0].fill_(1e30)
    opt = optim.AdamW(params, grads, max_grad_norm=1.0)
    assert abs(float(opt.step()) / (1e30 * 600 ** 0.5) - 1) < 1e-6
    assert torch.isfinite(params[0]).all() and opt.steps == 1


def test_small_changes_are_not_lost_in_8_bits():
    """After 1000 steps of random gradients the 8-bit v agrees with the fp32 one in the mean over
    elements.  One step changes v by up to 0.1 %; rounded stochastically with steps of 4.5 % of the
    root its variance is (0.001 x 0.09) / (2 x 0.001), 21 % of an element, 0.4 % of the mean of
    4096, and the square adds a bias below 3 %."""
    g = torch.Generator().manual_seed(1)
    size = torch.exp(torch.randn(4096, generator=g)).cuda() * 1e-3
    grad = torch.zeros(4096, device="cuda")
    opts = [optim.AdamW([torch.zeros(4096, device="cuda")], [grad], bits=b, lr=1e-4)
            for b in (32, 8)]
    cg = torch.Generator(device="cuda").manual_seed(2)
    for _ in range(1000):
        grad.copy_(torch.randn(4096, generator=cg, device="cuda") * size)
        for o in opts:
            o.step()
    v32, v8 = opts[0].moments()[1], opts[1].moments()[1]
    ratio = (v8 / v32).mean().item()
    assert 0.95 < ratio < 1.08, ratio


def test_same_bits_again_graph_and_state_dict():
    sizes = [1000, 65, 4096]

    def fresh():
        params, grads, masters = _lists(sizes, "master", F32, 8)
        return params, optim.AdamW(params, grads, masters, bits=8, max_grad_norm=0.1, seed=3), grads
    pa, a, ga = fresh()
    pb, b, gb = fresh()
    for _ in range(4):
        a.step()
    b.step()
    saved, kept = b.state_dict(), [t.clone() for t in (*b._bound[0], *b._bound[1])]
    # Captured: a replay takes the next step, with what the gradients then hold.
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b.step()
    b.load_state_dict(saved)
    for t, k in zip((*b._bound[0], *b._bound[1]), kept):
        t.copy_(k)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert b.steps == 4
    for x, y in zip((*pa, a.m, a.v, a.m_scale), (*pb, b.m, b.v, b.m_scale)):
        assert torch.equal(x, y)
    with pytest.raises(ValueError):
        optim.AdamW([torch.zeros(9, device="cuda")], [torch.zeros(9, device="cuda")]
                    ).load_state_dict(saved)


def test_learning_rate_on_the_device_and_assigned():
    p1, g1, _ = _lists([500], "f32", F32, 2)
    p2 = [p1[0].clone()]
    rate = torch.full((1,), 1e-3, device="cuda")
    a, b = optim.AdamW(p1, g1, lr=rate), optim.AdamW(p2, g1, lr=1e-3)
    for lr in (1e-3, 5e-4, 0.0):
        a.lr, b.lr = lr, lr
        a.step()
        b.step()
        assert torch.equal(p1[0], p2[0])
    assert float(a.lr) == 0.0 and b.lr == 0.0


def test_moments_are_separately_rounded():
    """The fp32 moments are products and sums rounded one by one, to the bit: what 8-bit codes are
    decided from."""
    n = 100_000
    g = torch.Generator(device="cuda").manual_seed(1)
    grad = torch.randn(n, generator=g, device="cuda")
    opt = optim.AdamW([torch.zeros(n, device="cuda")], [grad], betas=(0.9, 0.999),
                      max_grad_norm=0.3)
    m = v = torch.zeros(n, device="cuda")
    for _ in range(3):
        opt.step()
        norm = grad.double().square().sum().sqrt()
        part = grad * torch.clamp(0.3 / (norm + 1e-6), max=1.0).float()
        m = m * 0.9 + part * (1 - 0.9)
        v = v * 0.999 + part * part * (1 - 0.999)
        assert torch.equal(opt.m[:n], m) and torch.equal(opt.v[:n], v)
        grad.mul_(-0.7)


def test_square_roots_are_the_nearest():
    """Every mantissa under both parities of the exponent, at 1, and near both ends of the range."""
    from nf4_base_lora_blockwise_b200 import abi
    wrong = torch.zeros(4, dtype=torch.int32, device="cuda")
    for x in (1.0, 1.2e-30, 2.0 ** 90):
        first = int(np.float32(x).view(np.uint32))
        first = first if x == 1.0 else first & 0xFF800000
        if x == 1.2e-30:
            first += 1 << 23              # a whole binade above the low end
        abi.qlora_selftest_root(first, 1 << 24, wrong.data_ptr(),
                                torch.cuda.current_stream().cuda_stream)
    assert torch.count_nonzero(wrong) == 0


def test_refusals():
    z = lambda n=8, dtype=F32: torch.zeros(n, dtype=dtype, device="cuda")  # noqa: E731
    p = z()
    bad = [([z().half()], [z()]), ([z()], [z(9)]), ([z()], [torch.zeros(8)]),
           ([z(16)[::2]], [z()]), ([p, p], [z(), z()]), ([p[:4], p], [z(4), z()]), ([p], [p])]
    for params, grads in bad:
        with pytest.raises(ValueError):
            optim.AdamW(params, grads)
    with pytest.raises(ValueError):
        optim.AdamW([z()], [z()], masters=[z()])
    with pytest.raises(ValueError):
        optim.AdamW([z(8, BF16)], [z()], masters=[z(8, BF16)])
    with pytest.raises(ValueError):
        optim.AdamW([z()], [z()], step=-1)
    opt = optim.AdamW([z(9)[1:]], [z()])
    with pytest.raises(RuntimeError, match="ALIGN"):
        opt.step()
    with pytest.raises(RuntimeError, match="SHAPE"):
        optim.AdamW([z()], [z()], betas=(1.0, 0.9)).step()
    # What the caller does to its tensors afterwards does not free what is bound.
    q, g = z(), z()
    opt = optim.AdamW([q], [g])
    q.data, g.data = z(1), z(1)
    opt.step()
    torch.cuda.synchronize()


@pytest.mark.parametrize("lr,wd", [(2e-6, 0.01), (5e-6, 0.01), (2e-5, 0.01), (4e-4, 0.01),
                                   (1e-3, 0.1)])
@pytest.mark.parametrize("param", ["f32", "master"])
def test_small_decays_are_rounded_once(lr, wd, param):
    """p - lr wd p is rounded with p, not as 1 - lr wd before: for p in [1, 2) off by half a step, 2^-24,
    and by the roundings of lr, wd, their product and its product with p, 2^-22 of the decay."""
    n = 1 << 20
    p = 1.0 + torch.arange(n, dtype=torch.float64, device="cuda").div(n).float()
    before = p.double()
    grad = torch.zeros(n, device="cuda")
    if param == "f32":
        opt = optim.AdamW([p], [grad], lr=lr, weight_decay=wd)
    else:
        opt = optim.AdamW([p.to(BF16)], [grad], [p], bits=8, lr=lr, weight_decay=wd)
    opt.step()
    decay = lr * wd * before
    err = (p.double() - (before - decay)).abs()
    assert torch.all(err <= U + 4 * U * decay), float((err / (U + 4 * U * decay)).max())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("scale,applied", [(1.0, False), (1e-4, True)])
def test_the_reported_norm_decides(bits, scale, applied):
    """A norm past fp32's largest number, though the 64-bit sum holds it, is an infinity: what step()
    returns says whether the step was taken."""
    params, grads, masters = _lists([600, 300], "master", F32, 4)
    for g in grads:
        g.fill_(3e38)
    opt = optim.AdamW(params, grads, masters, bits=bits, max_grad_norm=1.0, grad_scale=scale)
    before = [t.clone() for t in (*params, *masters, opt.m, opt.v)]
    norm = opt.step()
    assert torch.isfinite(norm).item() == applied
    assert (opt.steps, opt.skipped) == ((1, 0) if applied else (0, 1))
    same = [torch.equal(a, b) for a, b in zip(before, (*params, *masters, opt.m, opt.v))]
    assert not any(same[2:4]) if applied else all(same)


def test_a_rate_in_written_memory_is_refused():
    """The learning rate is read while parameters and masters are written; a gradient may hold it."""
    w, g = torch.zeros(16, device="cuda"), torch.zeros(16, device="cuda")
    p = torch.zeros(16, dtype=BF16, device="cuda")
    for args in (([w], [g], None), ([p], [g], [w])):
        with pytest.raises(ValueError, match="shares memory"):
            optim.AdamW(*args, lr=w[3:4])
    for lr in (g[3:4], torch.full((), 1e-3, device="cuda")):
        optim.AdamW([w], [g], lr=lr).step()
    torch.cuda.synchronize()


def test_the_bound_rate_stays():
    """As with the tensors of the lists: what the caller does to its rate does not free what is bound."""
    rate = torch.full((1,), 1e-3, device="cuda")
    opt = optim.AdamW([torch.zeros(8, device="cuda")], [torch.ones(8, device="cuda")], lr=rate)
    bound = rate.data_ptr()
    rate.data = torch.zeros(1, device="cuda")
    assert opt.lr.data_ptr() == bound == opt._config.lr_device and opt.lr.item() == rate.new_tensor(1e-3).item()
    opt.lr = 2e-3
    opt.step()
    assert torch.all((opt._bound[0][0] + 2e-3).abs() < 1e-6)
