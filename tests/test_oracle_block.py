"""Pins of the oracles of the residual norm, rotary positions and AdamW (CPU): gradients against
differences, rotations against their composition law, 8-bit grids against their definition."""

import numpy as np
import pytest
import torch

from oracle import block, optim


def _norm_case(seed, M=3, D=7, post=True, gate="channel", pre=True):
    r = np.random.default_rng(seed)
    shape = {"none": None, "channel": (D,), "token": (M, 1), "full": (M, D)}[gate]
    return dict(h=r.normal(size=(M, D)), y=r.normal(size=(M, D)), eps=1e-3, res=0.7, br=1.3, o=0.5,
                w_pre=r.normal(size=D) if pre else None, w_post=r.normal(size=D) if post else None,
                gate=None if shape is None else r.normal(size=shape))


def _forward(c):
    h, _, r_post = block.update(c["h"], c["y"], c["w_post"], c["gate"], c["eps"], c["res"],
                                c["br"], c["o"])
    n, r_pre = block.norm(h, c["w_pre"], c["eps"], c["o"]) if c["w_pre"] is not None else (0, None)
    return h, n, r_pre, r_post


@pytest.mark.parametrize("post,gate,pre", [(True, "channel", True), (False, "token", True),
                                           (True, "full", True), (False, "none", False),
                                           (True, "none", True)])
def test_norm_backward_against_differences(post, gate, pre):
    c = _norm_case(1, post=post, gate=gate, pre=pre)
    r = np.random.default_rng(2)
    dn, dh = r.normal(size=c["h"].shape), r.normal(size=c["h"].shape)

    def loss(**change):
        h, n, _, _ = _forward({**c, **change})
        return np.sum(h * dh) + np.sum(n * dn)

    h, _, r_pre, r_post = _forward(c)
    got = block.backward(dn if pre else None, dh, h, c["y"], r_pre, r_post, c["w_pre"],
                         c["w_post"], c["gate"], c["res"], c["br"], c["o"])
    names = {"dh": "h", "dy": "y", "dw_pre": "w_pre", "dw_post": "w_post", "dgate": "gate"}
    for name, of in names.items():
        if c[of] is None:
            assert name not in got
            continue
        grad = got[name][0]
        if name == "dgate":  # summed along what it is broadcast over
            grad = {1: grad.sum(0), 2: grad.sum(1, keepdims=True)
                    if c["gate"].shape[1:] == (1,) else grad}[c["gate"].ndim]
        e = 1e-6
        for idx in np.ndindex(c[of].shape):
            d = np.zeros_like(c[of])
            d[idx] = e
            diff = (loss(**{of: c[of] + d}) - loss(**{of: c[of] - d})) / (2 * e)
            # central difference: O(e^2) plus rounding 1e-16 / e of a loss of size ~10
            assert abs(diff - grad[idx]) <= 1e-7 * (1 + abs(diff)), (name, idx)
        assert np.all(got[name][1] >= np.abs(got[name][0]) - 1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_rotation(interleaved):
    """Positions add, the inverse undoes, lengths stay, elements past rd pass through."""
    r = np.random.default_rng(3)
    x = r.normal(size=(4, 2, 10))
    f, s = block.frequencies(6, 100.0)
    turn = lambda x, p, inv=False: block.rope(x, p, f, s, 6, interleaved, inv)[0]  # noqa: E731
    p, q = [0, 3, -5, 1000], [7, 0, 2, 2 ** 40]
    both = turn(turn(x, p), q)
    assert np.allclose(both, turn(x, [a + b for a, b in zip(p, q)]), atol=1e-6)
    assert np.allclose(turn(turn(x, q), q, True), x, atol=1e-12)
    assert np.allclose(np.sum(both ** 2, -1), np.sum(x ** 2, -1))
    assert np.array_equal(both[..., 6:], x[..., 6:])
    assert np.array_equal(turn(x, [0] * 4), x)


def test_frequencies_kinds():
    f, _ = block.frequencies(64, 10000.0)
    same = lambda a, b: np.allclose(np.float64(a), np.float64(b), rtol=1e-12)  # noqa: E731
    assert same(f[0], 1.0) and same(f[-1], 10000.0 ** (-62 / 64))
    assert same(block.frequencies(64, 10000.0, {"kind": "linear", "factor": 4})[0], f / 4)
    g, _ = block.frequencies(64, 10000.0, {"kind": "base", "factor": 4})
    assert same(g[0], 1.0) and same(g[-1], f[-1] / 4)
    g, s = block.frequencies(64, 10000.0, {"kind": "bands", "factor": 8, "low": 1, "high": 4,
                                           "original": 2048})
    assert s == 1.0 and same(g[0], f[0]) and same(g[-1], f[-1] / 8)
    assert np.all(g <= f) and np.all(g >= f / 8)
    g, s = block.frequencies(64, 10000.0, {"kind": "ramp", "factor": 16, "slow": 1, "fast": 32,
                                           "original": 2048})
    assert same(g[0], f[0]) and same(g[-1], f[-1] / 16) and abs(s - (0.1 * np.log(16) + 1)) < 1e-12


def test_adamw_against_torch():
    r = np.random.default_rng(4)
    p0 = r.normal(size=50)
    p = torch.nn.Parameter(torch.tensor(p0))
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p0.copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = r.normal(size=50)
        p.grad = torch.tensor(g)
        opt.step()
        q, m, v, *_ = optim.step(q, g, m, v, t, 1e-2, 0.8, 0.95, 1e-6, 0.1, 1.0)
    assert np.allclose(p.detach().numpy(), q, rtol=1e-12, atol=1e-14)


def test_grids():
    assert optim.M_GRID[127] == 1.0 and optim.V_GRID[255] == 1.0
    assert optim.M_GRID[126] == 0.9375 and optim.V_GRID[254] == 1 - 1 / 32
    for values in (optim.M_GRID, optim.V_GRID):
        assert np.all(np.diff(values) > 0) and values[0] == 0 and 1e-5 < values[1] < 2e-5
        assert np.array_equal(values.astype(np.float32), values)
    # On a grid value no random number moves it; between two, the share of random numbers that
    # round up is the place between them.
    every = np.arange(65536)
    for k in (1, 77, 126):
        code, *_ = optim.encode(np.full(65536, optim.M_GRID[k]), optim.M_GRID, every, False)
        assert np.all(code == k)
        x = 0.75 * optim.M_GRID[k] + 0.25 * optim.M_GRID[k + 1]
        code, *_ = optim.encode(np.full(65536, x), optim.M_GRID, every, False)
        assert abs(np.mean(code == k + 1) - 0.25) < 2e-5
    code, *_ = optim.encode(np.full(65536, 1e-9), optim.V_GRID, every, True)
    assert np.all(code == 1)


def test_hash_is_spread():
    e = np.arange(1 << 16, dtype=np.uint64)
    a, b = optim.element_bits(1, 1, e), optim.element_bits(1, 2, e)
    for x in (a, b, a ^ b):
        bits = (x[:, None] >> np.arange(32, dtype=np.uint64)) & np.uint64(1)
        # each bit's mean of 65536 fair draws is 0.5 within 5 standard deviations of 1/512
        assert np.all(np.abs(bits.mean(0) - 0.5) < 0.01)
    assert not np.array_equal(optim.element_bits(1, 1, e + np.uint64(1 << 32)), a)
