"""The operators around the QLoRA linears, as they are measured: cases, inputs, plain forms and exact values.

* ``norm_fwd`` / ``norm_bwd``: the residual update and the norms before and after a block,
      a = rms(y) (w_post + o)   (y itself without w_post)
      h' = res h + br gate a    (stored in h's type)
      n = rms(h') (w_pre + o)   (of the stored h')
  with gate absent, per channel [D], per token [M, 1] or whole [M, D]; backward for dn and dh'.
* ``rope``: rotary positions on the heads of a packed or separate q / k, either pair layout, part of the
  head, scaled for long contexts; ``inverse`` is the backward pass.
* ``adamw``: one optimizer step over many tensors, states in 32 or 8 bits, with the global norm's clip.

``own = False`` computes elementary torch operations in fp32 (angles, norms over all tensors and bias
corrections in 64 bits); ``own = True`` makes the calls of this repository's package.
"""

import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
MASK32 = 0xFFFFFFFF


# ------------------------------------------------------------------------------------ cases

def _norm(name, op, M, D, resid="bf16", weight="bf16", post=True, gate="none", pre=True, res=1.0, br=1.0,
          offset=0.0, dw=True, alone=False):
    """A residual update, or with `alone` the norm before a block by itself.  `resid`, `weight`: types of the residual stream and of w_pre, w_post and a
    broadcast gate (a whole gate is bf16, as a linear leaves it); dw: the gradients of weights and gate too."""
    return {"name": name, "op": op, "M": M, "D": D, "resid": resid, "weight": weight, "post": post, "gate": gate,
            "pre": pre, "res": res, "br": br, "offset": offset, "dw": dw, "alone": alone}


def _rope(name, M, hq, hk, hv, hd, rd, interleaved=False, kind="none", inverse=False, inplace=True, far=0,
          base=10000.0, dtype="bf16", separate=False):
    """Rotary positions: hq + hk heads of hd elements rotated in their first rd, hv more columns of heads in
    the packed row left alone; `separate`: q and k are two tensors.  `far`: the positions' offset."""
    return {"name": name, "op": "rope", "M": M, "hq": hq, "hk": hk, "hv": hv, "hd": hd, "rd": rd,
            "interleaved": interleaved, "kind": kind, "inverse": inverse, "inplace": inplace, "far": far,
            "base": base, "dtype": dtype, "separate": separate}


def _adamw(name, layers, shapes, r, bits, param="master", grad="f32", clip=0.3, wd=0.01, ratio=1.0, t=100):
    """Adapters A [r, K] and B [N, r] of `layers` times the linears in `shapes` ("K:N,K:N"), plus, for
    "ragged", tensors of every odd size.  param: "master" (bf16 with an fp32 master copy), "f32", or "bf16"
    (no master, stochastic rounding); ratio: B's learning rate over A's; t: steps taken before."""
    return {"name": name, "op": "adamw", "layers": layers, "shapes": shapes, "r": r, "bits": bits, "param": param,
            "grad": grad, "clip": clip, "wd": wd, "ratio": ratio, "t": t}


# The adapted linears of a Llama-3-8B block (q, k, v, o, gate, up, down), as the benchmark's workloads have them.
BLOCK_8B = "4096:4096,4096:1024,4096:1024,4096:4096,4096:14336,4096:14336,14336:4096"


def listed():
    return [
        # One token of a decoder with pre-norms only: residual add and the next norm, where latency counts.
        _norm("norm fwd one token", "norm_fwd", 1, 4096, post=False),
        # A training batch of the 8B workloads, norms on both sides of the block, a gate per channel.
        _norm("norm fwd 4096 tokens", "norm_fwd", 4096, 4096, gate="channel", res=1.0, br=0.7),
        # A ragged batch with an fp32 residual stream, zero-centred fp32 weights and a whole gate; odd width.
        _norm("norm fwd ragged f32", "norm_fwd", 1531, 2051, resid="f32", weight="f32", gate="full", offset=1.0,
              res=0.5),
        # The backward of the training batch, with the gradients of both weights and of the gate.
        _norm("norm bwd 4096 tokens", "norm_bwd", 4096, 4096, gate="channel", br=0.7),
        # The largest: long batch at the 70B width, pre-norm only, weights frozen as QLoRA keeps them.
        _norm("norm bwd 16384 x 8192", "norm_bwd", 16384, 8192, post=False, dw=False),
        # A short ragged batch with an fp32 residual stream and a gate per token.
        _norm("norm bwd short f32", "norm_bwd", 203, 1000, resid="f32", weight="f32", gate="token"),
        # Sixteen sequences, one token each, far into a long context.
        _rope("rope 16 tokens far", 16, 32, 8, 8, 128, 128, kind="bands", far=120000, base=500000.0),
        # The packed q/k/v output of the 8B workload, rotated in place.
        _rope("rope qkv 4096 tokens", 4096, 32, 8, 8, 128, 128, base=500000.0),
        # The backward of a long batch with separate q and k, interleaved pairs in half of each head, ramp scaling.
        _rope("rope bwd partial", 16384, 40, 40, 0, 80, 40, interleaved=True, kind="ramp", inverse=True,
              inplace=False, separate=True),
        # One block's adapters: fourteen small tensors, 32-bit states, the clip of the QLoRA recipe.
        _adamw("adamw one block", 1, BLOCK_8B, 16, 32),
        # All adapters of the 8B model at r = 16, 42 M parameters in 448 tensors, states in 8 bits.
        _adamw("adamw 8b states in 8", 32, BLOCK_8B, 16, 8, ratio=16.0),
        # The same, rank 64 on the attention's linears, fp32 parameters and states, no clip.
        _adamw("adamw attention r64", 32, "4096:4096,4096:1024,4096:1024,4096:4096", 64, 32, param="f32", clip=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_fwd", "norm_bwd", "norm_bwd", "rope", "rope", "rope", "adamw", "adamw"])
    if op in ("norm_fwd", "norm_bwd"):
        D = _log(rng, 64, 16384)
        D = {0: D, 1: max(8, D // 8 * 8), 2: max(64, D // 64 * 64), 3: max(256, D // 256 * 256)}[rng.randrange(4)]
        M = max(1, min(_log(rng, 1, 16384), 16384 * 4096 // D))
        types, offset, dw = (rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "f32"])), rng.choice([0.0, 1.0]), \
            rng.random() < 0.7
        if rng.random() < 0.15:
            c = _norm("", op, M, D, *types, post=False, offset=offset, dw=dw, alone=True)
        else:
            c = _norm("", op, M, D, *types, rng.random() < 0.6, rng.choice(["none", "channel", "token", "full"]),
                      rng.random() < 0.85, rng.choice([1.0, 0.5]), rng.choice([1.0, 0.22]), offset, dw)
    elif op == "rope":
        hd = rng.choice([64, 80, 96, 128, 128, 192, 256])
        hk = rng.choice([1, 2, 4, 8, 8, 16])
        hq = hk * rng.choice([1, 2, 4, 8])
        rd = rng.choice([hd, hd, hd, hd // 2, hd // 4, 2 * rng.randint(1, hd // 2)])
        M = max(1, min(_log(rng, 1, 32768), (1 << 27) // (hd * (hq + 2 * hk))))
        separate = rng.random() < 0.4
        c = _rope("", M, hq, hk, 0 if separate else hk, hd, rd, rng.random() < 0.5,
                  rng.choice(["none", "linear", "base", "bands", "ramp"]), rng.random() < 0.4, rng.random() < 0.6,
                  rng.choice([0, 0, _log(rng, 1, 1000000)]), rng.choice([10000.0, 500000.0]),
                  rng.choice(["bf16", "bf16", "f32"]), separate)
    else:
        K, N, r = _log(rng, 64, 8192), _log(rng, 64, 16384), rng.choice([4, 8, 16, 32, 64])
        layers = max(1, min(_log(rng, 1, 64), 40_000_000 // (r * (K + N))))
        shapes = "%d:%d" % (K, N) + rng.choice(["", ",%d:%d" % (_log(rng, 1, 4096), _log(rng, 1, 4096)), ",ragged"])
        c = _adamw("", layers, shapes, r, rng.choice([8, 32]), rng.choice(["master", "master", "f32", "bf16"]),
                   rng.choice(["f32", "f32", "bf16"]), rng.choice([0.0, 0.3, 1.0]), rng.choice([0.0, 0.01, 0.1]),
                   rng.choice([1.0, 16.0]), _log(rng, 1, 100000))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs

def _dt(name):
    return {"bf16": BF16, "f32": F32}[name]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, std=1.0, dtype=F32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=F32).mul_(std).to(dtype)

    if case["op"] in ("norm_fwd", "norm_bwd"):
        return _prepare_norm(case, randn)
    if case["op"] == "rope":
        return _prepare_rope(case, randn)
    return _prepare_adamw(case, gen, randn)


def _prepare_norm(c, randn):
    M, D, R, W = c["M"], c["D"], _dt(c["resid"]), _dt(c["weight"])
    s = {"c": c, "eps": 1e-5}
    # A residual stream whose channels differ in size, as trained ones do.
    s["h"] = (randn(M, D) * torch.exp(randn(1, D, std=0.5))).to(R)
    s["y"] = None if c["alone"] else randn(M, D, std=0.8, dtype=BF16)
    weight = lambda std: (1.0 - c["offset"] + randn(D, std=std)).to(W)  # noqa: E731
    s["w_pre"] = weight(0.1) if c["pre"] else None
    s["w_post"] = weight(0.1) if c["post"] else None
    s["gate"] = {"none": lambda: None, "channel": lambda: randn(D, std=0.3, dtype=W),
                 "token": lambda: torch.sigmoid(randn(M, 1)).to(W),
                 "full": lambda: torch.sigmoid(randn(M, D)).to(BF16)}[c["gate"]]()
    s["res"], s["br"] = c["res"], c["br"]
    if c["op"] == "norm_bwd":
        # What the forward left: h', 1/rms of y and of h'.
        f = _norm_plain(s)
        s["h_out"], s["rstd_pre"], s["rstd_post"] = f["h"], f["rstd_pre"], f["rstd_post"]
        s["dn"] = randn(M, D, std=1e-2, dtype=BF16) if c["pre"] else None
        s["dh_out"] = randn(M, D, std=1e-2, dtype=R)
        del s["h"]
    return s


def _prepare_rope(c, randn):
    dt, rd = _dt(c["dtype"]), c["rd"]
    M, hd = c["M"], c["hd"]
    s = {"c": c}
    cols = (c["hq"] if c["separate"] else c["hq"] + c["hk"] + c["hv"]) * hd
    s["q"] = randn(M, cols, dtype=dt)
    s["k"] = randn(M, c["hk"] * hd, dtype=dt) if c["separate"] else None
    # Sequences of up to 2048 tokens one after the other, as a packed batch has them.
    s["pos"] = (torch.arange(M, device="cuda") % 2048 + c["far"]).to(torch.int32)
    scaling = {"none": None, "linear": {"kind": "linear", "factor": 4.0}, "base": {"kind": "base", "factor": 4.0},
               "bands": {"kind": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "original": 8192},
               "ramp": {"kind": "ramp", "factor": 16.0, "fast": 32.0, "slow": 1.0, "original": 4096}}[c["kind"]]
    s["freq"], s["mscale"] = _frequencies(rd, c["base"], scaling)
    if own:
        from nf4_base_lora_blockwise_b200 import block
        s["plan"] = block.rope_plan(hd, rotary_dim=rd, base=c["base"], scaling=scaling,
                                    interleaved=c["interleaved"], device="cuda")
    return s


def _frequencies(rd, base, scaling):
    """Radians per position of each pair, in 64 bits, and the factor on the rotated values."""
    i = torch.arange(0, rd, 2, dtype=F64, device="cuda")
    f = base ** (-i / rd)
    if scaling is None:
        return f, 1.0
    kind, factor = scaling["kind"], scaling["factor"]
    if kind == "linear":
        return f / factor, 1.0
    if kind == "base":  # the base grown so that the slowest pair is slowed by `factor`
        grown = base * factor ** (rd / (rd - 2.0)) if rd > 2 else base
        return grown ** (-i / rd), 1.0
    if kind == "bands":  # wavelengths over original/low slowed, under original/high kept, a blend between
        turns = scaling["original"] * f / (2 * math.pi)
        blend = ((turns - scaling["low"]) / (scaling["high"] - scaling["low"])).clamp(0, 1)
        return f * (blend + (1 - blend) / factor), 1.0
    # "ramp": pairs that turn over `fast` times in the original length kept, under `slow` times slowed
    pair = lambda turns: rd * math.log(scaling["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(pair(scaling["fast"])), 0), min(math.ceil(pair(scaling["slow"])), rd - 1)
    slow = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f * (1 - slow + slow / factor), 0.1 * math.log(factor) + 1.0


def _adapter_sizes(c):
    """[(number of elements, whether it is a B)] of the tensors, in order."""
    sizes = []
    for part in c["shapes"].split(","):
        if part == "ragged":
            sizes += [(n, k % 2 == 1) for k, n in enumerate((1, 7, 255, 256, 257, 4099, 1, 65537))]
        else:
            K, N = (int(x) for x in part.split(":"))
            sizes += [(c["r"] * K, False), (c["r"] * N, True)]
    return sizes * c["layers"]


def _prepare_adamw(c, gen, randn):
    sizes = _adapter_sizes(c)
    # Every tensor starts at a multiple of 256 elements of the flat buffers (zeros between tensors).
    starts, at = [], 0
    for n, _ in sizes:
        starts.append(at)
        at += -(-n // 256) * 256
    first = torch.tensor(starts, device="cuda")
    count = torch.tensor([n for n, _ in sizes], device="cuda")
    blocks = (count + 255) // 256
    live = torch.zeros(at, dtype=torch.bool, device="cuda")
    which = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), blocks)  # tensor of each block
    live = ((torch.arange(at, device="cuda") - first[which].repeat_interleave(256))
            < count[which].repeat_interleave(256))
    # Gradients whose size differs between blocks of channels, and moments that fit them.
    size = torch.exp(randn(at // 256, 1, std=1.0)) * 1e-3
    flat = lambda x: (x.reshape(-1) * live)  # noqa: E731
    grad = flat(randn(at // 256, 256) * size).to(_dt(c["grad"]))
    m = flat(randn(at // 256, 256, std=0.3) * size)
    v = flat((randn(at // 256, 256).square() * 0.5 + 0.5) * size.square())
    p32 = flat(randn(at // 256, 256, std=0.01))
    s = {"c": c, "grad": grad, "t": c["t"], "lr": 1e-4, "betas": (0.9, 0.999), "eps": 1e-8, "seed": 1234}
    is_b = torch.tensor([float(b) for _, b in sizes], device="cuda")[which].reshape(-1, 1)
    s["lr_scale"] = 1.0 + is_b * (c["ratio"] - 1.0)  # a column of one value a block
    if c["param"] == "f32":
        s["p32"], s["p16"] = p32, None
    else:
        s["p16"] = p32.to(BF16)
        s["p32"] = p32 if c["param"] == "master" else None
    if c["bits"] == 8:
        half = torch.full_like(grad, 32768, dtype=torch.int64)
        s["m"] = _encode_m(m.reshape(-1, 256), half.reshape(-1, 256))
        s["v"] = _encode_v(v.reshape(-1, 256), half.reshape(-1, 256))
    else:
        s["m"], s["v"] = m, v
    if own:
        from nf4_base_lora_blockwise_b200 import optim
        views = lambda x: [x[a:a + n] for a, (n, _) in zip(starts, sizes)] if x is not None else None  # noqa: E731
        lead = s["p32"] if c["param"] == "f32" else s["p16"]
        s["opt"] = optim.AdamW(views(lead), views(grad), masters=views(s["p32"]) if c["param"] == "master" else None,
                               bits=c["bits"], lr=s["lr"], betas=s["betas"], eps=s["eps"], weight_decay=c["wd"],
                               lr_scales=[c["ratio"] if b else 1.0 for _, b in sizes],
                               max_grad_norm=c["clip"] or None, seed=s["seed"], step=c["t"])
        if c["bits"] == 8:
            for name, (codes, scale) in (("m", s["m"]), ("v", s["v"])):
                getattr(s["opt"], name).copy_(codes.reshape(-1))
                getattr(s["opt"], name + "_scale").copy_(scale.reshape(-1))
        else:
            s["opt"].m.copy_(m)
            s["opt"].v.copy_(v)
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    op = s["c"]["op"]
    if op == "norm_fwd":
        if own:
            from nf4_base_lora_blockwise_b200 import block
            h, n, rstd_pre, rstd_post = block.residual_norm_forward(
                s["h"], s["y"], s["w_pre"], s["w_post"], s["gate"], eps=s["eps"], res_scale=s["res"],
                branch_scale=s["br"], weight_offset=s["c"]["offset"])
            return {"h": h, "n": n, "rstd_pre": rstd_pre, "rstd_post": rstd_post}
        return _norm_plain(s)
    if op == "norm_bwd":
        if own:
            from nf4_base_lora_blockwise_b200 import block
            dh, dy, dw_pre, dw_post, dgate = block.residual_norm_backward(
                s["dn"], s["dh_out"], s["h_out"], s["y"], s["rstd_pre"], s["rstd_post"], s["w_pre"], s["w_post"],
                s["gate"], res_scale=s["res"], branch_scale=s["br"], weight_offset=s["c"]["offset"],
                need_dw=s["c"]["dw"], need_dgate=s["c"]["dw"])
            return {"dh": dh, "dy": dy, "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}
        return _norm_bwd_plain(s)
    if op == "rope":
        c = s["c"]
        if own:
            from nf4_base_lora_blockwise_b200 import block
            heads = c["hq"] if c["separate"] else c["hq"] + c["hk"]
            out = block.rope(s["q"], s["pos"], s["plan"], n_heads=heads, k=s["k"], inverse=c["inverse"],
                             inplace=c["inplace"])
            return [out] if s["k"] is None else list(out)
        return _rope_plain(s)
    if own:
        opt = s["opt"]
        norm = opt.step()
        # The states of 8 bits as the values they stand for: five or ten bits times a scale, so bf16 holds them
        # to a fraction of their own step.
        m, v = opt.moments(BF16) if s["c"]["bits"] == 8 else (opt.m, opt.v)
        return {"p32": s["p32"], "p16": s["p16"], "m": m, "v": v, "norm": norm}
    return _adamw_plain(s)


# ------------------------------------------------------------------------------------ plain forms

def _norm_plain(s):
    c, h, y = s["c"], s["h"], s["y"]
    rstd_post = None
    h_out = h
    if y is not None:
        a = y.float()
        if s["w_post"] is not None:
            rstd_post = torch.rsqrt(a.square().mean(1, keepdim=True) + s["eps"])
            a = a * rstd_post * (s["w_post"].float() + c["offset"])
        if s["gate"] is not None:
            a = a * s["gate"].float()
        h_out = (h.float() * s["res"] + a * s["br"]).to(h.dtype)
    n = rstd_pre = None
    if s["w_pre"] is not None:
        x = h_out.float()
        rstd_pre = torch.rsqrt(x.square().mean(1, keepdim=True) + s["eps"])
        n = (x * rstd_pre * (s["w_pre"].float() + c["offset"])).to(BF16)
    flat = lambda r: None if r is None else r.reshape(-1)  # noqa: E731
    return {"h": h_out, "n": n, "rstd_pre": flat(rstd_pre), "rstd_post": flat(rstd_post)}


def _norm_bwd_plain(s):
    c, gate = s["c"], s["gate"]
    G = s["dh_out"].float()
    dw_pre = dw_post = dgate = None
    if s["w_pre"] is not None:
        r = s["rstd_pre"][:, None]
        x, dn = s["h_out"].float() * r, s["dn"].float()
        u = dn * (s["w_pre"].float() + c["offset"])
        G = G + r * (u - x * (u * x).mean(1, keepdim=True))
        dw_pre = (dn * x).sum(0)
    dh = (G * s["res"]).to(s["dh_out"].dtype)
    if s["y"] is None:
        return {"dh": dh, "dy": None, "dw_pre": dw_pre if c["dw"] else None, "dw_post": None, "dgate": None}
    y = s["y"].float()
    E = G * s["br"]
    a = y
    if s["w_post"] is not None:
        r = s["rstd_post"][:, None]
        x = y * r
        a = x * (s["w_post"].float() + c["offset"])
    if gate is not None:
        dgate = E * a
        dgate = (dgate.sum(0) if gate.dim() == 1 else dgate.sum(1, keepdim=True) if gate.shape[1] == 1
                 else dgate.to(gate.dtype))
        E = E * gate.float()
    dy = E
    if s["w_post"] is not None:
        dw_post = (E * x).sum(0)
        t = E * (s["w_post"].float() + c["offset"])
        dy = r * (t - x * (t * x).mean(1, keepdim=True))
    if not c["dw"]:
        dw_pre = dw_post = dgate = None
    return {"dh": dh, "dy": dy.to(BF16), "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}


def _rope_plain(s):
    c, rd, hd = s["c"], s["c"]["rd"], s["c"]["hd"]
    angle = s["pos"].to(F64)[:, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["mscale"]).float()[:, None], (torch.sin(angle) * s["mscale"]).float()[:, None]
    if c["inverse"]:
        sin = -sin
    outs = []
    for x, heads in ((s["q"], c["hq"] if c["separate"] else c["hq"] + c["hk"]), (s["k"], c["hk"])):
        if x is None:
            continue
        every = x.view(x.shape[0], -1, hd)
        turned = every[:, :heads, :rd].float()
        a, b = (turned[..., 0::2], turned[..., 1::2]) if c["interleaved"] else turned.chunk(2, -1)
        pair = (a * cos - b * sin, b * cos + a * sin)
        new = (torch.stack(pair, -1).flatten(-2) if c["interleaved"] else torch.cat(pair, -1)).to(x.dtype)
        if not c["inplace"]:
            every = every[:, :heads].clone()
            x = every.view(x.shape[0], heads * hd)
        every[:, :heads, :rd] = new
        outs.append(x)
    return outs


def _hash(seed, t, n):
    """32 random bits for each of n elements: an integer hash of (seed, step, element) by multiplications and
    shifted exclusive ors, modulo 2^32."""
    def mix(x):
        x = ((x ^ (x >> 16)) * 0x7FEB352D) & MASK32
        x = ((x ^ (x >> 15)) * 0x846CA68B) & MASK32
        return x ^ (x >> 16)
    word = mix((mix(seed & MASK32) + t) & MASK32)
    e = torch.arange(n, dtype=torch.int64, device="cuda")
    return mix(((e & MASK32) ^ mix_high(e >> 32)) + word & MASK32)


def mix_high(high):
    return (high * 0x9E3779B1) & MASK32


def _encode_m(m, r16):
    """Blocks of 256: sign, 4 bits of exponent and 3 of mantissa of m over its block's largest; rounded up
    where the dropped bits and r16 (0..65535) carry."""
    scale = m.abs().amax(1, keepdim=True)
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    x = m.abs() * torch.where(scale > 0, 1.0 / scale, scale)
    code = ((x.view(torch.int32).to(torch.int64) + (r16 << 4)) >> 20) - 889
    low = x < 1.25 * 2.0 ** -16
    code = torch.where(low, (r16.float() * (1.25 * 2.0 ** -32) < x).to(torch.int64), code.clamp(max=127))
    code = torch.where(m < 0, code + 128, code)
    return torch.where(scale > 0, code, torch.zeros_like(code)).to(torch.uint8), scale


def _decode_m(code, scale):
    mag = (code & 127).to(torch.int32)
    x = torch.where(mag > 0, ((mag + 889) << 20).view(F32), torch.zeros_like(scale))
    return torch.where(code > 127, -x, x) * scale


def _encode_v(v, r16):
    """Blocks of 256: 4 bits of exponent and 4 of mantissa of sqrt(v) over its block's largest; never 0 for a
    v above 0."""
    root = torch.sqrt(v)
    scale = root.amax(1, keepdim=True)
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    x = root * torch.where(scale > 0, 1.0 / scale, scale)
    code = ((x.view(torch.int32).to(torch.int64) + (r16 << 3)) >> 19) - 1777
    code = torch.where(x > 0, code.clamp(1, 255), torch.zeros_like(code))
    return torch.where(scale > 0, code, torch.zeros_like(code)).to(torch.uint8), scale


def _decode_v(code, scale):
    c = code.to(torch.int32)
    root = torch.where(c > 0, ((c + 1777) << 19).view(F32), torch.zeros_like(scale)) * scale
    return root * root


def _adamw_plain(s):
    c, (b1, b2) = s["c"], s["betas"]
    s["t"] += 1
    t, norm, factor = s["t"], None, 1.0
    if c["clip"]:
        norm = s["grad"].to(F64).square().sum().sqrt()
        factor = torch.clamp(c["clip"] / (norm + 1e-6), max=1.0).float()
        norm = norm.float().reshape(1)
    g = (s["grad"].float() * factor).reshape(-1, 256)
    if c["bits"] == 8:
        m, v = _decode_m(*s["m"]), _decode_v(*s["v"])
    else:
        m, v = s["m"].view(-1, 256), s["v"].view(-1, 256)
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    step = m / (torch.sqrt(v) * (1 / math.sqrt(1 - b2 ** t)) + s["eps"])
    rate = s["lr"] * s["lr_scale"]
    p = (s["p32"] if s["p32"] is not None else s["p16"].float()).view(-1, 256)
    p = p * (1 - rate * c["wd"]) - rate * (1 / (1 - b1 ** t)) * step
    if s["p32"] is not None:
        s["p32"].copy_(p.view(-1))
    bits = _hash(s["seed"], t, p.numel()).view(-1, 256) if c["bits"] == 8 or c["param"] == "bf16" else None
    if c["param"] == "master":
        s["p16"].copy_(p.view(-1))
    elif c["param"] == "bf16":  # rounded up where the dropped bits and 16 random ones carry
        extra = _hash(s["seed"] ^ 0x55555555, t, p.numel()).view(-1, 256) & 0xFFFF
        word = (p.view(torch.int32).to(torch.int64) + extra) >> 16 << 16
        s["p16"].copy_(word.to(torch.int32).view(F32).view(-1))
    if c["bits"] == 8:
        s["m"], s["v"] = _encode_m(m, bits & 0xFFFF), _encode_v(v, bits >> 16)
        out_m, out_v = _decode_m(*s["m"]).view(-1).to(BF16), _decode_v(*s["v"]).view(-1).to(BF16)
    else:
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
        out_m, out_v = s["m"], s["v"]
    return {"p32": s["p32"], "p16": s["p16"], "m": out_m, "v": out_v, "norm": norm}


# ------------------------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] in ("norm_fwd", "norm_bwd"):
        n, R = c["M"] * c["D"], 4 if c["resid"] == "f32" else 2
        W = 4 if c["weight"] == "f32" else 2
        gate = {"none": 0, "channel": c["D"] * W, "token": c["M"] * W, "full": n * 2}[c["gate"]]
        small = gate + c["D"] * W * (c["pre"] + c["post"]) + 4 * c["M"] * (c["pre"] + c["post"])
        if c["op"] == "norm_fwd":
            return {"bytes": n * (R + (2 + R) * (not c["alone"]) + 2 * c["pre"]) + small,
                    "flops": n * (6 + 4 * c["post"])}
        dgate = 0 if c["gate"] == "none" or not c["dw"] else \
            {"channel": 4 * c["D"], "token": 4 * c["M"], "full": n * 2}[c["gate"]]
        whole_y = c["post"] or (c["gate"] != "none" and c["dw"])  # y is needed for the post-norm or the gate alone
        read = R + (2 + R) * c["pre"] + 2 * whole_y
        return {"bytes": n * (read + R + 2 * (not c["alone"])) + small + dgate + 4 * c["D"] * c["dw"] * (c["pre"] + c["post"]),
                "flops": n * (10 + 8 * c["post"])}
    if c["op"] == "rope":
        e = 4 if c["dtype"] == "f32" else 2
        heads = c["hq"] + c["hk"]
        touched = c["rd"] if c["inplace"] else c["hd"]  # the rest of each head is copied when out of place
        return {"bytes": 2 * c["M"] * heads * touched * e + 4 * c["M"], "flops": 3 * c["M"] * heads * c["rd"]}
    n = sum(k for k, _ in _adapter_sizes(c))
    param = {"master": 10, "f32": 8, "bf16": 4}[c["param"]]
    state = 16 if c["bits"] == 32 else 4 + 4 + 16 / 256  # codes read and written, the values returned, the scales
    return {"bytes": n * (param + state + (4 if c["grad"] == "f32" else 2)), "flops": n * (15 + 2 * bool(c["clip"]))}


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_fwd":
        return _exact_norm(s)
    if case["op"] == "norm_bwd":
        return _exact_norm_bwd(s)
    return _exact_rope(s) if case["op"] == "rope" else _exact_adamw(s)


def _d(x):
    return None if x is None else x.to(F64)


def _unit(x, eps):
    """x over its root mean square, and one over that."""
    r = (torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / x.shape[1] + eps) ** -0.5
    return x * r, r.flatten()


def _exact_norm(s):
    c, h, y = s["c"], _d(s["h"]), _d(s["y"])
    rstd_post = None
    if y is not None:
        if s["w_post"] is not None:
            y, rstd_post = _unit(y, s["eps"])
            y = y * (_d(s["w_post"]) + c["offset"])
        h = s["res"] * h + s["br"] * (y if s["gate"] is None else y * _d(s["gate"]))
    if s["w_pre"] is None:
        return {"h": h, "n": None, "rstd_pre": None, "rstd_post": rstd_post}
    x, rstd_pre = _unit(h.to(s["h"].dtype).to(F64), s["eps"])  # the norm is defined on what is stored
    return {"h": h, "n": x * (_d(s["w_pre"]) + c["offset"]), "rstd_pre": rstd_pre, "rstd_post": rstd_post}


def _unit_bwd(x, r, w, d):
    """Gradients of w x r, r one over the rms of x, for the upstream gradient d."""
    z = d * w
    inner = torch.linalg.vecdot(z, x)[:, None] / x.shape[1]
    return r * z - x * (r ** 3 * inner), (d * x * r).sum(0)


def _exact_norm_bwd(s):
    c = s["c"]
    total = _d(s["dh_out"])
    dw_pre = dw_post = dgate = None
    if s["w_pre"] is not None:
        d, dw_pre = _unit_bwd(_d(s["h_out"]), _d(s["rstd_pre"])[:, None], _d(s["w_pre"]) + c["offset"], _d(s["dn"]))
        total = total + d
    if s["y"] is None:
        return {"dh": s["res"] * total, "dy": None, "dw_pre": dw_pre if c["dw"] else None, "dw_post": None,
                "dgate": None}
    y = _d(s["y"])
    branch = s["br"] * total
    w = None if s["w_post"] is None else _d(s["w_post"]) + c["offset"]
    a = y if w is None else y * _d(s["rstd_post"])[:, None] * w
    if s["gate"] is not None:
        along = {"channel": (0, False), "token": (1, True)}.get(c["gate"])
        dgate = branch * a
        dgate = dgate if along is None else dgate.sum(along[0], keepdim=along[1])
        branch = branch * _d(s["gate"])
    if w is not None:
        branch, dw_post = _unit_bwd(y, _d(s["rstd_post"])[:, None], w, branch)
    if not c["dw"]:
        dw_pre = dw_post = dgate = None
    return {"dh": s["res"] * total, "dy": branch, "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}


def _exact_rope(s):
    c, hd, rd = s["c"], s["c"]["hd"], s["c"]["rd"]
    outs = []
    turn = torch.polar(torch.full_like(s["freq"], s["mscale"]).expand(c["M"], -1).contiguous(),
                       (s["pos"].to(F64)[:, None] * s["freq"]) * (-1.0 if c["inverse"] else 1.0))[:, None]
    for x, heads in ((s["q"], c["hq"] if c["separate"] else c["hq"] + c["hk"]), (s["k"], c["hk"])):
        if x is None:
            continue
        w = _d(x).view(c["M"], -1, hd)
        first, second = (slice(0, rd, 2), slice(1, rd, 2)) if c["interleaved"] else (slice(0, rd // 2),
                                                                                    slice(rd // 2, rd))
        z = torch.complex(w[:, :heads, first].contiguous(), w[:, :heads, second].contiguous()) * turn
        w[:, :heads, first] = z.real
        w[:, :heads, second] = z.imag
        outs.append((w if c["inplace"] else w[:, :heads]).reshape(c["M"], -1))
    return outs


def _grid(x, mantissa, r16):
    """x in [0, 1] on the grid of floats with `mantissa` bits, rounded up where its place between two of them
    and r16 / 65536 reach the next one."""
    e = torch.floor(torch.log2(x.clamp(min=2.0 ** -60)))
    place = x * torch.exp2(mantissa - e)
    return torch.floor(place + r16.to(F64) / 65536) * torch.exp2(e - mantissa)


def _exact_adamw(s):
    c, (b1, b2), t = s["c"], s["betas"], s["t"] + 1
    g = _d(s["grad"]).view(-1, 256)
    norm = torch.linalg.vector_norm(g)
    if c["clip"]:
        g = g * min(1.0, c["clip"] / (float(norm) + 1e-6))
    m, v = (_decode_m(*s["m"]), _decode_v(*s["v"])) if c["bits"] == 8 else (s["m"], s["v"])
    m, v = torch.lerp(g, _d(m).view(-1, 256), b1), torch.lerp(g * g, _d(v).view(-1, 256), b2)
    p = _d(s["p32"] if s["p32"] is not None else s["p16"]).view(-1, 256)
    rate = s["lr"] * _d(s["lr_scale"])
    p = p - rate * (c["wd"] * p + (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + s["eps"]))
    p32 = None if s["p32"] is None else p.flatten()
    # Without a master copy the parameter is rounded at random: its values have an exact form before that only.
    p16 = p.flatten() if s["p16"] is not None else None
    if c["bits"] == 8:
        bits = _hash(s["seed"], t, p.numel()).view(-1, 256)
        top, root = m.abs().amax(1, keepdim=True), v.sqrt()
        x, r16 = m.abs() / top.clamp(min=2.0 ** -126), bits & 0xFFFF
        least = 1.25 * 2.0 ** -16
        x = torch.where(x < least, least * (r16.to(F64) / 65536 * least < x), _grid(x, 3, r16).clamp(max=1.0))
        m = torch.sign(m) * x * top
        top = root.amax(1, keepdim=True)
        x = root / top.clamp(min=2.0 ** -126)
        v = torch.where(x > 0, _grid(x, 4, bits >> 16).clamp(1.125 * 2.0 ** -16, 1.0) * top, 0.0).square()
    return {"p32": p32, "p16": p16, "m": m.flatten(), "v": v.flatten(), "norm": norm.view(1) if c["clip"] else None}
