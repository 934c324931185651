"""Operators around a DoRA module in training and serving, as cases to be measured.

Three families, each in its plain form (elementary torch operations, 32 bits or
more, rounded once) and, where ``own`` is true, as the library's calls:

* ``block``, ``block_backward``: the norms on both sides of a residual addition:
  the block's output normed, gated and scaled, added to the scaled residual
  stream, and the sum normed for the next block; and its gradients.
* ``weight4``, ``linear4``: a merged weight in 4 bits (e2m1 codes, one scale for
  each group of columns): made and restored, and its linear layer.
* ``muon``: matrices orthogonalised by Newton-Schulz products, alone or as the
  step of an optimiser that moves the adapters' factors along the orthogonalised
  momentum.

4-bit values are returned as the values they stand for.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
TINY = 1e-7  # added to the norm that a matrix is divided by
STEPS, QUINTIC = 5, (3.4445, -4.7750, 2.0315)
MU, DECAY, LR = 0.95, 0.1, 0.02
LEAST, MOST = 2.0 ** -125, 1.3125 * 2.0 ** 125  # the scales of 4-bit groups


def listed():
    return [
        # one decoded token behind a block of a square 4096 module: latency
        {"name": "block_token", "op": "block", "T": 1, "d": 4096, "dtype": "bf16", "gate_rows": 1,
         "post": True},
        # a training batch or a prompt at the training module's input width, a gate a channel
        {"name": "block_train", "op": "block", "T": 8192, "d": 8192, "dtype": "bf16",
         "gate_rows": 8192, "post": True},
        # its backward pass
        {"name": "block_backward_train", "op": "block_backward", "T": 8192, "d": 8192,
         "dtype": "bf16", "gate_rows": 8192, "post": True},
        # eleven sequences of 47 tokens with a gate vector each, odd width
        {"name": "block_backward_odd", "op": "block_backward", "T": 517, "d": 2047,
         "dtype": "f32", "gate_rows": 47, "post": True},
        # the training module's merged weight to 4 bits and back
        {"name": "weight4_train", "op": "weight4", "rows": 28672, "d": 8192, "dtype": "bf16",
         "group": 128},
        # a weight whose sizes are multiples of nothing
        {"name": "weight4_odd", "op": "weight4", "rows": 2051, "d": 1029, "dtype": "f32",
         "group": 32},
        # one decoded token through the training module's merged weight: latency
        {"name": "linear4_token", "op": "linear4", "T": 1, "d_in": 8192, "d_out": 28672,
         "dtype": "bf16", "group": 128},
        # a decoding batch through an 8B-class decoder's MLP up projection
        {"name": "linear4_batch", "op": "linear4", "T": 24, "d_in": 4096, "d_out": 14336,
         "dtype": "bf16", "group": 64},
        # a prompt through a square 8192 module's merged weight
        {"name": "linear4_prompt", "op": "linear4", "T": 2048, "d_in": 8192, "d_out": 8192,
         "dtype": "bf16", "group": 128},
        # one factor of odd sizes, without the optimiser around it
        {"name": "orthogonal_odd", "op": "muon", "step": False, "rows": 37, "cols": 1027,
         "dtype": "f32"},
        # the training module's two factors, rank 384
        {"name": "muon_train", "op": "muon", "step": True, "d_in": 8192, "d_out": 28672, "r": 384,
         "modules": 1, "dtype": "bf16"},
        # the fourteen modules of two decoder layers at rank 64: many small factors
        {"name": "muon_layers", "op": "muon", "step": True, "d_in": 4096, "d_out": 4096,
         "r": 64, "modules": 14, "dtype": "bf16"},
    ]


def _size(rng, lo, hi, step=1):
    """Spread over the logarithm of [lo, hi]; a multiple of `step`, or odd."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    v = max(step, v // step * step) if rng.random() < 0.6 else v | 1
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["block", "block_backward", "weight4", "linear4", "muon"])
    c = {"op": op, "dtype": "bf16" if rng.random() < 0.7 else "f32"}
    if op in ("block", "block_backward"):
        c["post"] = rng.random() < 0.8
        c["d"] = _size(rng, 256, 14336, 64)
        most = 8192 * 8192 // c["d"] // (2 if c["dtype"] == "f32" else 1)
        kind = rng.choice(["none", "channel", "token", "sequence"])
        if kind == "sequence":  # sequences of one length, a gate vector each
            c["gate_rows"] = _size(rng, 2, 256)
            c["T"] = c["gate_rows"] * rng.randint(1, max(1, min(64, most // c["gate_rows"])))
        else:
            c["T"] = _size(rng, 1, min(8192, most), 16)
            c["gate_rows"] = {"none": 0, "channel": c["T"], "token": 1}[kind]
    elif op == "weight4":
        c["rows"] = _size(rng, 256, 14336, 64)
        c["d"] = _size(rng, 256, 8192, 64)
        c["group"] = rng.choice([32, 64, 128, 256])
    elif op == "linear4":
        c["d_in"] = _size(rng, 256, 8192, 64)
        c["d_out"] = _size(rng, 256, 28672 if c["dtype"] == "bf16" else 8192, 64)
        c["T"] = _size(rng, 1, 64) if rng.random() < 0.75 else _size(rng, 64, 512, 16)
        c["group"] = rng.choice([32, 64, 128, 256])
    elif rng.random() < 0.3:
        c["step"] = False
        short, long = _size(rng, 8, 384, 8), _size(rng, 256, 8192, 64)
        c["rows"], c["cols"] = (short, long) if rng.random() < 0.5 else (long, short)
    else:
        c["step"] = True
        c["d_in"] = _size(rng, 256, 8192, 64)
        c["d_out"] = _size(rng, 256, 8192, 64)
        c["r"] = _size(rng, 8, 384, 8)
        c["modules"] = rng.choice([1, 2, 3])
    return c


# ------------------------------------------------------------------- inputs
def _to4(v, group):
    """Packed e2m1 codes and scales of the rows of v (float), as a program has
    them in hand: two codes a byte, the even column in the low half, rows of
    whole groups; a scale is max / 6 with six significant bits, in bf16."""
    rows, d = v.shape
    n = -(-d // group)
    if n * group != d:
        v = torch.nn.functional.pad(v, (0, n * group - d))
    v = v.view(rows, n, group)
    m, e = torch.frexp(v.abs().amax(dim=2) / 6)
    scale = torch.ldexp(torch.round(m * 64) / 64, e).clamp_min(2.0 ** -100)
    t = v.abs() / scale[:, :, None]
    code = torch.bucketize(t, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0],
                                           device=v.device)).to(torch.uint8)
    code = (code | ((v < 0).to(torch.uint8) << 3)).view(rows, n * group)
    return (code[:, ::2] | (code[:, 1::2] << 4)).contiguous(), scale.to(torch.bfloat16)


def _acts(gen, T, d, dev):
    """Activations: unit normal, with one channel in 256 twelve times larger."""
    x = torch.randn(T, d, generator=gen, device=dev)
    big = torch.randperm(d, generator=gen, device=dev)[: max(1, d // 256)]
    x[:, big] *= 12.0
    return x


def _gradient(gen, rows, cols, dev):
    """A factor's gradient: singular values that fall off over a floor of noise."""
    k = min(rows, cols)
    left = torch.randn(rows, k, generator=gen, device=dev)
    right = torch.randn(k, cols, generator=gen, device=dev)
    fall = 1.0 / torch.arange(1, k + 1, device=dev, dtype=torch.float32).sqrt()
    g = (left * fall) @ right + 0.1 * torch.randn(rows, cols, generator=gen, device=dev)
    return g * 1e-3


def _factors(case):
    """The shapes of A [r, d_in] and B [d_out, r] of every module."""
    return [(case["r"], case["d_in"]), (case["d_out"], case["r"])] * case["modules"]


def prepare(case, seed):
    dev = "cuda:0"
    gen = torch.Generator(dev).manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    st = {"case": case, "out": {}}

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * std

    if op in ("block", "block_backward"):
        T, d = case["T"], case["d"]
        st["x"] = normal(T, d, std=0.5).to(dt)
        st["res"] = _acts(gen, T, d, dev).to(dt)
        st["w_pre"] = (1 + normal(d, std=0.1)).to(dt)
        st["w_post"] = (1 + normal(d, std=0.1)).to(dt) if case["post"] else None
        rows = case["gate_rows"]
        st["gate"] = normal(T // rows, d, std=0.3).to(dt) if rows else None
        if op == "block_backward":  # what the forward pass kept, and two gradients
            kept = _plain_block(st)
            st["h"] = kept["h"]
            st["r_pre"] = 1 / torch.sqrt(kept["h"].double().square().mean(1) + EPS).float()
            st["r_post"] = 1 / torch.sqrt(st["x"].double().square().mean(1) + EPS).float() \
                if case["post"] else None
            del st["res"]
            st["dy"] = normal(T, d).to(dt)
            st["dh"] = normal(T, d).to(dt)
    elif op == "weight4":
        st["W"] = normal(case["rows"], case["d"], std=case["d"] ** -0.5).to(dt)
    elif op == "linear4":
        st["x"] = _acts(gen, case["T"], case["d_in"], dev).to(dt)
        W = normal(case["d_out"], case["d_in"], std=case["d_in"] ** -0.5)
        st["codes"], st["scale"] = _to4(W, case["group"])
    elif not case["step"]:
        st["U"] = _gradient(gen, case["rows"], case["cols"], dev).to(dt)
    else:
        shapes = _factors(case)
        st["p"] = [normal(*s, std=s[1] ** -0.5).to(dt) for s in shapes]
        st["g"] = [_gradient(gen, *s, dev).to(dt) for s in shapes]
        st["M"] = [_gradient(gen, *s, dev) * 4 for s in shapes]
    return st


RESIDUAL, BRANCH = 0.9, 1.25  # the residual's scale and the block's


# --------------------------------------------------------------- plain forms
def _plain_block(st):
    c = st["case"]
    dt = DTYPES[c["dtype"]]
    u = st["x"].float()
    if c["post"]:
        u = u / torch.sqrt(u.square().mean(dim=1, keepdim=True) + EPS) * st["w_post"].float()
    if c["gate_rows"]:
        u = u * st["gate"].float().repeat_interleave(c["gate_rows"], dim=0)
    h = (RESIDUAL * st["res"].float() + BRANCH * u).to(dt)
    hf = h.float()
    r = 1 / torch.sqrt(hf.square().mean(dim=1, keepdim=True) + EPS)
    return {"h": h, "y": (hf * r * st["w_pre"].float()).to(dt)}


def _plain_block_backward(st):
    c = st["case"]
    dt, d = DTYPES[c["dtype"]], c["d"]
    dy, r2 = st["dy"].float(), st["r_pre"][:, None]
    hhat = st["h"].float() * r2
    wdy = st["w_pre"].float() * dy
    dh = st["dh"].float() + r2 * (wdy - hhat * (wdy * hhat).mean(1, keepdim=True))
    out = {"dresidual": (RESIDUAL * dh).to(dt), "dw_pre": (dy * hhat).sum(0)}
    x, r1, w1 = st["x"].float(), 1.0, 1.0
    if c["post"]:
        r1, w1 = st["r_post"][:, None], st["w_post"].float()
    xhat = x * r1
    du = BRANCH * dh
    if c["gate_rows"]:
        out["dgate"] = (du * (xhat * w1)).view(-1, c["gate_rows"], d).sum(1).to(dt)
        du = du * st["gate"].float().repeat_interleave(c["gate_rows"], dim=0)
    if c["post"]:
        out["dw_post"] = (du * xhat).sum(0)
        du = w1 * du
        du = r1 * (du - xhat * (du * xhat).mean(1, keepdim=True))
    out["dx"] = du.to(dt)
    return out


def _six_bits(v):
    """Positive floats rounded to six significant bits, ties to even."""
    u = v.view(torch.int32)
    return ((u + 0x1FFFF + ((u >> 18) & 1)) & ~0x3FFFF).view(torch.float32)


def _plain_weight4(W, group):
    """What 4-bit codes and scales stand for, in 32 bits (no rounding: a scale's
    six bits times a code's two are bf16 numbers), the rounding decided in 64."""
    rows, d = W.shape
    n = -(-d // group)
    v = W.float()
    if n * group != d:
        v = torch.nn.functional.pad(v, (0, n * group - d))
    v = v.view(rows, n, group)
    top = v.abs().amax(dim=2)
    scale = torch.where(top > 0, _six_bits(top / 6).clamp(LEAST, MOST), 0.0)
    t = v.abs().double() / torch.where(top > 0, scale, 1.0)[:, :, None]
    step = torch.where(t < 2, 0.5, torch.where(t < 4, 1.0, 2.0))
    t = (torch.round(t / step) * step).clamp_max(6).float()
    values = torch.sign(v) * t * scale[:, :, None]
    return values.reshape(rows, n * group)[:, :d], scale


def _restored4(codes, scale, d, group):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=2).view(codes.shape[0], -1)
    v = table[(c & 7).int()] * torch.where(c >= 8, -1.0, 1.0)
    return (v.view(v.shape[0], -1, group) * scale.float()[:, :, None]).view(v.shape)[:, :d]


def _plain_orthogonal(U):
    """Newton-Schulz steps on U / norm in 32 bits, on the shorter side."""
    a, b, c = QUINTIC
    X = U.float()
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    X = X / (X.square().sum().sqrt() + TINY)
    for _ in range(STEPS):
        G = X @ X.T
        X = a * X + (b * G + c * (G @ G)) @ X
    return X.T if tall else X


def _reach(shape):
    """The size of a step: that of the update's elements is brought to 0.2."""
    return 0.2 * max(shape) ** 0.5


def _plain(st):
    c = st["case"]
    op, dt = c["op"], DTYPES[c["dtype"]]
    if op == "block":
        return _plain_block(st)
    if op == "block_backward":
        return _plain_block_backward(st)
    if op == "weight4":
        values, scale = _plain_weight4(st["W"], c["group"])
        return {"values": values.to(dt), "scale": scale.to(torch.bfloat16)}
    if op == "linear4":
        W = _restored4(st["codes"], st["scale"], c["d_in"], c["group"])
        return (st["x"].float() @ W.T).to(dt)
    if not c["step"]:
        return _plain_orthogonal(st["U"]).to(dt).contiguous()
    out = {}
    for k, (p, g, M) in enumerate(zip(st["p"], st["g"], st["M"])):
        new = MU * M + g.float()
        O = _plain_orthogonal(g.float() + MU * new)
        q = p.float()
        out[f"p{k}"] = (q - LR * (DECAY * q + _reach(p.shape) * O)).to(dt)
        out[f"M{k}"] = new
    return out


# ------------------------------------------------------- the library's calls
def _kept(st, name, make):
    """A buffer that the program keeps from call to call."""
    if name not in st["out"]:
        st["out"][name] = make()
    return st["out"][name]


def _own(st):
    from dora_adapter_amd import dora as D

    c = st["case"]
    op, dt = c["op"], DTYPES[c["dtype"]]

    def empty(name, *shape, dtype=dt):
        return _kept(st, name, lambda: torch.empty(*shape, dtype=dtype, device="cuda:0"))

    def space(nbytes):
        return empty("ws", max(nbytes, 16), dtype=torch.uint8)

    lib_dt = D.DORA_BF16 if dt == torch.bfloat16 else D.DORA_F32
    if op in ("block", "block_backward"):
        T, d = c["T"], c["d"]
        kw = {"w_post": st["w_post"], "gate": st["gate"], "residual_scale": RESIDUAL,
              "branch_scale": BRANCH}
        if op == "block":
            out = {"h": empty("h", T, d), "y": empty("y", T, d)}
            return D.dora_block_norm(st["x"], st["res"], st["w_pre"], eps=EPS, out=out, **kw)
        out = {"dresidual": empty("dresidual", T, d),
               "dw_pre": empty("dw_pre", d, dtype=torch.float32)}
        if c["gate_rows"]:
            out["dgate"] = empty("dgate", T // c["gate_rows"], d)
        if c["post"]:
            out["dw_post"] = empty("dw_post", d, dtype=torch.float32)
        out["dx"] = empty("dx", T, d)
        need = D.dora_block_norm_backward_workspace(T, d, c["gate_rows"], lib_dt)
        return D.dora_block_norm_backward(st["dy"], st["x"], st["h"], st["w_pre"], st["r_pre"],
                                          rstd_post=st["r_post"], dh=st["dh"], ws=space(need),
                                          out=out, **kw)
    if op == "weight4":
        rows, d, g = c["rows"], c["d"], c["group"]
        n = -(-d // g)
        codes, scale = D.dora_quantize_fourbit(
            st["W"], group=g, codes=empty("codes", rows, n * g // 2, dtype=torch.uint8),
            scale=empty("scale", rows, n, dtype=torch.bfloat16))
        values = D.dora_dequantize_fourbit(codes, scale, d, group=g, out=empty("values", rows, d))
        return {"values": values, "scale": scale}
    if op == "linear4":
        T, d_in, d_out = c["T"], c["d_in"], c["d_out"]
        need = D.dora_linear_fourbit_workspace(T, d_in, d_out, lib_dt)
        return D.dora_linear_fourbit(st["x"], st["codes"], st["scale"], group=c["group"],
                                   y=empty("y", T, d_out), ws=space(need))
    if not c["step"]:
        rows, cols = c["rows"], c["cols"]
        need = D.dora_orthogonalize_workspace(rows, cols, lib_dt)
        return D.dora_orthogonalize(st["U"], steps=STEPS, coefficients=QUINTIC, eps=TINY,
                                    out=empty("O", rows, cols), ws=space(need))
    k = range(len(st["p"]))
    p = [empty(f"p{i}", *st["p"][i].shape) for i in k]
    M = [empty(f"M{i}", *st["M"][i].shape, dtype=torch.float32) for i in k]
    need = D.dora_muon_workspace(st["p"])
    D.dora_muon(st["p"], st["g"], st["M"], LR, mu=MU, weight_decay=DECAY,
                scales=[_reach(q.shape) for q in p], nesterov=True, steps=STEPS,
                coefficients=QUINTIC, eps=TINY, params_out=p, momenta_out=M, ws=space(need))
    out = {}
    for i in k:
        out |= {f"p{i}": p[i], f"M{i}": M[i]}
    return out


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("block", "block_backward"):
        T, d, rows = case["T"], case["d"], case["gate_rows"]
        gate = T // rows * d * e if rows else 0
        vectors = (2 if case["post"] else 1) * d
        if op == "block":  # x, residual -> h, y
            return {"bytes": 4 * T * d * e + gate + vectors * e, "flops": 14 * T * d}
        # dy, dh, x, h -> dx, dresidual; gradients of the gate and the weights
        return {"bytes": 6 * T * d * e + 2 * gate + vectors * (e + 4), "flops": 31 * T * d}
    if op == "weight4":
        size, n = case["rows"] * case["d"], case["rows"] * -(-case["d"] // case["group"])
        return {"bytes": 2 * size * e + 2 * n, "flops": 8 * size}
    if op == "linear4":
        T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
        n = -(-d_in // case["group"])
        return {"bytes": d_out * (n * case["group"] // 2 + 2 * n) + T * (d_in + d_out) * e,
                "flops": 2 * T * d_in * d_out}
    if not case["step"]:
        shapes, each = [(case["rows"], case["cols"])], 2 * e
    else:  # parameter, gradient and momentum -> parameter and momentum
        shapes, each = _factors(case), 3 * e + 8
    flops = 0
    for s in shapes:
        k, long = min(s), max(s)
        # the Gram matrix of the long side once (one half), its polynomials
        # (symmetric, three products a step) and the product with the long side
        flops += k * k * long * 3 + STEPS * 3 * k ** 3
    return {"bytes": sum(s[0] * s[1] for s in shapes) * each, "flops": flops}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits on the inputs of prepare."""
    i = prepare(case, seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    f64 = torch.float64

    def wide(name):
        return None if i[name] is None else i[name].to(f64)

    if op in ("block", "block_backward"):
        T, d = case["T"], case["d"]
        x, w2, w1, gate = (wide(k) for k in ("x", "w_pre", "w_post", "gate"))
        g = torch.ones(1, 1, d, dtype=f64, device=x.device) if gate is None else gate[:, None, :]
        fold = (g.shape[0], -1, d)
        s1 = (torch.sum(x * x, dim=1, keepdim=True) / d + EPS).sqrt() if case["post"] else 1.0
        u = x / s1 * (w1 if case["post"] else 1.0)
        if op == "block":
            # the sum is stored in the inputs' type, and normed as stored
            h = RESIDUAL * wide("res") + BRANCH * (u.view(fold) * g).view(T, d)
            h = h.float().to(dt).to(f64)
            s2 = (torch.sum(h * h, dim=1, keepdim=True) / d + EPS).sqrt()
            return {"h": h, "y": h * w2 / s2}
        dy, h = wide("dy"), wide("h")
        s2 = (torch.sum(h * h, dim=1, keepdim=True) / d + EPS).sqrt()
        along = torch.sum(dy * w2 * h, dim=1, keepdim=True) / (d * s2 * s2)
        dh = wide("dh") + (dy * w2 - h * along) / s2
        out = {"dresidual": RESIDUAL * dh, "dw_pre": torch.sum(dy * h / s2, dim=0)}
        if gate is not None:
            out["dgate"] = BRANCH * torch.sum((dh * u).view(fold), dim=1)
        du = BRANCH * (dh.view(fold) * g).view(T, d)
        if case["post"]:
            out["dw_post"] = torch.sum(du * x / s1, dim=0)
            along = torch.sum(du * w1 * x, dim=1, keepdim=True) / (d * s1 * s1)
            du = (du * w1 - x * along) / s1
        out["dx"] = du
        return out
    if op == "weight4":
        W, d, group = wide("W"), case["d"], case["group"]
        values, scales = torch.empty_like(W), []
        for lo in range(0, d, group):
            part = W[:, lo:lo + group]
            top = part.abs().max(dim=1, keepdim=True).values
            m, e = torch.frexp(top / 6)
            s = torch.ldexp(torch.round(m * 64) / 64, e)
            s = torch.where(top > 0, s.clamp(LEAST, MOST), 0.0)
            a = part.abs()
            v = 0.5 * (a > 0.25 * s) + 0.5 * (a >= 0.75 * s) + 0.5 * (a > 1.25 * s) \
                + 0.5 * (a >= 1.75 * s) + (a > 2.5 * s) + (a >= 3.5 * s) + 2.0 * (a > 5.0 * s)
            values[:, lo:lo + group] = torch.where(part < 0, -v, v) * s
            scales.append(s)
        return {"values": values, "scale": torch.cat(scales, dim=1)}
    if op == "linear4":
        d_in, codes, scale = case["d_in"], i["codes"], wide("scale")
        W = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=f64, device=codes.device)
        for half, nibble in ((0, codes % 16), (1, torch.div(codes, 16, rounding_mode="floor"))):
            size = (nibble % 8).to(f64)
            # e2m1: one bit of fraction, below 1 in steps of a half
            e = torch.div(size, 2, rounding_mode="floor")
            v = torch.where(e > 0, (1 + 0.5 * (size % 2)) * 2.0 ** (e - 1), 0.5 * size)
            W[:, half::2] = torch.where(nibble >= 8, -v, v)
        W *= scale.repeat_interleave(case["group"], dim=1)
        return torch.mm(wide("x"), W[:, :d_in].t())
    a, b, c = QUINTIC

    def orthogonal(U):
        flip = U.shape[0] < U.shape[1]
        X = U.t() if flip else U
        X = X / (torch.linalg.vector_norm(X) + TINY)
        for _ in range(STEPS):
            K = torch.mm(X.t(), X)
            X = a * X + b * torch.mm(X, K) + c * torch.mm(torch.mm(X, K), K)
        return X.t().contiguous() if flip else X

    if not case["step"]:
        return orthogonal(wide("U"))
    out = {}
    for k, (p, g, M) in enumerate(zip(i["p"], i["g"], i["M"])):
        p, g = p.to(f64), g.to(f64)
        new = M.to(f64) * MU + g
        out[f"p{k}"] = (1 - LR * DECAY) * p - LR * _reach(p.shape) * orthogonal(g + MU * new)
        out[f"M{k}"] = new
    return out
