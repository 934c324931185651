"""Plain fp64 forms of the operators around a module, for their tests (CPU tensors).

Written from the formulas: the norms on both sides of a residual addition and
their gradients.  Each comes with what its error bound needs."""
import torch

U = 2.0 ** -24


def half(dt):
    """Half a step of a type, relative: the most one rounding is off by."""
    return torch.finfo(dt).eps / 2


def sum_error(d):
    """A row's sum of d terms in fp32 by partial sums of at most d / 64 + 64 terms."""
    return (d / 64 + 64) * U


def _gate(gate, T, d):
    if gate is None:
        return torch.ones(1, 1, dtype=torch.float64)
    g = gate.double().reshape(-1, d)
    return g.repeat_interleave(max(T // g.shape[0], 1), dim=0)[:T]


def rms_factor(v, eps):
    v = v.double()
    return ((v * v).mean(dim=1) + eps).rsqrt()


def block_h(x, res, w_post, gate, a, b, eps):
    """(h unrounded, its bound for an fp32 evaluation rounded to x's type)."""
    T, d = x.shape
    u = x.double()
    E = 0.0
    if w_post is not None:
        u = u * rms_factor(x, eps)[:, None] * w_post.double()
        E = sum_error(d) + 5 * U
    branch = b * _gate(gate, T, d) * u
    h = a * res.double() + branch
    bound = branch.abs() * (E + 4 * U) + (a * res.double()).abs() * 3 * U
    return h, bound + (h.abs() + bound) * half(x.dtype)


def block_grad(dy, dh, x, h, w_pre, r2, w_post, r1, gate, a, b):
    """{name: (gradient, bound)} from the stored h and the kept factors r1, r2."""
    T, d = x.shape
    dt = x.dtype
    dy, x, h, w2, r2 = dy.double(), x.double(), h.double(), w_pre.double(), r2.double()[:, None]
    dh = torch.zeros_like(dy) if dh is None else dh.double()
    E = sum_error(d) + 8 * U
    hath = h * r2
    wdy = w2 * dy
    m1 = (wdy * hath).mean(1, keepdim=True)
    e1 = E * (wdy * hath).abs().mean(1, keepdim=True)
    Dh = dh + r2 * (wdy - m1 * hath)
    eD = 8 * U * (dh.abs() + r2 * (wdy.abs() + (m1 * hath).abs())) + r2 * hath.abs() * e1
    each = dy * hath
    out = {"dresidual": (a * Dh, abs(a) * eD + (a * Dh).abs() * (half(dt) + 2 * U)),
           "dw_pre": (each.sum(0), (T + 8) * U * each.abs().sum(0))}
    G = _gate(gate, T, d)
    w1 = torch.ones(d, dtype=torch.float64) if w_post is None else w_post.double()
    f1 = torch.ones(T, 1, dtype=torch.float64) if w_post is None else r1.double()[:, None]
    hatx = x * f1
    if gate is not None:
        n = gate.numel() // d
        each, err = b * Dh * hatx * w1, abs(b) * eD * (hatx * w1).abs()
        fold = lambda t: t.reshape(n, -1, d).sum(1).reshape(gate.shape)  # noqa: E731
        g = fold(each)
        e = fold(err) + (T // max(n, 1) + 10) * U * fold(each.abs())
        out["dgate"] = (g, e + (g.abs() + e) * half(dt))
    du = b * G * Dh
    edu = (b * G).abs() * eD + 4 * U * du.abs()
    if w_post is None:
        out["dx"] = (du, edu + (du.abs() + edu) * half(dt))
        return out
    each = du * hatx
    out["dw_post"] = (each.sum(0), (edu * hatx.abs()).sum(0) + (T + 8) * U * each.abs().sum(0))
    k = (b * G * w1 * hatx).abs()
    A = (k * (dh.abs() + r2 * wdy.abs())).mean(1, keepdim=True)
    B = (k * r2 * hath.abs()).mean(1, keepdim=True)
    m2 = (w1 * du * hatx).mean(1, keepdim=True)
    e2 = E * (A + m1.abs() * B) + B * e1
    dx = f1 * (w1 * du - m2 * hatx)
    e = f1 * (w1.abs() * edu + 8 * U * ((w1 * du).abs() + (m2 * hatx).abs()) + hatx.abs() * e2)
    out["dx"] = (dx, e + (dx.abs() + e) * half(dt))
    return out


# -------------------------------------------------------------- 4-bit rows
E2M1 = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def fourbit(v, group):
    """(values the codes stand for without their scale, scales) of the rows of v, in 64 bits:
    the nearest e2m1 values, ties to the even code; the scale max / 6 at six bits."""
    v = v.double()
    T, d = v.shape
    n = -(-d // group)
    p = torch.zeros(T, n * group, dtype=torch.float64)
    p[:, :d] = v
    p = p.view(T, n, group)
    bad = ~torch.isfinite(p).all(dim=2)
    top = torch.where(bad[:, :, None], torch.zeros_like(p), p).abs().amax(dim=2)
    m, e = torch.frexp(top / 6)
    s = torch.ldexp(torch.round(m * 64) / 64, e).clamp(2.0 ** -125, 1.3125 * 2.0 ** 125)
    s = torch.where(top > 0, s, torch.zeros_like(s))
    t = p.abs() / torch.where(s > 0, s, torch.ones_like(s))[:, :, None]
    near = (t[..., None] - E2M1).abs()
    # the least distance, and of two the even code
    order = near + torch.tensor([0.0, 1e-15] * 4, dtype=torch.float64)
    code = order.argmin(dim=-1)
    values = torch.sign(p) * E2M1[code]
    s = torch.where(bad, torch.full_like(s, float("nan")), s)
    return values.view(T, n * group)[:, :d], s


def unpack(codes):
    """The values of packed codes, scale apart."""
    c = torch.stack([codes & 15, codes >> 4], dim=2).view(codes.shape[0], -1).long()
    return E2M1[c & 7] * torch.where(c >= 8, -1.0, 1.0).double()


def restored(codes, scale, d, group):
    return (unpack(codes) * scale.double().repeat_interleave(group, dim=1))[:, :d]


# ---------------------------------------------------------- Newton-Schulz steps
QUINTIC = (3.4445, -4.7750, 2.0315)


def orthogonal(U, steps=5, coefficients=QUINTIC, eps=1e-7):
    """The literal steps in 64 bits."""
    a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in coefficients)
    X = U.double()
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    X = X / (torch.linalg.vector_norm(X) + float(torch.tensor(eps, dtype=torch.float32)))
    for _ in range(steps):
        G = X @ X.T
        X = a * X + (b * G + c * (G @ G)) @ X
    return X.T if tall else X


def steepest(steps, coefficients):
    """The largest |f'| on [0, 1] of what the steps do to a singular value."""
    a, b, c = coefficients
    s = torch.linspace(0, 1, 20001, dtype=torch.float64)
    d = torch.ones_like(s)
    for _ in range(steps):
        d = d * (a + 3 * b * s ** 2 + 5 * c * s ** 4)
        s = a * s + b * s ** 3 + c * s ** 5
    return float(d.abs().max())


def orthogonal_bound(U, O, dt, steps=5, coefficients=QUINTIC, eps=1e-7, moved=0.0):
    """How far (Frobenius norm) an O formed from U may be from the 64-bit one.

    A change of U by d moves O by at most steepest |d| / |U| (the steps act on
    singular values, and the divided differences of an odd f are no steeper than
    f); bf16 matrices keep U to 2^-17 of each element, and `moved` is what U
    itself is off by.  The product at the end is Q U with O = Q U: its elements
    are off by 2^-15 of |Q| |U| with two bf16 numbers an operand (16 bits each, the
    product of the low parts left out, fp32 sums), by (6 n + 8) 2^-24 with three.
    (The n x n part of bf16 matrices is in 32 bits; its roundings have no share of
    their own here: a product's are 2^-24 of what the 2^-15 is taken of.)
    Then the output's rounding."""
    X = U.double() if U.shape[0] <= U.shape[1] else U.double().T
    n = X.shape[0]
    size = float(torch.linalg.vector_norm(X)) + eps
    a, b, c = coefficients
    G = X @ X.T / size ** 2
    Q = torch.eye(n, dtype=torch.float64)
    for _ in range(steps):
        P = a * torch.eye(n, dtype=torch.float64) + b * G + c * (G @ G)
        Q, G = P @ Q, P @ G @ P
    QU = float(torch.linalg.vector_norm((Q / size).abs() @ X.abs()))
    bf = dt == torch.bfloat16
    off = (2.0 ** -17 if bf else 0.0) + moved
    return (steepest(steps, coefficients) * off * min(1.0, float(torch.linalg.vector_norm(X)) / size)
            + QU * (2.0 ** -15 if bf else (6 * n + 8) * U_) + float(torch.linalg.vector_norm(O)) * half(dt)
            + 1e-12)


U_ = U
