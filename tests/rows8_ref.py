"""Plain fp64 forms of the 8-bit row operators, for their tests (CPU tensors).

Written from the formulas: the norm with the residual's addition and its
gradient, rows held as int8 with absolute-maximum scales, the int8 linear
layer, and the module's backward with the norm held constant or not."""
import torch

MIN_SCALE = 2.0 ** -126
MAX_SCALE = float.fromhex("0x1.020406p+121")


def spread(scale, d, group):
    """scales [T, groups] over the d columns they belong to (fp64)."""
    s = scale.double()
    return s.expand(-1, d) if group == 0 else s.repeat_interleave(group, dim=1)[:, :d]


def quantize(v, group):
    """(q int8, scale fp32) of the rows of v, in 64 bits apart from the scale's
    own type; groups with an infinity or NaN get a NaN scale and q = 0."""
    v = v.double()
    T, d = v.shape
    width = group or d
    q = torch.zeros(T, d, dtype=torch.int8)
    scales = []
    for lo in range(0, d, width):
        part = v[:, lo:lo + width]
        top = part.abs().amax(dim=1, keepdim=True)
        bad = ~torch.isfinite(part).all(dim=1, keepdim=True)
        s = (top / 127).float().double().clamp(MIN_SCALE, MAX_SCALE)
        s = torch.where(top == 0, torch.zeros_like(s), s)
        s = torch.where(bad, torch.full_like(s, float("nan")), s)
        r = torch.where(s > 0, part / torch.where(s > 0, s, torch.ones_like(s)),
                        torch.zeros_like(part))
        q[:, lo:lo + width] = torch.round(r).clamp(-127, 127).to(torch.int8)
        scales.append(s.float())
    return q, torch.cat(scales, dim=1)


def norm_h(x, res):
    return x if res is None else (x.float() + res.float()).to(x.dtype)


def norm(h, w, eps):
    """(y, rstd) in 64 bits from the stored h."""
    h = h.double()
    rstd = ((h * h).mean(dim=1) + eps).rsqrt()
    return h * rstd[:, None] * w.double(), rstd


def norm_grad(dy, h, w, rstd, dres):
    """(dx, dw, sum_j |w dy h|, sum_t |dy h rstd|) in 64 bits."""
    dy, h, w, rstd = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    g = w * dy
    dx = rstd * g - h * rstd ** 3 * (g * h).mean(dim=1, keepdim=True)
    if dres is not None:
        dx = dx + dres.double()
    each = dy * h * rstd
    return dx, each.sum(0), (g * h).abs().sum(dim=1, keepdim=True), each.abs().sum(0)


def linear(xq, xs, wq, ws):
    """Exact int32 sums (fp64 products of int8 values are), scaled in 64 bits."""
    return (xq.double() @ wq.double().T) * xs.double() * ws.double().T


def backward(dy, x, W, A, B, m, n, s, P, y, through_norm):
    """Gradients in 64 bits of the module from x and y as restored (fp64)."""
    dy, W, A, B, m, n, P = (t.double() for t in (dy, W, A, B, m, n, P))
    dm = (dy * y).sum(0) / m
    dh = dy * (m / n)
    Q = s * dh @ B
    out = {"dx": dh @ W + Q @ A, "dA": Q.T @ x, "dB": s * dh.T @ P, "dm": dm}
    if through_norm:
        cV = (m * dm / n ** 2)[:, None] * (W + s * B @ A)
        out["dA"] = out["dA"] - s * B.T @ cV
        out["dB"] = out["dB"] - s * cV @ A.T
    return out
