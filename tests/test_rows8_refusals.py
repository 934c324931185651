"""CPU: the 8-bit row calls refuse bad arguments on the host (fake pointers,
nothing is launched), size their workspaces, and the plain forms their GPU
tests compare with agree with differences of the formula."""
import ctypes

import pytest
import torch

import rows8_ref as R
from dora_adapter_amd import dora as D

E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_WS, E_ALIAS, E_VALUE = 1, 2, 3, 4, 5, 6, 8
F32, BF16 = 0, 1
FAKE = 1 << 40
AT = [FAKE + (k << 33) for k in range(24)]


def _p(addr):
    return ctypes.c_void_p(addr)


def norm(x=AT[0], res=AT[1], w=AT[2], eps=1e-6, T=16, d=64, dt=BF16, group=0, y=AT[3], h=AT[4],
         rstd=AT[5], q=AT[6], scale=AT[7]):
    return D.lib().dora_rmsnorm(_p(x), _p(res), _p(w), eps, T, d, dt, group, _p(y), _p(h),
                                _p(rstd), _p(q), _p(scale), None)


@pytest.mark.parametrize("kw,code", [
    ({"x": 0}, E_NULL), ({"w": 0}, E_NULL), ({"y": 0, "q": 0}, E_NULL), ({"scale": 0}, E_NULL),
    ({"dt": 2}, E_DTYPE), ({"T": -1}, E_SHAPE), ({"d": 0}, E_SHAPE), ({"T": 1 << 31}, E_SHAPE),
    ({"group": 16}, E_SHAPE), ({"group": 96}, E_SHAPE), ({"group": 1024}, E_SHAPE),
    ({"group": -32}, E_SHAPE), ({"eps": -1e-6}, E_VALUE), ({"eps": float("nan")}, E_VALUE),
    ({"eps": float("inf")}, E_VALUE), ({"x": AT[0] + 8}, E_ALIGN), ({"rstd": AT[5] + 4}, E_ALIGN),
    ({"q": AT[6] + 1}, E_ALIGN),
    ({"h": AT[0] + 16}, E_ALIAS),            # a shifted view of x
    ({"h": AT[1] + 16}, E_ALIAS),            # of the residual
    ({"y": AT[0] + 64}, E_ALIAS), ({"y": AT[1]}, E_ALIAS), ({"y": AT[4]}, E_ALIAS),
    ({"y": AT[0], "h": AT[0]}, E_ALIAS),     # both in place of x
    ({"q": AT[0]}, E_ALIAS), ({"scale": AT[6] + 64}, E_ALIAS), ({"rstd": AT[2]}, E_ALIAS),
    ({"q": AT[2] + 16}, E_ALIAS),
])
def test_rmsnorm_refuses(kw, code):
    assert norm(**kw) == code
    assert D.lib().dora_last_error()


def test_rmsnorm_scale_extent_counts_in_the_overlap_check():
    # 16 rows of 2 groups: 128 bytes of scales, the last of them over rstd
    assert norm(group=32, scale=AT[5] - 112) == E_ALIAS


def norm_bwd(dy=AT[0], h=AT[1], w=AT[2], rstd=AT[3], dres=AT[4], T=16, d=64, dt=BF16, dx=AT[5],
             dw=AT[6], ws=AT[7], ws_bytes=1 << 20):
    return D.lib().dora_rmsnorm_backward(_p(dy), _p(h), _p(w), _p(rstd), _p(dres), T, d, dt,
                                         _p(dx), _p(dw), _p(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    ({"dy": 0}, E_NULL), ({"h": 0}, E_NULL), ({"rstd": 0}, E_NULL), ({"dx": 0}, E_NULL),
    ({"dt": 9}, E_DTYPE), ({"d": -1}, E_SHAPE), ({"ws": 0}, E_WS), ({"ws_bytes": 8}, E_WS),
    ({"dw": AT[6] + 4}, E_ALIGN), ({"dx": AT[0]}, E_ALIAS), ({"dx": AT[1] + 32}, E_ALIAS),
    ({"dx": AT[4] + 16}, E_ALIAS), ({"dw": AT[2]}, E_ALIAS), ({"ws": AT[4]}, E_ALIAS),
])
def test_rmsnorm_backward_refuses(kw, code):
    assert norm_bwd(**kw) == code


def quant(x=AT[0], rows=16, d=64, dt=BF16, group=0, q=AT[1], scale=AT[2]):
    return D.lib().dora_quantize_rows(_p(x), rows, d, dt, group, _p(q), _p(scale), None)


def dequant(q=AT[0], scale=AT[1], rows=16, d=64, dt=BF16, group=0, out=AT[2]):
    return D.lib().dora_dequantize_rows(_p(q), _p(scale), rows, d, dt, group, _p(out), None)


@pytest.mark.parametrize("kw,code", [
    ({"q": 0}, E_NULL), ({"scale": 0}, E_NULL), ({"rows": -1}, E_SHAPE), ({"d": 0}, E_SHAPE),
    ({"group": 8}, E_SHAPE), ({"dt": 3}, E_DTYPE), ({"q": AT[1] + 2}, E_ALIGN),
])
def test_quantize_and_dequantize_refuse(kw, code):
    assert quant(**kw) == code
    assert dequant(**kw) == code


def test_quantize_and_dequantize_refuse_overlap():
    assert quant(q=AT[0] + 32) == E_ALIAS and quant(scale=AT[1]) == E_ALIAS
    assert dequant(out=AT[0]) == E_ALIAS and dequant(out=AT[1]) == E_ALIAS


def linear(xq=AT[0], xs=AT[1], wq=AT[2], ws_=AT[3], T=16, d_in=64, d_out=48, dt=BF16, y=AT[4],
           ws=AT[5], ws_bytes=1 << 30):
    return D.lib().dora_linear_quantized(_p(xq), _p(xs), _p(wq), _p(ws_), T, d_in, d_out, dt,
                                         _p(y), _p(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    ({"xq": 0}, E_NULL), ({"xs": 0}, E_NULL), ({"wq": 0}, E_NULL), ({"ws_": 0}, E_NULL),
    ({"y": 0}, E_NULL), ({"dt": -1}, E_DTYPE), ({"d_in": 0}, E_SHAPE), ({"T": -1}, E_SHAPE),
    ({"d_in": 131072}, E_SHAPE), ({"wq": AT[2] + 4}, E_ALIGN), ({"y": AT[0]}, E_ALIAS),
    ({"y": AT[2] + 16}, E_ALIAS), ({"y": AT[3]}, E_ALIAS),
])
def test_linear_quantized_refuses(kw, code):
    assert linear(**kw) == code


def test_linear_quantized_workspace():
    L = D.lib()
    assert L.dora_linear_quantized_workspace(16, 131072, 64, BF16) == 0
    assert L.dora_linear_quantized_workspace(-1, 64, 64, BF16) == 0
    assert L.dora_linear_quantized_workspace(16, 64, 64, 4) == 0
    # no d_in x d_out term: only int32 partial sums of y, 32 at most
    for T in (1, 64, 300, 8192):
        for d_in, d_out in ((8192, 28672), (28672, 8192), (131071, 64), (1029, 2051)):
            need = L.dora_linear_quantized_workspace(T, d_in, d_out, BF16)
            assert need <= 32 * T * d_out * 4 + 256
            if need:
                assert linear(T=T, d_in=d_in, d_out=d_out, ws=0) == E_WS
                assert linear(T=T, d_in=d_in, d_out=d_out, ws_bytes=need - 1) == E_WS
                assert linear(T=T, d_in=d_in, d_out=d_out, ws=AT[2]) == E_ALIAS


def ckpt(through=0, T=16, d_in=128, d_out=64, r=8, dt=BF16, group=0, ws_bytes=None, s=1.0, **at):
    names = ["dy", "xq", "xs", "W", "A", "B", "m", "n", "P", "yq", "ys", "U", "dx", "dA", "dB",
             "dm", "ws"]
    a = {k: AT[i] for i, k in enumerate(names)}
    a["U"] = 0
    a.update(at)
    L = D.lib()
    if ws_bytes is None:
        ws_bytes = max(1, L.dora_backward_checkpoint_workspace(T, d_in, d_out, r, dt, through))
    v = {k: _p(x) for k, x in a.items()}
    return L.dora_backward_checkpoint(v["dy"], v["xq"], v["xs"], v["W"], v["A"], v["B"], v["m"],
                                      v["n"], s, v["P"], v["yq"], v["ys"], group, v["U"], through,
                                      T, d_in, d_out, r, dt, v["dx"], v["dA"], v["dB"], v["dm"],
                                      v["ws"], ws_bytes, None)


@pytest.mark.parametrize("through", [0, 1])
@pytest.mark.parametrize("kw,code", [
    ({"xq": 0}, E_NULL), ({"xs": 0}, E_NULL), ({"yq": 0}, E_NULL), ({"ys": 0}, E_NULL),
    ({"dm": 0}, E_NULL), ({"group": 48}, E_SHAPE), ({"r": 0}, E_SHAPE), ({"dt": 6}, E_DTYPE),
    ({"ws_bytes": 64}, E_WS), ({"ys": AT[10] + 4}, E_ALIGN), ({"dx": AT[1]}, E_ALIAS),
    ({"dA": AT[10]}, E_ALIAS), ({"dB": AT[9] + 16}, E_ALIAS), ({"ws": AT[2]}, E_ALIAS),
])
def test_backward_checkpoint_refuses(through, kw, code):
    assert ckpt(through, **kw) == code


def test_backward_checkpoint_takes_U_through_the_norm_only():
    assert ckpt(0, U=AT[17]) == E_VALUE
    assert ckpt(1, U=AT[13]) == E_ALIAS


def test_backward_checkpoint_workspace_holds_no_dense_weight():
    L = D.lib()
    for through in (0, 1):
        a = L.dora_backward_checkpoint_workspace(64, 8192, 8192, 64, BF16, through)
        assert 0 < a < 8192 * 8192 * 2
    assert L.dora_backward_checkpoint_workspace(64, 0, 8192, 64, BF16, 0) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64)
    for call in (lambda: D.dora_rmsnorm(x, x[0]), lambda: D.dora_quantize_rows(x),
                 lambda: D.dora_rmsnorm_backward(x, x, x[0], x[:, 0])):
        with pytest.raises(ValueError):
            call()


# --------------------------------------------- the plain forms by differences
def test_norm_gradient_of_the_plain_form_matches_differences():
    g = torch.Generator().manual_seed(5)
    T, d, eps = 3, 7, 1e-3
    h, dy, dres = (torch.randn(T, d, generator=g, dtype=torch.float64) for _ in range(3))
    w = 1 + 0.3 * torch.randn(d, generator=g, dtype=torch.float64)

    def loss(h, w):
        return float((R.norm(h, w, eps)[0] * dy).sum() + (h * dres).sum())

    dx, dw, _, _ = R.norm_grad(dy, h, w, R.norm(h, w, eps)[1], dres)
    step = 1e-6
    # central differences: error O(step^2) and 2^-52 / step, both under 1e-8
    for t in range(T):
        for j in range(d):
            e = torch.zeros(T, d, dtype=torch.float64)
            e[t, j] = step
            assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * step) - dx[t, j]) < 1e-7
    for j in range(d):
        e = torch.zeros(d, dtype=torch.float64)
        e[j] = step
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * step) - dw[j]) < 1e-7


@pytest.mark.parametrize("through", [False, True])
def test_module_gradient_of_the_plain_form_matches_differences(through):
    g = torch.Generator().manual_seed(6)
    T, d_in, d_out, r, s = 4, 6, 5, 2, 1.5
    rnd = lambda *sh: torch.randn(*sh, generator=g, dtype=torch.float64)  # noqa: E731
    x, W, A, B, dy = rnd(T, d_in), rnd(d_out, d_in), rnd(r, d_in), rnd(d_out, r), rnd(T, d_out)
    m = 1 + rnd(d_out).abs()
    n0 = (W + s * B @ A).norm(dim=1)

    def loss(x, A, B, m):
        V = W + s * B @ A
        n = V.norm(dim=1) if through else n0
        return float((dy * (m / n) * (x @ V.T)).sum())

    y = (m / n0) * (x @ (W + s * B @ A).T)
    ref = R.backward(dy, x, W, A, B, m, n0, s, x @ A.T, y, through)
    step = 1e-6
    for key, at in (("dx", 0), ("dA", 1), ("dB", 2), ("dm", 3)):
        args = [x, A, B, m]
        flat = args[at].reshape(-1)
        for k in range(flat.numel()):
            e = torch.zeros_like(flat)
            e[k] = step
            e = e.reshape(args[at].shape)
            up, down = list(args), list(args)
            up[at], down[at] = args[at] + e, args[at] - e
            diff = (loss(*up) - loss(*down)) / (2 * step)
            assert abs(diff - ref[key].reshape(-1)[k]) < 1e-6, (key, k)
