"""CPU: the calls around a module refuse bad arguments on the host (fake
pointers, nothing is launched), size their workspaces, and the plain forms
that their GPU tests compare with agree with differentiation."""
import ctypes

import pytest
import torch

import around_ref as R
from dora_adapter_amd import dora as D

E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_WS, E_ALIAS, E_VALUE = 1, 2, 3, 4, 5, 6, 8
F32, BF16 = 0, 1
FAKE = 1 << 40
AT = [FAKE + (k << 33) for k in range(24)]


def _p(addr):
    return ctypes.c_void_p(addr)


def block(x=AT[0], res=AT[1], w1=AT[2], gate=AT[3], rows=4, w2=AT[4], a=1.0, b=1.0, eps=1e-6, T=16,
          d=64, dt=BF16, h=AT[5], y=AT[6], r1=AT[7], r2=AT[8]):
    return D.lib().dora_block_norm(_p(x), _p(res), _p(w1), _p(gate), rows, _p(w2), a, b, eps, T, d,
                                   dt, _p(h), _p(y), _p(r1), _p(r2), None)


@pytest.mark.parametrize("kw,code", [
    ({"x": 0}, E_NULL), ({"res": 0}, E_NULL), ({"w2": 0}, E_NULL), ({"h": 0}, E_NULL),
    ({"y": 0}, E_NULL), ({"dt": 2}, E_DTYPE), ({"T": -1}, E_SHAPE), ({"d": 0}, E_SHAPE),
    ({"T": 1 << 31}, E_SHAPE), ({"rows": 0}, E_SHAPE), ({"rows": -3}, E_SHAPE),
    ({"rows": 1 << 31}, E_SHAPE), ({"eps": -1e-6}, E_VALUE), ({"eps": float("nan")}, E_VALUE),
    ({"eps": float("inf")}, E_VALUE), ({"a": float("nan")}, E_VALUE), ({"b": float("inf")}, E_VALUE),
    ({"w1": 0}, E_VALUE),                     # rstd_post without it
    ({"x": AT[0] + 8}, E_ALIGN), ({"gate": AT[3] + 2}, E_ALIGN), ({"r2": AT[8] + 4}, E_ALIGN),
    ({"h": AT[1] + 16}, E_ALIAS), ({"h": AT[0]}, E_ALIAS), ({"y": AT[0] + 64}, E_ALIAS),
    ({"y": AT[1]}, E_ALIAS), ({"y": AT[5]}, E_ALIAS), ({"y": AT[2]}, E_ALIAS),
    ({"h": AT[3] + 3 * 128}, E_ALIAS),        # the last of four gate rows
    ({"r1": AT[0]}, E_ALIAS), ({"r1": AT[8]}, E_ALIAS), ({"r2": AT[4] + 64}, E_ALIAS),
])
def test_block_norm_refuses(kw, code):
    assert block(**kw) == code
    assert D.lib().dora_last_error()


def block_bwd(dy=AT[0], dh=AT[1], x=AT[2], h=AT[3], w1=AT[4], gate=AT[5], rows=4, w2=AT[6], r1=AT[7],
              r2=AT[8], a=1.0, b=1.0, T=16, d=64, dt=BF16, dx=AT[9], dres=AT[10], dgate=AT[11],
              dw1=AT[12], dw2=AT[13], ws=AT[14], ws_bytes=1 << 24):
    return D.lib().dora_block_norm_backward(
        _p(dy), _p(dh), _p(x), _p(h), _p(w1), _p(gate), rows, _p(w2), _p(r1), _p(r2), a, b, T, d, dt,
        _p(dx), _p(dres), _p(dgate), _p(dw1), _p(dw2), _p(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    ({"dy": 0}, E_NULL), ({"x": 0}, E_NULL), ({"h": 0}, E_NULL), ({"w2": 0}, E_NULL),
    ({"r1": 0}, E_NULL), ({"r2": 0}, E_NULL), ({"dx": 0}, E_NULL), ({"dres": 0}, E_NULL),
    ({"dt": 7}, E_DTYPE), ({"d": -4}, E_SHAPE), ({"rows": 0}, E_SHAPE),
    ({"a": float("inf")}, E_VALUE), ({"w1": 0}, E_VALUE), ({"gate": 0}, E_VALUE),
    ({"ws": 0}, E_WS), ({"ws_bytes": 64}, E_WS), ({"ws": AT[14] + 8}, E_ALIGN),
    ({"dw2": AT[13] + 4}, E_ALIGN), ({"dx": AT[0]}, E_ALIAS), ({"dx": AT[1]}, E_ALIAS),
    ({"dx": AT[2]}, E_ALIAS), ({"dres": AT[1] + 16}, E_ALIAS), ({"dres": AT[3]}, E_ALIAS),
    ({"dres": AT[9] + 512}, E_ALIAS), ({"dgate": AT[5]}, E_ALIAS), ({"dgate": AT[9]}, E_ALIAS),
    ({"dw1": AT[13]}, E_ALIAS), ({"dw1": AT[4]}, E_ALIAS), ({"ws": AT[2]}, E_ALIAS),
    ({"ws": AT[1]}, E_ALIAS), ({"ws": AT[12]}, E_ALIAS),
])
def test_block_norm_backward_refuses(kw, code):
    assert block_bwd(**kw) == code
    assert D.lib().dora_last_error()


def test_block_norm_workspaces():
    q = D.dora_block_norm_backward_workspace
    assert q(-1, 64, 0, BF16) == 0 and q(4, 0, 0, BF16) == 0 and q(4, 64, -1, BF16) == 0
    assert q(4, 64, 0, 9) == 0
    # sums of a few rows a workgroup: never more than the matrix in fp32, about
    for T, d in ((8192, 8192), (65536, 128), (4096, 28672), (100000, 40000)):
        for rows in (0, 1, 2, 47, 1000, T):
            for dt in (F32, BF16):
                assert q(T, d, rows, dt) <= 2 * T * d * 4 + (1 << 20), (T, d, rows, dt)
    assert q((1 << 31) - 1, (1 << 31) - 1, 3, BF16) > 0


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, (20,), (6, 20), (2, 20)])
def test_plain_block_gradients_are_those_of_differentiation(post, gate):
    g = torch.Generator().manual_seed(3)
    T, d, eps, a, b = 6, 20, 1e-3, 0.75, 1.5

    def leaf(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64, requires_grad=True)

    x, res, w1, w2 = leaf(T, d), leaf(T, d), leaf(d), leaf(d)
    gt = None if gate is None else leaf(*gate)
    dy, dh = torch.randn(T, d, generator=g).double(), torch.randn(T, d, generator=g).double()
    h, _ = R.block_h(x, res, w1 if post else None, gt, a, b, eps)
    r2 = R.rms_factor(h, eps)
    y = h * r2[:, None] * w2
    ((y * dy).sum() + (h * dh).sum()).backward()
    r1 = R.rms_factor(x, eps)
    with torch.no_grad():
        ref = R.block_grad(dy, dh, x, h, w2, r2, w1 if post else None, r1, gt, a, b)
    leaves = {"dx": x, "dresidual": res, "dw_pre": w2}
    if post:
        leaves["dw_post"] = w1
    if gate is not None:
        leaves["dgate"] = gt
    assert set(ref) == set(leaves)
    for k, t in leaves.items():
        assert torch.allclose(ref[k][0], t.grad, rtol=1e-10, atol=1e-12), k


def quant4(x=AT[0], rows=16, d=64, dt=BF16, group=32, codes=AT[1], scale=AT[2]):
    return D.lib().dora_quantize_fourbit(_p(x), rows, d, dt, group, _p(codes), _p(scale), None)


def dequant4(codes=AT[0], scale=AT[1], rows=16, d=64, dt=BF16, group=32, out=AT[2]):
    return D.lib().dora_dequantize_fourbit(_p(codes), _p(scale), rows, d, dt, group, _p(out), None)


@pytest.mark.parametrize("kw,code", [
    ({"codes": 0}, E_NULL), ({"scale": 0}, E_NULL), ({"rows": -1}, E_SHAPE), ({"d": 0}, E_SHAPE),
    ({"group": 0}, E_SHAPE), ({"group": 16}, E_SHAPE), ({"group": 96}, E_SHAPE),
    ({"group": 1024}, E_SHAPE), ({"group": -32}, E_SHAPE), ({"dt": 3}, E_DTYPE),
    ({"codes": AT[1] + 8}, E_ALIGN), ({"scale": AT[0] + 512}, E_ALIAS), ({"codes": AT[0]}, E_ALIAS),
])
def test_fourbit_rows_refuse(kw, code):
    if kw.get("codes") == AT[0]:  # (its own default in the second call)
        assert quant4(**kw) == code
        return
    assert quant4(**kw) == code
    back = {k: v for k, v in kw.items() if k != "scale" or v == 0}
    if "codes" in back and back["codes"]:
        back["codes"] = AT[0] + 8
    if back:
        assert dequant4(**back) == code


@pytest.mark.parametrize("kw,code", [
    ({"out": 0}, E_NULL), ({"out": AT[0] + 16}, E_ALIAS), ({"out": AT[1]}, E_ALIAS),
    ({"out": AT[2] + 4}, E_ALIGN),
])
def test_fourbit_restore_refuses(kw, code):
    assert dequant4(**kw) == code


def test_fourbit_extents_count_in_the_overlap_check():
    # 16 rows of 65 columns: three groups, 48 bytes of codes and 6 of scales a row
    assert quant4(d=65, scale=AT[1] + 15 * 48) == E_ALIAS
    assert dequant4(d=65, out=AT[1] + 80) == E_ALIAS


def linear4(x=AT[0], codes=AT[1], scale=AT[2], group=32, T=4, d_in=64, d_out=32, dt=BF16, y=AT[3],
            ws=AT[4], ws_bytes=1 << 28):
    return D.lib().dora_linear_fourbit(_p(x), _p(codes), _p(scale), group, T, d_in, d_out, dt, _p(y),
                                       _p(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    ({"x": 0}, E_NULL), ({"codes": 0}, E_NULL), ({"scale": 0}, E_NULL), ({"y": 0}, E_NULL),
    ({"T": -1}, E_SHAPE), ({"d_in": 0}, E_SHAPE), ({"d_out": 0}, E_SHAPE), ({"group": 48}, E_SHAPE),
    ({"dt": 4}, E_DTYPE), ({"x": AT[0] + 2}, E_ALIGN), ({"codes": AT[1] + 1}, E_ALIGN),
    ({"T": 257, "ws": 0}, E_WS), ({"T": 257, "ws_bytes": 100}, E_WS), ({"y": AT[0]}, E_ALIAS),
    ({"y": AT[1] + 16}, E_ALIAS), ({"y": AT[2]}, E_ALIAS), ({"T": 257, "ws": AT[1]}, E_ALIAS),
    ({"T": 257, "ws": AT[3]}, E_ALIAS),
])
def test_linear_fourbit_refuses(kw, code):
    assert linear4(**kw) == code
    assert D.lib().dora_last_error()


def test_linear_fourbit_workspace_holds_no_dense_weight():
    q = D.dora_linear_fourbit_workspace
    for T in (0, 1, 256):
        assert q(T, 8192, 28672, BF16) == 0
    assert q(-1, 8, 8, BF16) == 0 and q(300, 0, 8, BF16) == 0 and q(300, 8, 8, 5) == 0
    for dt, e in ((BF16, 2), (F32, 4)):
        for d_in, d_out in ((8192, 28672), (28672, 8192), (1 << 17, 1 << 14), (100, 1 << 20)):
            part = 32 * 257 * d_out * 4
            assert 0 < q(257, d_in, d_out, dt) <= max(128 << 20, 256 * d_in * e) + part + 512


def test_plain_fourbit_is_the_nearest_value():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40, 96, generator=g).double()
    values, s = R.fourbit(x, 32)
    v = (values * s.repeat_interleave(32, dim=1))
    each = R.E2M1 * s.repeat_interleave(32, dim=1)[..., None]
    both = torch.cat([each, -each], dim=-1)
    best = (x[..., None] - both).abs().amin(dim=-1)
    assert torch.equal((x - v).abs(), best)
    assert torch.equal(s.to(torch.bfloat16).double(), s)
    assert torch.equal(v.to(torch.bfloat16).double(), v)


def ortho(U=AT[0], rows=16, cols=64, dt=BF16, steps=5, c=(3.0, -4.0, 2.0), eps=1e-7, O=AT[1], ws=AT[2],
          ws_bytes=1 << 30):
    k = None if c is None else (ctypes.c_float * 3)(*c)
    return D.lib().dora_orthogonalize(_p(U), rows, cols, dt, steps, k, eps, _p(O), _p(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    ({"U": 0}, E_NULL), ({"O": 0}, E_NULL), ({"dt": 5}, E_DTYPE), ({"rows": 0}, E_SHAPE),
    ({"cols": -1}, E_SHAPE), ({"rows": 1 << 31}, E_SHAPE), ({"rows": 8193, "cols": 9000}, E_SHAPE),
    ({"rows": 64, "cols": 1 << 30}, E_SHAPE), ({"steps": 0}, E_VALUE), ({"steps": 17}, E_VALUE),
    ({"c": (float("inf"), 0, 0)}, E_VALUE), ({"eps": -1.0}, E_VALUE), ({"eps": float("nan")}, E_VALUE),
    ({"U": AT[0] + 8}, E_ALIGN), ({"ws": 0}, E_WS), ({"ws_bytes": 1000}, E_WS),
    ({"O": AT[0] + 16}, E_ALIAS), ({"ws": AT[0]}, E_ALIAS), ({"ws": AT[1] + 512}, E_ALIAS),
])
def test_orthogonalize_refuses(kw, code):
    assert ortho(**kw) == code
    assert D.lib().dora_last_error()


def muon(count=2, dt=BF16, mu=0.9, steps=5, eps=1e-7, ws=AT[20], ws_bytes=1 << 32, null=False, **kw):
    arr = (D.DoraUpdate * 2)()
    for k in range(2):
        at = AT[5 * k:5 * k + 5]
        v = dict(param=at[0], grad=at[1], momentum=at[2], param_out=at[3], momentum_out=at[4], rows=16,
                 cols=64, lr=0.1, weight_decay=0.0, scale=1.0)
        v.update({n[:-1]: x for n, x in kw.items() if n[-1] == str(k)})
        arr[k] = D.DoraUpdate(**{n: (x or None) if n in ("param", "grad", "momentum", "param_out",
                                                         "momentum_out") else x for n, x in v.items()})
    return D.lib().dora_muon(None if null else arr, count, dt, mu, 1, steps, None, eps, _p(ws), ws_bytes,
                             None)


@pytest.mark.parametrize("kw,code", [
    ({"null": True}, E_NULL), ({"count": -1}, E_SHAPE), ({"count": (1 << 16) + 1}, E_SHAPE),
    ({"param0": 0}, E_NULL), ({"grad1": 0}, E_NULL), ({"momentum0": 0}, E_NULL),
    ({"param_out1": 0}, E_NULL), ({"momentum_out0": 0}, E_NULL), ({"dt": 2}, E_DTYPE),
    ({"rows1": 0}, E_SHAPE), ({"cols0": -5}, E_SHAPE), ({"mu": float("nan")}, E_VALUE),
    ({"lr1": float("inf")}, E_VALUE), ({"weight_decay0": float("nan")}, E_VALUE),
    ({"scale1": float("nan")}, E_VALUE), ({"steps": 0}, E_VALUE), ({"eps": -1.0}, E_VALUE),
    ({"grad0": AT[1] + 4}, E_ALIGN), ({"ws": 0}, E_WS), ({"ws_bytes": 4096}, E_WS),
    ({"param_out0": AT[0] + 16}, E_ALIAS),            # a shifted view of its parameter
    ({"param_out0": AT[1]}, E_ALIAS),                 # its gradient
    ({"param_out1": AT[3]}, E_ALIAS),                 # the other's output
    ({"param_out1": AT[0]}, E_ALIAS),                 # the other's parameter
    ({"momentum_out0": AT[2] + 64}, E_ALIAS), ({"momentum_out1": AT[2]}, E_ALIAS),
    ({"momentum_out0": AT[0]}, E_ALIAS), ({"ws": AT[6]}, E_ALIAS), ({"ws": AT[4]}, E_ALIAS),
    # in place, but another update reads or writes it too
    ({"param_out0": AT[0], "param1": AT[0]}, E_ALIAS),
    ({"param_out0": AT[0], "param1": AT[0], "param_out1": AT[0]}, E_ALIAS),
    ({"momentum_out0": AT[2], "momentum1": AT[2] + 32}, E_ALIAS),
])
def test_muon_refuses(kw, code):
    assert muon(**kw) == code
    assert D.lib().dora_last_error()


def test_newton_schulz_workspaces():
    q = D.dora_orthogonalize_workspace
    assert q(0, 5, BF16) == 0 and q(5, 5, 7) == 0 and q(9000, 9000, F32) == 0
    for dt in (BF16, F32):
        # U, the Gram partials of 32 splits at most, six squares in 64 bits and the planes of Q
        for rows, cols in ((16, 4096), (384, 8192), (28672, 384), (37, 1027)):
            n, long = min(rows, cols), max(rows, cols)
            n = 64 if n <= 64 else -(-n // 128) * 128
            long = -(-long // 128) * 128
            assert 0 < q(rows, cols, dt) <= n * long * 4 + n * n * (32 * 8 + 48 + 6) + 4096

    def list_of(shapes):
        arr = (D.DoraUpdate * len(shapes))()
        for k, (r, c) in enumerate(shapes):
            arr[k].rows, arr[k].cols = r, c
        return D.lib().dora_muon_workspace(arr, len(shapes), BF16)

    one = list_of([(384, 8192)])
    assert one == q(384, 8192, BF16) and list_of([]) == 0
    # sets of matrices take the workspace in turn
    assert list_of([(384, 8192)] * 400) <= max(256 << 20, one)
    assert list_of([(384, 8192), (0, 5)]) == 0


@pytest.mark.parametrize("shape", [(5, 12), (12, 5), (7, 7)])
def test_plain_steps_act_on_singular_values(shape):
    U = torch.randn(*shape, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    u, s, v = torch.linalg.svd(U, full_matrices=False)
    s = s / (torch.linalg.vector_norm(s) + float(torch.tensor(1e-7)))
    a, b, c = (float(torch.tensor(k)) for k in R.QUINTIC)
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    assert torch.allclose(R.orthogonal(U), u @ torch.diag(s) @ v, atol=1e-11)
    assert R.steepest(5, R.QUINTIC) == pytest.approx(3.4445 ** 5, rel=1e-3)
