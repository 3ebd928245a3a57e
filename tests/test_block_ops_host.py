"""Block norm, act8 and adapters without a GPU: refusals, and the 64-bit forms against differences."""

import numpy as np
import pytest
import torch

import aware_block_transforms_amd as W
from oracle import block_ops as bo

L = W.lib
P = 4096          # a pointer that is only looked at
ODD = 4100        # not 16-byte aligned
NAN, INF = float("nan"), float("inf")


def norm(**kw):
    a = dict(ydt=0, rdt=0, udt=0, n=4, d=64, Y=P, wp=P, kind=0, gate=None, branch=1.0, R=P, res=1.0, w=P, eps=1e-6,
             Rout=P, U=P, k1=None, k2=None)
    a.update(kw)
    return L.wush_block_norm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(ydt=2), W.WUSH_E_ARG), (dict(rdt=-1), W.WUSH_E_ARG), (dict(udt=7), W.WUSH_E_ARG),
    (dict(rdt=1, udt=0), W.WUSH_E_UNSUPPORTED),
    (dict(n=-1), W.WUSH_E_SHAPE), (dict(d=0), W.WUSH_E_SHAPE), (dict(d=12), W.WUSH_E_SHAPE),
    (dict(d=24584), W.WUSH_E_SHAPE),
    (dict(kind=4), W.WUSH_E_ARG), (dict(kind=1), W.WUSH_E_ARG), (dict(gate=P), W.WUSH_E_ARG),
    (dict(Y=None), W.WUSH_E_ARG), (dict(Y=None, wp=None, w=None, U=None), W.WUSH_E_ARG),
    (dict(branch=NAN), W.WUSH_E_ARG), (dict(res=INF), W.WUSH_E_ARG), (dict(eps=0.0), W.WUSH_E_ARG),
    (dict(eps=NAN), W.WUSH_E_ARG), (dict(eps=INF), W.WUSH_E_ARG),
    (dict(w=None), W.WUSH_E_ARG), (dict(U=None), W.WUSH_E_ARG), (dict(R=None), W.WUSH_E_ARG),
    (dict(w=None, U=None, Rout=None), W.WUSH_E_ARG),
    (dict(Y=ODD), W.WUSH_E_ARG), (dict(R=ODD), W.WUSH_E_ARG), (dict(U=ODD), W.WUSH_E_ARG),
    (dict(wp=ODD), W.WUSH_E_ARG), (dict(kind=3, gate=ODD), W.WUSH_E_ARG), (dict(kind=1, gate=ODD), W.WUSH_E_ARG)])
def test_block_norm_refusals(kw, status):
    assert norm(**kw) == status
    assert L.wush_last_error().startswith(b"wush_block_norm:")


def test_block_norm_of_no_rows_returns_at_once():
    assert norm(n=0) == W.WUSH_OK


def norm_bwd(**kw):
    a = dict(ydt=0, rdt=0, udt=0, n=4, d=64, dU=P, dRout=P, Y=P, wp=P, kind=0, gate=None, branch=1.0, Rout=P, res=1.0,
             w=P, k1=P, k2=P, dY=P, dR=P, dgate=None, dwp=P, dw=P, ws=P, wsb=1 << 30)
    a.update(kw)
    return L.wush_block_norm_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(ydt=2), W.WUSH_E_ARG), (dict(rdt=1, udt=0), W.WUSH_E_UNSUPPORTED), (dict(n=-1), W.WUSH_E_SHAPE),
    (dict(d=4), W.WUSH_E_SHAPE), (dict(dU=None), W.WUSH_E_ARG), (dict(dw=None), W.WUSH_E_ARG),
    (dict(w=None), W.WUSH_E_ARG), (dict(dwp=None), W.WUSH_E_ARG), (dict(dY=None), W.WUSH_E_ARG),
    (dict(kind=1, gate=P), W.WUSH_E_ARG), (dict(dgate=P), W.WUSH_E_ARG),
    (dict(dU=None, w=None, dw=None, dRout=None), W.WUSH_E_ARG), (dict(k1=None), W.WUSH_E_ARG),
    (dict(k2=None), W.WUSH_E_ARG), (dict(Rout=None), W.WUSH_E_ARG), (dict(dU=ODD), W.WUSH_E_ARG),
    (dict(ws=ODD), W.WUSH_E_ARG), (dict(wsb=16), W.WUSH_E_ARG)])
def test_block_norm_bwd_refusals(kw, status):
    assert norm_bwd(**kw) == status
    assert L.wush_last_error().startswith(b"wush_block_norm_bwd:")


def test_act8_refusals():
    ok, arg, shape = W.WUSH_OK, W.WUSH_E_ARG, W.WUSH_E_SHAPE
    for f in (lambda dt, n, d, a, b, c: L.wush_act8_pack(dt, n, d, a, b, c, None),
              lambda dt, n, d, a, b, c: L.wush_act8_unpack(dt, n, d, b, c, a, None)):
        assert f(2, 4, 64, P, P, P) == arg and f(0, -1, 64, P, P, P) == shape and f(0, 4, 48, P, P, P) == shape
        assert f(0, 4, 0, P, P, P) == shape and f(0, 0, 64, None, None, None) == ok
        assert f(0, 4, 64, None, P, P) == arg and f(0, 4, 64, P, None, P) == arg and f(0, 4, 64, P, P, None) == arg
        assert f(0, 4, 64, ODD, P, P) == arg and f(0, 4, 64, P, ODD, P) == arg
        assert f(0, 2 ** 31 - 1, 32 * 2 ** 20, P, P, P) == shape

    def fwd(xdt=0, hdt=0, n=4, d=64, G=P, U=P, ld=64, H=P, gc=P, gs=P, uc=P, us=P):
        return L.wush_act8_swiglu(xdt, hdt, n, d, G, U, ld, H, gc, gs, uc, us, None)
    assert fwd(xdt=3) == arg and fwd(hdt=3) == arg and fwd(n=-2) == shape and fwd(d=40) == shape
    assert fwd(ld=56) == shape and fwd(ld=68) == shape and fwd(G=None) == arg and fwd(H=None) == arg
    assert fwd(gc=None) == arg and fwd(us=None) == arg and fwd(G=ODD) == arg and fwd(uc=ODD) == arg
    assert fwd(n=0) == ok

    def bwd(hdt=0, xdt=0, n=4, d=64, dH=P, gc=P, gs=P, uc=P, us=P, dG=P, dU=P, ld=64):
        return L.wush_act8_swiglu_bwd(hdt, xdt, n, d, dH, gc, gs, uc, us, dG, dU, ld, None)
    assert bwd(hdt=3) == arg and bwd(n=-2) == shape and bwd(d=40) == shape and bwd(ld=32) == shape
    assert bwd(gc=None) == arg and bwd(us=None) == arg and bwd(dG=None) == arg and bwd(dU=ODD) == arg
    assert bwd(n=0) == ok


def adapter(**kw):
    a = dict(xdt=1, ydt=0, n=4, d_in=64, d_out=64, X=P, ldx=64, nseg=2, off=P, ids=P, nad=2, rmax=16, A=P, Bt=P,
             rank=P, alpha=P, Y0=P, ldy0=64, Y=P, ldy=64, V=None, ws=P, wsb=1 << 30)
    a.update(kw)
    return L.wush_adapter_forward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(xdt=2), W.WUSH_E_ARG), (dict(ydt=2), W.WUSH_E_ARG), (dict(n=-1), W.WUSH_E_SHAPE),
    (dict(n=(1 << 24) + 1), W.WUSH_E_SHAPE), (dict(d_in=60), W.WUSH_E_SHAPE), (dict(d_out=4), W.WUSH_E_SHAPE),
    (dict(nseg=0), W.WUSH_E_SHAPE), (dict(nseg=(1 << 20) + 1), W.WUSH_E_SHAPE), (dict(nad=0), W.WUSH_E_SHAPE),
    (dict(rmax=8), W.WUSH_E_SHAPE), (dict(rmax=48), W.WUSH_E_SHAPE), (dict(rmax=256), W.WUSH_E_SHAPE),
    (dict(ldx=56), W.WUSH_E_SHAPE), (dict(ldx=68), W.WUSH_E_SHAPE), (dict(ldy=32), W.WUSH_E_SHAPE),
    (dict(ldy0=63), W.WUSH_E_SHAPE), (dict(n=1 << 24, d_out=1 << 23, ldy=1 << 23, ldy0=1 << 23), W.WUSH_E_SHAPE),
    (dict(X=None), W.WUSH_E_ARG), (dict(off=None), W.WUSH_E_ARG), (dict(ids=None), W.WUSH_E_ARG),
    (dict(A=None), W.WUSH_E_ARG), (dict(Bt=None), W.WUSH_E_ARG), (dict(rank=None), W.WUSH_E_ARG),
    (dict(alpha=None), W.WUSH_E_ARG), (dict(Y=None), W.WUSH_E_ARG), (dict(X=ODD), W.WUSH_E_ARG),
    (dict(Y0=ODD), W.WUSH_E_ARG), (dict(V=ODD), W.WUSH_E_ARG), (dict(ws=ODD), W.WUSH_E_ARG),
    (dict(wsb=8), W.WUSH_E_ARG)])
def test_adapter_forward_refusals(kw, status):
    assert adapter(**kw) == status
    assert L.wush_last_error().startswith(b"wush_adapter_forward:")


def adapter_bwd(**kw):
    a = dict(gdt=1, xdt=1, ydt=0, n=4, d_in=64, d_out=64, dY=P, ldg=64, X=P, xs=None, ldx=64, nseg=2, off=P, ids=P,
             nad=2, rmax=16, A=P, Bt=P, rank=P, alpha=P, V=P, dX0=P, ldd0=64, dX=P, ldd=64, dA=P, dBt=P, ws=P,
             wsb=1 << 30)
    a.update(kw)
    return L.wush_adapter_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(gdt=2), W.WUSH_E_ARG), (dict(xdt=2), W.WUSH_E_ARG), (dict(ydt=-1), W.WUSH_E_ARG),
    (dict(n=-1), W.WUSH_E_SHAPE), (dict(d_in=60), W.WUSH_E_SHAPE), (dict(rmax=24), W.WUSH_E_SHAPE),
    (dict(ldg=56), W.WUSH_E_SHAPE), (dict(ldx=100), W.WUSH_E_SHAPE), (dict(ldd=8), W.WUSH_E_SHAPE),
    (dict(ldd0=8), W.WUSH_E_SHAPE), (dict(xs=P, ldx=128), W.WUSH_E_SHAPE),
    (dict(xs=P, d_in=72, ldx=72, ldd=72, ldd0=72), W.WUSH_E_SHAPE), (dict(nad=1 << 17), W.WUSH_E_SHAPE),
    (dict(dY=None), W.WUSH_E_ARG), (dict(X=None), W.WUSH_E_ARG), (dict(V=None), W.WUSH_E_ARG),
    (dict(dA=None), W.WUSH_E_ARG), (dict(dBt=None), W.WUSH_E_ARG), (dict(alpha=None), W.WUSH_E_ARG),
    (dict(dY=ODD), W.WUSH_E_ARG), (dict(dX=ODD), W.WUSH_E_ARG), (dict(dA=ODD), W.WUSH_E_ARG),
    (dict(wsb=8), W.WUSH_E_ARG)])
def test_adapter_backward_refusals(kw, status):
    assert adapter_bwd(**kw) == status
    assert L.wush_last_error().startswith(b"wush_adapter_backward:")


def test_calls_past_the_launch_limit_are_refused():
    # 2^32 threads: a row of the norm has at least 64, 512 values of act8 have 64, 64 x 256 values of Y have 256
    assert norm(n=1 << 26) == W.WUSH_E_SHAPE and b"launch limit" in L.wush_last_error()
    assert L.wush_act8_pack(0, 1 << 26, 512, P, P, P, None) == W.WUSH_E_SHAPE and b"launch limit" in L.wush_last_error()
    wide = 1 << 22
    assert adapter(n=1 << 24, nseg=1, d_out=wide, ldy=wide, ldy0=wide) == W.WUSH_E_SHAPE
    assert b"launch limit" in L.wush_last_error()


def test_workspace_sizes_of_bad_shapes_are_zero():
    assert L.wush_block_norm_bwd_ws_bytes(0, 64) == 0 and L.wush_block_norm_bwd_ws_bytes(4, 12) == 0
    assert L.wush_block_norm_bwd_ws_bytes(1, 64) >= 3 * 64 * 4
    assert L.wush_adapter_ws_bytes(4, 60, 1, 16) == 0 and L.wush_adapter_ws_bytes(4, 64, 1, 17) == 0
    assert L.wush_adapter_ws_bytes(4, 64, 1, 16) >= 4 * 16 * 4
    assert L.wush_adapter_backward_ws_bytes(4, 64, 64, 0, 1, 16) == 0
    assert L.wush_adapter_backward_ws_bytes(0, 64, 64, 1, 1, 16) > 0


def test_binding_refuses_wrong_tensors():
    z = torch.zeros
    n, d = 4, 64
    bf, f32 = torch.bfloat16, torch.float32
    with pytest.raises(TypeError):
        W.wush_block_norm(None, None, None, z(n, d, dtype=torch.float16), z(d), None, z(n, d), stream=0)
    with pytest.raises(ValueError):
        W.wush_block_norm(z(n, d + 8), None, None, z(n, d), z(d), None, z(n, d), stream=0)
    with pytest.raises(ValueError):
        W.wush_block_norm(z(d, n).t(), None, None, z(n, d), z(d), None, z(n, d), stream=0)
    with pytest.raises(TypeError):
        W.wush_block_norm(z(n, d), z(d, dtype=bf), None, z(n, d), z(d), None, z(n, d), stream=0)
    with pytest.raises(ValueError):
        W.wush_block_norm(z(n, d), z(d), z(n + 1, 1), z(n, d), z(d), None, z(n, d), stream=0)
    c, s = z(n, d, dtype=torch.int8), z(n, d // 32, dtype=torch.uint8)
    with pytest.raises(TypeError):
        W.wush_act8_pack(z(n, d), c.view(torch.uint8), s, stream=0)
    with pytest.raises(ValueError):
        W.wush_act8_pack(z(n, d), c, s[:, :1], stream=0)
    with pytest.raises(ValueError):
        W.wush_act8_swiglu(z(n, 2 * d)[:, :d], z(n, d), z(n, d), stream=0)
    ids, off = z(2, dtype=torch.int32), z(3, dtype=torch.int32)
    A, B = z(1, 16, d, dtype=bf), z(1, 16, d, dtype=bf)
    rk, al = z(1, dtype=torch.int32), z(1)
    with pytest.raises(TypeError):
        W.wush_adapter_forward(z(n, d), off.long(), ids, A, B, rk, al, None, z(n, d), stream=0)
    with pytest.raises(TypeError):
        W.wush_adapter_forward(z(n, d), off, ids, A.to(f32), B, rk, al, None, z(n, d), stream=0)
    with pytest.raises(ValueError):
        W.wush_adapter_forward(z(n, d), off[:2], ids, A, B, rk, al, None, z(n, d), stream=0)
    with pytest.raises(TypeError):
        W.wush_adapter_forward(z(n, d), off, ids, A, B, rk, al, z(n, d, dtype=bf), z(n, d), stream=0)
    with pytest.raises(ValueError):
        W.wush_adapter_forward(z(d, n).t(), off, ids, A, B, rk, al, None, z(n, d), stream=0)


# ----------------------------------------------------------------------------- the 64-bit forms against differences
# With step h the centred difference of a smooth function is off by O(h^2) and 2^-53/h: 1e-8 at h = 1e-5.

H = 1e-5


def _slope(f, x, v):
    return (f(x + H * v) - f(x - H * v)) / (2 * H)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("post", [True, False])
def test_norm_gradient_against_differences(gate, post):
    r = np.random.default_rng([7, len(gate), post])
    n, d, branch, res, eps = 3, 24, 0.7, 0.9, 1e-3
    Y, R, cR, cU = (r.standard_normal((n, d)) for _ in range(4))
    wp, w = 1 + 0.3 * r.standard_normal(d), 1 + 0.3 * r.standard_normal(d)
    if not post:
        wp = None
    g = {"none": None, "channel": r.standard_normal(d), "token": r.standard_normal((n, 1)),
         "element": r.standard_normal((n, d))}[gate]

    def loss(Y=Y, R=R, wp=wp, w=w, g=g):
        o, U, _, _ = bo.block_norm(Y, wp, g, R, w, branch, res, eps)
        return (o * cR).sum() + (U * cU).sum()
    o, _, k1, k2 = bo.block_norm(Y, wp, g, R, w, branch, res, eps)
    grad = bo.block_norm_bwd(cU, cR, Y, wp, g, o, w, k1, k2, branch, res)
    pairs = [("Y", Y, grad["dY"]), ("R", R, grad["dR"]), ("w", w, grad["dw_pre"].sum(0))]
    if post:
        pairs.append(("wp", wp, grad["dw_post"].sum(0)))
    if g is not None:
        dg = grad["dgate"]
        pairs.append(("g", g, {"channel": dg.sum(0), "token": dg.sum(1, keepdims=True)}.get(gate, dg)))
    for name, x, gx in pairs:
        v = r.standard_normal(x.shape)
        assert abs(_slope(lambda t: loss(**{name: t}), x, v) - (gx * v).sum()) < 1e-6, name


def test_swiglu_gradient_against_differences():
    r = np.random.default_rng(8)
    G, U, c = (r.standard_normal((4, 32)) * 3 for _ in range(3))
    dG, dU = bo.swiglu_bwd(c, G, U)
    for x, gx, f in ((G, dG, lambda t: (bo.swiglu(t, U) * c).sum()), (U, dU, lambda t: (bo.swiglu(G, t) * c).sum())):
        v = r.standard_normal(x.shape)
        assert abs(_slope(f, x, v) - (gx * v).sum()) < 1e-6


def test_adapter_gradients_against_differences():
    r = np.random.default_rng(9)
    n, d_in, d_out, nad, rmax = 9, 16, 24, 3, 16
    off, ids, rank, alpha = [0, 2, 2, 6, 7, 9], [1, 0, 0, -1, 1], [3, 16, 5], [0.5, -2.0, 1.0]
    X, Y0, dX0, c = (r.standard_normal(s) for s in ((n, d_in), (n, d_out), (n, d_in), (n, d_out)))
    A, B = r.standard_normal((nad, rmax, d_in)), r.standard_normal((nad, rmax, d_out))

    def loss(X=X, A=A, B=B):
        return (bo.adapter_forward(X, off, ids, A, B, rank, alpha, Y0, d_out)[0][0] * c).sum()
    (_, V), _ = bo.adapter_forward(X, off, ids, A, B, rank, alpha, Y0, d_out)
    (dX, dA, dB), _ = bo.adapter_backward(c, X, off, ids, A, B, rank, alpha, V, None)
    for name, x, gx in (("X", X, dX), ("A", A, dA), ("B", B, dB)):
        v = r.standard_normal(x.shape)
        assert abs(_slope(lambda t: loss(**{name: t}), x, v) - (gx * v).sum()) < 1e-5, name
    assert not dA[2].any() and not dA[0, 3:].any()


def test_act8_definition():
    x = np.zeros((1, 32), np.float32)
    x[0, :6] = [1.0, -0.5, 1.0 / 128, 3.0 / 128, 127.6 / 64, -1.999]
    c, s = bo.act8_pack(x)
    assert s[0, 0] == 127 and list(c[0, :6]) == [64, -32, 0, 2, 127, -127]     # halves go to the even code
    assert list(bo.act8_values(c, s)[0, :3]) == [1.0, -0.5, 0.0]
    x[0, 7] = np.inf
    c, s = bo.act8_pack(x)
    assert s[0, 0] == 255 and not c.any() and np.isnan(bo.act8_values(c, s)).all()
