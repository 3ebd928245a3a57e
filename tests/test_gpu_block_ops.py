"""Block norm, act8 and adapters on the GPU against the 64-bit forms of oracle/block_ops.py.

Bounds.  An fp32 sum of K terms is off by at most (K - 1) 2^-24 times the sum of the terms' magnitudes, in whatever
order; the products, scales and roots around it add a few roundings of 2^-24 each.  So an fp32 result must lie within
(K + 32) 2^-24 M of the 64-bit one, with M the result computed from magnitudes (where two sums follow each other, K
counts both).  A bf16 result may be a further 2^-8 of its value away (half of that by rounding).  Codes and scale bytes
must be equal.
"""

import numpy as np
import pytest
import torch

import aware_block_transforms_amd as W
from oracle import block_ops as bo
from gpu_util import DEV, to_dev

pytestmark = pytest.mark.gpu

EPS24 = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def new(*shape, dt=torch.float32):
    return torch.full(shape, 99, dtype=dt, device=DEV) if dt in (torch.int8, torch.uint8) else \
        torch.full(shape, float("nan"), dtype=dt, device=DEV)


def dev(a, dt="f32"):
    return None if a is None else to_dev(np.asarray(a, np.float32)).to(DT[dt])


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, ref, mag, K, what):
    lim = (K + 32) * EPS24 * np.asarray(mag)
    if got.dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * (np.abs(ref) + lim)
    g = f64(got)
    assert g.shape == ref.shape, what
    bad = ~(np.abs(g - ref) <= lim + 1e-37)
    assert not bad.any(), (what, np.argwhere(bad)[:4], g[bad][:4], ref[bad][:4])


# ----------------------------------------------------------------------------- block norm

TYPES = [("f32", "bf16", "bf16"), ("f32", "f32", "bf16"), ("f32", "f32", "f32"), ("bf16", "bf16", "bf16"),
         ("bf16", "f32", "bf16"), ("bf16", "f32", "f32")]


def _norm_inputs(seed, n, d, types, gate, post=True):
    r = np.random.default_rng([seed, n, d])
    Y = dev(r.standard_normal((n, d)) * np.exp(r.standard_normal((n, 1))), types[0])
    R = dev(3 * r.standard_normal((n, d)), types[1])
    if n > 2:
        Y[1] = 0          # a row without a norm
        R[2] = 0
    g = {"none": None, "channel": dev(r.standard_normal(d)), "token": dev(r.standard_normal((n, 1))),
         "element": dev(r.standard_normal((n, d)), types[0])}[gate]
    wp = dev(1 + 0.2 * r.standard_normal(d)) if post else None
    return r, Y, wp, g, R, dev(1 + 0.2 * r.standard_normal(d))


def _norm_check(Y, wp, g, R, w, branch, res, eps, Rout, U, k1, k2, d):
    ref = bo.block_norm(f64(Y), f64(wp), f64(g), f64(R), f64(w), branch, res, eps)
    mag = np.abs(res * f64(R)) + (0 if Y is None else np.abs(ref[0] - res * f64(R)))
    if Rout is not None:
        near(Rout, ref[0], mag, d, "Rout")
    if w is not None:
        # both roots' relative error is bounded by that of their sums of squares; r' itself carries mag
        m = (mag + np.abs(ref[0]) + mag.max(axis=1, keepdims=True)) * ref[3][:, None] * np.abs(f64(w))
        near(U, ref[1], m, 2 * d, "U")
    if wp is not None and k1 is not None:
        near(k1, ref[2], ref[2], d, "rstd_post")
    if w is not None and k2 is not None:
        near(k2, ref[3], ref[3] * (1 + mag.max(axis=1) * ref[3]), 2 * d, "rstd_pre")


@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("types", TYPES)
def test_norm_types_and_gates(types, gate):
    for n, d in ((1, 8), (5, 520), (7, 2600)):
        _, Y, wp, g, R, w = _norm_inputs(1, n, d, types, gate)
        Rout, U = new(n, d, dt=DT[types[1]]), new(n, d, dt=DT[types[2]])
        k1, k2 = new(n), new(n)
        W.wush_block_norm(Y, wp, g, R, w, Rout, U, k1, k2, branch_scale=0.7, res_scale=0.9)
        torch.cuda.synchronize()
        _norm_check(Y, wp, g, R, w, np.float32(0.7), np.float32(0.9), np.float32(1e-6), Rout, U, k1, k2, d)


@pytest.mark.parametrize("d", [64, 4096, 8192, 8200, 12296, 16384, 16392, 17408, 24576])
def test_norm_widths(d):
    n = 3
    types = ("f32", "bf16", "bf16")
    r, Y, wp, g, R, w = _norm_inputs(2, n, d, types, "channel")
    Rout, U = new(n, d, dt=DT["bf16"]), new(n, d, dt=DT["bf16"])
    k1, k2 = new(n), new(n)
    W.wush_block_norm(Y, wp, g, R, w, Rout, U, k1, k2, branch_scale=1.5, res_scale=1.0)
    torch.cuda.synchronize()
    _norm_check(Y, wp, g, R, w, 1.5, 1.0, np.float32(1e-6), Rout, U, k1, k2, d)
    _norm_grads(r, Y, wp, g, R, w, types, 1.5, 1.0, d)


def test_norm_parts_left_out():
    n, d, types = 6, 264, ("f32", "f32", "bf16")
    _, Y, wp, g, R, w = _norm_inputs(3, n, d, types, "channel")
    for y, p, gate, pre, keep in ((None, None, None, w, True), (None, None, None, w, False), (Y, None, g, w, True),
                                  (Y, wp, None, None, True), (Y, None, None, None, True), (Y, wp, g, w, False)):
        Rout = new(n, d) if keep else None
        U = None if pre is None else new(n, d, dt=DT["bf16"])
        W.wush_block_norm(y, p, gate, R, pre, Rout, U, branch_scale=-0.5, res_scale=2.0)
        torch.cuda.synchronize()
        _norm_check(y, p, gate, R, pre, -0.5, 2.0, np.float32(1e-6), Rout, U, None, None, d)


def test_norm_in_place_and_rows_apart():
    n, d, types = 5, 1032, ("bf16", "bf16", "bf16")
    _, Y, wp, g, R, w = _norm_inputs(4, n, d, types, "element")
    want, U, U2 = new(n, d, dt=DT["bf16"]), new(n, d, dt=DT["bf16"]), new(n, d, dt=DT["bf16"])
    W.wush_block_norm(Y, wp, g, R, w, want, U)
    Y2, R2 = Y.clone(), R.clone()
    Y2[2, 5], Y2[3, 7] = float("nan"), float("inf")     # two bad rows leave the others as they were
    W.wush_block_norm(Y2, wp, g, R2, w, R2, U2)
    torch.cuda.synchronize()
    for i in (0, 1, 4):
        assert torch.equal(R2[i], want[i]) and torch.equal(U2[i], U[i])
    assert not torch.isfinite(U2[2]).any() and torch.isnan(U2[3]).any()


def _norm_grads(r, Y, wp, g, R, w, types, branch, res, d, du=True, dr=True, want_dR=True):
    n = R.shape[0]
    Rout, U = new(n, d, dt=DT[types[1]]), None if w is None else new(n, d, dt=DT[types[2]])
    k1, k2 = new(n), new(n)
    W.wush_block_norm(Y, wp, g, R, w, Rout, U, k1, k2, branch_scale=branch, res_scale=res)
    dU = dev(r.standard_normal((n, d)), types[2]) if w is not None else None
    dRo = dev(r.standard_normal((n, d)), types[1]) if dr else None
    dY = None if Y is None else torch.full_like(Y, float("nan"))
    dR = torch.full_like(R, float("nan")) if want_dR else None
    dg = None if g is None else torch.full_like(g, float("nan"))
    dwp, dw = (None if wp is None else new(d)), (None if w is None else new(d))
    ws = torch.full((max(16, W.wush_block_norm_bwd_ws_bytes(n, d)),), 0xFF, dtype=torch.uint8, device=DEV)
    args = (dU, dRo, Y, wp, g, Rout, w, k1 if wp is not None else None, k2 if w is not None else None)
    W.wush_block_norm_bwd(*args, dY, dR, dg, dwp, dw, branch_scale=branch, res_scale=res, ws=ws)
    torch.cuda.synchronize()
    a = [f64(t) for t in args]
    ref = bo.block_norm_bwd(*a, branch, res)
    # magnitudes: |t| and the row sums behind it, carried through the products
    t = np.zeros((n, d)) if dRo is None else np.abs(a[1])
    if w is not None:
        xh, q = np.abs(a[5] * a[8][:, None]), np.abs(a[0] * a[6])
        t = t + np.abs(a[8])[:, None] * (q + xh * np.mean(q * xh, axis=1, keepdims=True))
        near(dw, ref["dw_pre"].sum(0), np.abs(ref["dw_pre"]).sum(0), n, "dw_pre")
    if dR is not None:
        near(dR, ref["dR"], abs(res) * t, d, "dR")
    if Y is None:
        return
    z = np.abs(a[2]) if wp is None else np.abs(a[2] * a[7][:, None])
    wz = z if wp is None else z * np.abs(a[3])
    mg = abs(branch) * t * wz
    gg = 1.0 if g is None else np.abs(a[4])
    p = abs(branch) * t * gg * (1.0 if wp is None else np.abs(a[3]))
    if wp is None:
        near(dY, ref["dY"], p, d, "dY")
    else:
        near(dY, ref["dY"], a[7][:, None] * (p + z * np.mean(p * z, axis=1, keepdims=True)), 2 * d, "dY")
        near(dwp, ref["dw_post"].sum(0), (abs(branch) * t * gg * z).sum(0), n + d, "dw_post")
    if g is not None:
        if g.dim() == 1:
            near(dg, ref["dgate"].sum(0), mg.sum(0), n + d, "dgate")
        elif g.shape[1] == 1:
            near(dg, ref["dgate"].sum(1, keepdims=True), mg.sum(1, keepdims=True), 2 * d, "dgate")
        else:
            near(dg, ref["dgate"], mg, d, "dgate")


@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("types", TYPES)
def test_norm_gradients(types, gate):
    for n, d in ((1, 8), (300, 520), (9, 2600), (4000, 64)):
        r, Y, wp, g, R, w = _norm_inputs(5, n, d, types, gate)
        _norm_grads(r, Y, wp, g, R, w, types, 0.75, 1.25, d)


def test_norm_gradients_parts_left_out():
    n, d, types = 600, 136, ("bf16", "bf16", "bf16")
    r, Y, wp, g, R, w = _norm_inputs(6, n, d, types, "token")
    _norm_grads(r, None, None, None, R, w, types, 1.0, 0.5, d)
    _norm_grads(r, None, None, None, R, w, types, 1.0, 0.5, d, dr=False)
    _norm_grads(r, Y, None, g, R, w, types, 1.0, 0.5, d)
    _norm_grads(r, Y, wp, g, R, None, types, 1.0, 0.5, d)
    _norm_grads(r, Y, None, None, R, None, types, 1.0, 0.5, d, want_dR=False)


def test_norm_gradient_of_no_rows_clears_the_sums():
    d = 64
    z = torch.zeros((0, d), device=DEV)
    dwp, dw = new(d), new(d)
    e = torch.zeros(0, device=DEV)
    W.wush_block_norm_bwd(z, z, z, dev(np.ones(d)), None, z, dev(np.ones(d)), e, e, z.clone(), z.clone(), None, dwp, dw)
    torch.cuda.synchronize()
    assert not dwp.any() and not dw.any()


def test_norm_gradient_against_differences():
    # the slope of a loss along a direction, from the 64-bit form, against the kernel's gradients
    r = np.random.default_rng(77)
    n, d, branch, res, eps, h = 5, 264, 0.5, 1.0, np.float32(1e-3), 1e-5
    Y, R, cR, cU = (dev(r.standard_normal((n, d))) for _ in range(4))
    wp, w, g = (dev(1 + 0.3 * r.standard_normal(d)) for _ in range(3))
    Rout, U, k1, k2 = new(n, d), new(n, d), new(n), new(n)
    W.wush_block_norm(Y, wp, g, R, w, Rout, U, k1, k2, branch_scale=branch, res_scale=res, eps=eps)
    dY, dR, dg, dwp, dw = new(n, d), new(n, d), new(d), new(d), new(d)
    W.wush_block_norm_bwd(cU, cR, Y, wp, g, Rout, w, k1, k2, dY, dR, dg, dwp, dw, branch_scale=branch, res_scale=res)
    torch.cuda.synchronize()
    base = dict(Y=f64(Y), w_post=f64(wp), gate=f64(g), R=f64(R), w_pre=f64(w))

    def loss(**kw):
        o, u, _, _ = bo.block_norm(**{**base, **kw}, branch=branch, res=res, eps=float(eps))
        return (o * f64(cR)).sum() + (u * f64(cU)).sum()
    for name, grad in (("Y", dY), ("R", dR), ("gate", dg), ("w_post", dwp), ("w_pre", dw)):
        v = r.standard_normal(base[name].shape)
        slope = (loss(**{name: base[name] + h * v}) - loss(**{name: base[name] - h * v})) / (2 * h)
        mag = np.abs(f64(grad) * v).sum()
        assert abs(slope - (f64(grad) * v).sum()) <= (2 * d + n + 64) * EPS24 * mag + 1e-6, name


# ----------------------------------------------------------------------------- act8


def _awkward(seed, n, d):
    r = np.random.default_rng([seed, n, d])
    X = (r.standard_normal((n, d)) * np.exp(8 * r.standard_normal((n, d // 32))).repeat(32, axis=1)).astype(np.float32)
    v = X.reshape(-1, 32)
    k = v.shape[0]
    rows = [np.zeros(32), np.full(32, -0.0), np.full(32, 1e-40), np.full(32, 3.4e38), np.full(32, 2.0 ** -120),
            np.full(32, 2.0 ** -126), np.arange(32) * 2.0 ** -7 + 2.0 ** -8, np.full(32, 127.5 / 64),
            np.full(32, np.nextafter(np.float32(2), np.float32(0))), np.where(np.arange(32) == 3, np.inf, 1.0),
            np.where(np.arange(32) == 31, np.nan, 1.0), np.where(np.arange(32) == 0, -np.inf, 0.0)]
    for i, row in enumerate(rows[:k]):
        v[(i * 7) % k if k >= 84 else i] = row
    return X


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", [(1, 32), (3, 96), (61, 544), (130, 4096), (5, 17408)])
def test_act8_pack_and_unpack(n, d, dt):
    X = dev(_awkward(11, n, d), dt)
    c, s = new(n, d, dt=torch.int8), new(n, d // 32, dt=torch.uint8)
    W.wush_act8_pack(X, c, s)
    outs = {k: new(n, d, dt=v) for k, v in DT.items()}
    for y in outs.values():
        W.wush_act8_unpack(c, s, y)
    torch.cuda.synchronize()
    rc, rs = bo.act8_pack(X.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(c.cpu().numpy(), rc)
    ref = bo.act8_values(rc, rs)
    for y in outs.values():
        assert np.array_equal(f64(y), ref, equal_nan=True)


@pytest.mark.parametrize("hdt", ["f32", "bf16"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,d,split", [(1, 32, False), (7, 544, True), (65, 1024, True), (2, 17408, False)])
def test_swiglu(n, d, split, dt, hdt):
    r = np.random.default_rng([12, n, d])
    x = dev(r.standard_normal((n, 2 * d)) * 4, dt)
    x[0, :4] = torch.tensor([-90.0, -30.0, 30.0, 90.0], device=DEV)
    G, U = (x[:, :d], x[:, d:]) if split else (x[:, :d].contiguous(), x[:, d:].contiguous())
    H, H2 = new(n, d, dt=DT[hdt]), new(n, d, dt=DT[hdt])
    gc, uc = new(n, d, dt=torch.int8), new(n, d, dt=torch.int8)
    gs, us = new(n, d // 32, dt=torch.uint8), new(n, d // 32, dt=torch.uint8)
    W.wush_act8_swiglu(G, U, H, gc, gs, uc, us)
    W.wush_act8_swiglu(G, U, H2)
    dH = dev(r.standard_normal((n, d)), hdt)
    out = torch.full((n, 2 * d), float("nan"), dtype=DT[dt], device=DEV)
    dG, dU = (out[:, :d], out[:, d:]) if split else (new(n, d, dt=DT[dt]), new(n, d, dt=DT[dt]))
    W.wush_act8_swiglu_bwd(dH, gc, gs, uc, us, dG, dU)
    torch.cuda.synchronize()
    assert torch.equal(H, H2)
    for t, c, s in ((G, gc, gs), (U, uc, us)):
        rc, rs = bo.act8_pack(t.float().cpu().numpy())
        assert np.array_equal(c.cpu().numpy(), rc) and np.array_equal(s.cpu().numpy(), rs)
    # exp(-g) carries the rounding of 1.44 g, so |g| counts into its relative error; below g = -88 it overflows and
    # the sigmoid, at most 1e-38 there, becomes zero
    g, u = f64(G), f64(U)
    near(H, bo.swiglu(g, u), np.abs(bo.swiglu(g, u)) + 1e-30 * np.abs(u), 3 * np.abs(g), "H")
    gv, uv = (bo.act8_values(*(t.cpu().numpy() for t in p)) for p in ((gc, gs), (uc, us)))
    rg, ru = bo.swiglu_bwd(f64(dH), gv, uv)
    s = bo.sigmoid(gv)
    near(dU, ru, np.abs(ru) + 1e-30 * np.abs(f64(dH)), 3 * np.abs(gv), "dU")
    near(dG, rg, np.abs(f64(dH) * uv) * (s * (1 + np.abs(gv)) + 1e-30), 3 * np.abs(gv), "dG")


def test_swiglu_keeps_bad_groups_apart():
    n, d = 2, 96
    x = torch.ones((n, d), device=DEV)
    G = x.clone()
    G[0, 40] = float("nan")
    H, gc, uc = new(n, d), new(n, d, dt=torch.int8), new(n, d, dt=torch.int8)
    gs, us = new(n, 3, dt=torch.uint8), new(n, 3, dt=torch.uint8)
    W.wush_act8_swiglu(G, x, H, gc, gs, uc, us)
    dG, dU = new(n, d), new(n, d)
    W.wush_act8_swiglu_bwd(x, gc, gs, uc, us, dG, dU)
    torch.cuda.synchronize()
    assert torch.isnan(H).sum() == 1
    for t in (dG, dU):
        assert torch.isnan(t[0, 32:64]).all() and torch.isnan(t).sum() == 32


# ----------------------------------------------------------------------------- adapters


def _requests(r, n, nseg, nad, kind):
    if kind == "single":
        off = list(range(n + 1))
        ids = [int(r.integers(nad)) for _ in range(n)]
    else:
        off = [0] + sorted(int(v) for v in r.integers(0, n + 1, nseg - 1)) + [n]
        ids = [int(r.integers(nad)) for _ in range(nseg)]
    if len(ids) > 2:
        ids[1], ids[-1] = -1, nad + 5           # no adapter
    return off, ids


class Case:
    def __init__(self, seed, n, d_in, d_out, nseg, nad, rmax, xdt="bf16", ydt="f32", kind="ragged", ranks=None):
        r = self.r = np.random.default_rng([seed, n, d_in, d_out, rmax])
        self.n, self.d_in, self.d_out, self.nad, self.rmax = n, d_in, d_out, nad, rmax
        self.off, self.ids = _requests(r, n, nseg, nad, kind)
        pool = [rmax, rmax // 2 + 1, 1, 0, 7]
        self.rank = ranks or [pool[i % len(pool)] for i in range(nad)]
        self.alpha = (r.standard_normal(nad) * 2).astype(np.float32)
        self.A = dev(r.standard_normal((nad, rmax, d_in)) * d_in ** -0.5, "bf16")
        self.B = dev(r.standard_normal((nad, rmax, d_out)) * 0.1, "bf16")
        for a, k in enumerate(self.rank):       # rows that do not count hold anything
            self.A[a, k:], self.B[a, k:] = float("nan"), float("inf")
        self.X = dev(r.standard_normal((n, d_in)), xdt)
        self.Y0 = dev(r.standard_normal((n, d_out)), ydt)
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
        self.dev = (i32(self.off), i32(self.ids), self.A, self.B, i32(self.rank), to_dev(self.alpha))

    def plain(self):
        return (self.off, self.ids, np.nan_to_num(f64(self.A), posinf=0, neginf=0),
                np.nan_to_num(f64(self.B), posinf=0, neginf=0), self.rank, self.alpha.astype(np.float64))

    def forward(self, Y0="own", ws=True, keep=True):
        y0 = self.Y0 if isinstance(Y0, str) else Y0
        Y = torch.full_like(self.Y0, float("nan"))
        V = new(self.n, self.rmax) if keep else None
        w = None
        if ws:
            need = W.wush_adapter_ws_bytes(self.n, self.d_in, len(self.ids), self.rmax)
            w = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device=DEV)
        W.wush_adapter_forward(self.X, *self.dev, y0, Y, V=V, ws=w)
        torch.cuda.synchronize()
        return Y, V

    def check(self, Y, V, y0=None):
        ref, mag = bo.adapter_forward(f64(self.X), *self.plain(), None if y0 is None else f64(y0), self.d_out)
        near(Y, ref[0], mag[0], self.d_in + self.rmax, "Y")
        if V is not None:
            near(V, ref[1], mag[1], self.d_in, "V")


@pytest.mark.parametrize("rmax", [16, 32, 64, 128])
@pytest.mark.parametrize("xdt,ydt", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_adapter_forward(xdt, ydt, rmax):
    for i, (n, d_in, d_out, nseg, nad, kind) in enumerate([
            (1, 8, 8, 1, 1, "ragged"), (1, 4096, 136, 1, 3, "single"), (70, 264, 520, 70, 5, "single"),
            (150, 520, 264, 9, 5, "ragged"), (333, 96, 1032, 5, 2, "ragged"), (40, 1096, 24, 12, 7, "ragged")]):
        c = Case(20 + i, n, d_in, d_out, nseg, nad, rmax, xdt, ydt, kind)
        Y, V = c.forward()
        c.check(Y, V, c.Y0)


def test_adapter_base_absent_and_in_place():
    c = Case(30, 90, 264, 136, 6, 3, 32)
    Y, V = c.forward(Y0=None, ws=False)
    c.check(Y, V, None)
    want, _ = c.forward(keep=False)
    Y = c.Y0.clone()
    W.wush_adapter_forward(c.X, *c.dev, Y, Y)
    torch.cuda.synchronize()
    assert torch.equal(Y, want)


def test_adapter_rows_inside_wider_tensors():
    # a slice of a fused projection's output, and of a wider input
    c = Case(31, 77, 264, 136, 5, 3, 16, ydt="bf16")
    want, _ = c.forward()
    big = torch.full((77, 400), 5.0, dtype=torch.bfloat16, device=DEV)
    wide = torch.full((77, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 64:328] = c.X
    W.wush_adapter_forward(wide[:, 64:328], *c.dev, c.Y0, big[:, 200:336])
    torch.cuda.synchronize()
    assert torch.equal(big[:, 200:336], want)
    assert (big[:, :200] == 5).all() and (big[:, 336:] == 5).all()


def test_adapter_tokens_stay_apart():
    c = Case(32, 40, 264, 136, 4, 3, 16, ranks=[16, 16, 16])
    want, wv = c.forward()
    c.X[5, 3] = float("nan")
    Y, V = c.forward()
    rows = [i for i in range(40) if i != 5]
    assert torch.equal(Y[rows], want[rows]) and torch.equal(V[rows], wv[rows])


@pytest.mark.parametrize("rmax", [16, 32, 64, 128])
@pytest.mark.parametrize("xdt,gdt,ydt", [("bf16", "bf16", "bf16"), ("act8", "bf16", "bf16"), ("f32", "f32", "f32"),
                                         ("act8", "f32", "f32"), ("bf16", "f32", "bf16"), ("f32", "bf16", "f32")])
def test_adapter_backward(xdt, gdt, ydt, rmax):
    for i, (n, d_in, d_out, nseg, nad, kind) in enumerate([
            (1, 32, 8, 1, 1, "ragged"), (70, 288, 520, 70, 5, "single"), (150, 544, 264, 9, 6, "ragged"),
            (3000, 160, 136, 20, 2, "ragged")]):
        c = Case(40 + i, n, d_in, d_out, nseg, nad, rmax, "f32" if xdt == "f32" else "bf16", "f32", kind)
        X, xs, xv = c.X, None, f64(c.X)
        if xdt == "act8":
            codes, xs = new(n, d_in, dt=torch.int8), new(n, d_in // 32, dt=torch.uint8)
            W.wush_act8_pack(c.X, codes, xs)
            X, xv = codes, bo.act8_values(codes.cpu().numpy(), xs.cpu().numpy())
        dY = dev(c.r.standard_normal((n, d_out)), gdt)
        dX0 = dev(c.r.standard_normal((n, d_in)), ydt)
        _, V = c.forward()
        for base in (True, False):
            dX = torch.full_like(dX0, float("nan"))
            dA, dB = new(nad, rmax, d_in), new(nad, rmax, d_out)
            need = W.wush_adapter_backward_ws_bytes(n, d_in, d_out, len(c.ids), nad, rmax)
            ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
            W.wush_adapter_backward(dY, X, *c.dev, V, dX0 if base else None, dX, dA, dB, x_scales=xs, ws=ws)
            torch.cuda.synchronize()
            ref, mag = bo.adapter_backward(f64(dY), xv, *c.plain(), f64(V), f64(dX0) if base else None)
            near(dX, ref[0], mag[0], d_out + rmax, "dX")
            near(dA, ref[1], mag[1], d_out + n, "dA")
            near(dB, ref[2], mag[2], n, "dBt")
        # without dX the same sums, and twice the same bits
        dA2, dB2 = new(nad, rmax, d_in), new(nad, rmax, d_out)
        W.wush_adapter_backward(dY, X, *c.dev, V, None, None, dA2, dB2, x_scales=xs)
        torch.cuda.synchronize()
        assert torch.equal(dA, dA2) and torch.equal(dB, dB2)


def test_adapter_backward_of_no_tokens():
    c = Case(50, 8, 64, 64, 2, 3, 16)
    z = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV)
    dA, dB = new(3, 16, 64), new(3, 16, 64)
    W.wush_adapter_backward(z, z, torch.zeros(3, dtype=torch.int32, device=DEV), *c.dev[1:], new(0, 16), None, None, dA,
                            dB)
    torch.cuda.synchronize()
    assert not dA.any() and not dB.any()


def test_adapter_gradients_against_differences():
    # slopes of a loss from the 64-bit form; the loss is linear in X and in each factor, so centred differences are
    # exact up to their own rounding
    c = Case(51, 33, 96, 136, 4, 2, 16, xdt="f32", ranks=[16, 9])
    dY = dev(c.r.standard_normal((33, 136)))
    _, V = c.forward()
    dX, dA, dB = new(33, 96), new(2, 16, 96), new(2, 16, 136)
    W.wush_adapter_backward(dY, c.X, *c.dev, V, None, dX, dA, dB)
    torch.cuda.synchronize()
    off, ids, A, B, rank, alpha = c.plain()
    base = dict(X=f64(c.X), A=A, B=B)

    def loss(**kw):
        k = {**base, **kw}
        return (bo.adapter_forward(k["X"], off, ids, k["A"], k["B"], rank, alpha, None, 136)[0][0] * f64(dY)).sum()
    for name, g in (("X", dX), ("A", dA), ("B", dB)):
        v = c.r.standard_normal(base[name].shape)
        slope = (loss(**{name: base[name] + v}) - loss(**{name: base[name] - v})) / 2
        mag = np.abs(f64(g) * v).sum()
        assert abs(slope - (f64(g) * v).sum()) <= (136 + 33 + 96 + 64) * EPS24 * 8 * mag, name


# ----------------------------------------------------------------------------- streams, graphs, long tensors


def test_calls_follow_their_stream_and_replay_in_a_graph():
    c = Case(60, 64, 544, 520, 64, 4, 32, kind="single")
    d = c.d_out
    R, w = dev(c.r.standard_normal((64, d))), dev(np.ones(d))
    Y, Rout, U, H = torch.empty_like(c.Y0), new(64, d), new(64, d), new(64, 256)
    codes, sc = new(64, 544, dt=torch.int8), new(64, 17, dt=torch.uint8)
    gc, uc, gs, us = new(64, 256, dt=torch.int8), new(64, 256, dt=torch.int8), new(64, 8, dt=torch.uint8), \
        new(64, 8, dt=torch.uint8)
    ws = torch.empty(W.wush_adapter_ws_bytes(64, 544, 64, 32), dtype=torch.uint8, device=DEV)
    wb = torch.empty(W.wush_adapter_backward_ws_bytes(64, 544, d, 64, 4, 32), dtype=torch.uint8, device=DEV)
    V, dX, dA, dB = new(64, 32), new(64, 544), new(4, 32, 544), new(4, 32, d)

    def step():
        W.wush_act8_pack(c.X, codes, sc)
        W.wush_adapter_forward(c.X, *c.dev, c.Y0, Y, V=V, ws=ws)
        W.wush_block_norm(Y, w, None, R, w, Rout, U)
        W.wush_act8_swiglu(U[:, :256], U[:, 256:512], H, gc, gs, uc, us)
        W.wush_adapter_backward(U, codes, *c.dev, V, None, dX, dA, dB, x_scales=sc, ws=wb)
    outs = (codes, sc, Y, Rout, U, H, V, dX, dA, dB)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in outs:
            t.zero_()
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for t in outs:
            t.zero_()
        c.X.mul_(1.0 if i < 2 else 0.5)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        step()                                   # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs)), i


def test_offsets_beyond_32_bits():
    # 2.4e9 values: byte and element offsets pass 2^32 and 2^31; the last rows are compared with a short call's
    n, d, k = 140000, 17408, 40
    X = torch.empty((n, d), dtype=torch.bfloat16, device=DEV)
    X.fill_(0.5)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    tail = torch.randn((k, d), generator=g, device=DEV).to(torch.bfloat16)
    X[n - k:] = tail
    c, s = torch.empty((n, d), dtype=torch.int8, device=DEV), torch.empty((n, d // 32), dtype=torch.uint8, device=DEV)
    W.wush_act8_pack(X, c, s)
    c2, s2 = c[:k].clone(), s[:k].clone()
    W.wush_act8_pack(tail, c2, s2)
    assert torch.equal(c[n - k:], c2) and torch.equal(s[n - k:], s2)
    Y = torch.empty_like(X)
    W.wush_act8_unpack(c, s, Y)
    y2 = torch.empty_like(tail)
    W.wush_act8_unpack(c2, s2, y2)
    assert torch.equal(Y[n - k:], y2)
    del c, s
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    A = torch.randn((1, 16, d), generator=g, device=DEV).mul_(0.01).to(torch.bfloat16)
    rank, alpha = i32([16]), torch.ones(1, device=DEV)
    W.wush_adapter_forward(X, i32([0, n]), i32([0]), A, A, rank, alpha, X, Y)
    W.wush_adapter_forward(tail, i32([0, k]), i32([0]), A, A, rank, alpha, tail, y2)
    # the split of k differs with n, so the fp32 sums may differ in their last bits: one bf16 step at most
    assert ((Y[n - k:].float() - y2.float()).abs() <= 2.0 ** -7 * y2.float().abs() + 1e-6).all()
    w = torch.ones(d, device=DEV)
    U = torch.empty_like(X)
    W.wush_block_norm(X, w, None, X, w, None, U)
    W.wush_block_norm(tail, w, None, tail, w, None, y2)
    torch.cuda.synchronize()
    assert torch.equal(U[n - k:], y2)


def test_gradient_offsets_beyond_32_bits():
    # 2.4e9 values of X, only the last tokens with a gradient: the sums are those of a short call on them
    n, d, k = 140000, 17408, 40
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    tail = torch.randn((k, d), generator=g, device=DEV).to(torch.bfloat16)
    X = torch.full((n, d), 0.5, dtype=torch.bfloat16, device=DEV)
    X[n - k:] = tail
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    A = torch.randn((1, 16, d), generator=g, device=DEV).mul_(0.01).to(torch.bfloat16)
    Bt = torch.randn((1, 16, 64), generator=g, device=DEV).mul_(0.1).to(torch.bfloat16)
    rank, alpha = i32([16]), torch.ones(1, device=DEV)
    dY, V = torch.zeros((n, 64), device=DEV), torch.zeros((n, 16), device=DEV)
    dY[n - k:] = torch.randn((k, 64), generator=g, device=DEV)
    V[n - k:] = torch.randn((k, 16), generator=g, device=DEV)
    c, s = torch.empty((n, d), dtype=torch.int8, device=DEV), torch.empty((n, d // 32), dtype=torch.uint8, device=DEV)
    W.wush_act8_pack(X, c, s)
    for x, xs, xt in ((X, None, tail.double()), (c, s, bo.act8_values(c[n - k:].cpu().numpy(), s[n - k:].cpu().numpy()))):
        dA, dB = new(1, 16, d), new(1, 16, 64)
        W.wush_adapter_backward(dY, x, i32([0, n]), i32([0]), A, Bt, rank, alpha, V, None, None, dA, dB, x_scales=xs)
        torch.cuda.synchronize()
        xt = f64(xt) if torch.is_tensor(xt) else xt
        ref, mag = bo.adapter_backward(f64(dY[n - k:]), xt, [0, k], [0], f64(A), f64(Bt), [16], [1.0], f64(V[n - k:]), None)
        near(dA, ref[1], mag[1], 64 + k, "dA")
        near(dB, ref[2], mag[2], k, "dBt")


def test_nothing_to_do():
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
    w = z(64)
    W.wush_block_norm(z(0, 64), w, None, z(0, 64), w, z(0, 64), z(0, 64))
    W.wush_act8_pack(z(0, 64), z(0, 64, dt=torch.int8), z(0, 2, dt=torch.uint8))
    W.wush_act8_swiglu(z(0, 64), z(0, 64), z(0, 64))
    A = z(1, 16, 64, dt=torch.bfloat16)
    W.wush_adapter_forward(z(0, 64), z(2, dt=torch.int32), z(1, dt=torch.int32), A, A, z(1, dt=torch.int32), z(1), None,
                           z(0, 64))
    torch.cuda.synchronize()


def test_tokens_without_an_adapter_are_not_read():
    # NaN in the rows of requests without an adapter reaches nothing but their own base values
    c = Case(70, 200, 264, 136, 5, 2, 32, ranks=[32, 17])
    c.off, c.ids = [0, 60, 61, 130, 180, 200], [0, -1, 1, 7, 0]
    c.dev = (torch.tensor(c.off, dtype=torch.int32, device=DEV), torch.tensor(c.ids, dtype=torch.int32, device=DEV)) + c.dev[2:]
    clean, cv = c.forward()
    dY = dev(c.r.standard_normal((200, 136)), "bf16")
    out = []
    for bad in (False, True):
        if bad:
            c.X[60], c.X[130:180], dY[60], dY[130:180] = float("nan"), float("inf"), float("inf"), float("nan")
            Y, V = c.forward()
            assert torch.equal(Y, clean) and torch.equal(V, cv)
        dX, dA, dB = new(200, 264), new(2, 32, 264), new(2, 32, 136)
        W.wush_adapter_backward(dY, c.X, *c.dev, cv, None, dX, dA, dB)
        torch.cuda.synchronize()
        out.append((dX, dA, dB))
    assert all(torch.equal(a, b) for a, b in zip(*out))
