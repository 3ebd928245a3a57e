"""Block norm, act8 and adapters on the GPU at their edges: infinities, wide rows in numbers, many adapters, outputs
beyond the last-level cache, streams and graphs.

Bounds are those of test_gpu_block_ops: (K + 32) 2^-24 times the result computed from magnitudes, and 2^-8 of its value
for bf16 results.
"""

import os
import sys

import numpy as np
import pytest
import torch

import aware_block_transforms_amd as W
from aware_block_transforms_amd.layer import AdapterSet, W4A4Layer, request_table
from oracle import block_ops as bo
from gpu_util import DEV
from test_gpu_block_ops import DT, TYPES, Case, _norm_check, _norm_grads, _norm_inputs, dev, f64, near, new

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def same_kind(got, ref):
    """NaN where the definition has NaN, and its infinities."""
    g = f64(got)
    return np.array_equal(np.isnan(g), np.isnan(ref)) and np.array_equal(np.where(np.isinf(g), g, 0),
                                                                        np.where(np.isinf(ref), ref, 0))


# ----------------------------------------------------------------------------- block norm


@pytest.mark.parametrize("d", [264, 512, 520, 2600, 4104])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
def test_norm_gradient_of_an_infinity_in_the_last_column(gate, d):
    # the row's gradients are the definition's, infinite or NaN, whether or not threads lie past the last column; the
    # other rows stay as they were
    n, types = 3, ("f32", "f32", "f32")
    r, Y, wp, g, R, w = _norm_inputs(101, n, d, types, gate)
    Y[1], R[2] = dev(r.standard_normal(d)), dev(r.standard_normal(d))
    Rout, U, k1, k2 = new(n, d), new(n, d), new(n), new(n)
    W.wush_block_norm(Y, wp, g, R, w, Rout, U, k1, k2)

    def grads(dU, dRo):
        dY, dR, dg, dwp, dw = new(n, d), new(n, d), None if g is None else torch.full_like(g, 7.0), new(d), new(d)
        W.wush_block_norm_bwd(dU, dRo, Y, wp, g, Rout, w, k1, k2, dY, dR, dg, dwp, dw)
        torch.cuda.synchronize()
        return dY, dR, dg
    clean = [dev(r.standard_normal((n, d))) for _ in range(2)]
    want = grads(*clean)
    for which in (0, 1):
        bad = [t.clone() for t in clean]
        bad[which][1, d - 1] = float("inf")
        dY, dR, dg = grads(*bad)
        for t, o in zip((dY, dR), want):
            assert torch.equal(t[[0, 2]], o[[0, 2]])
        with np.errstate(invalid="ignore"):
            ref = bo.block_norm_bwd(f64(bad[0]), f64(bad[1]), f64(Y), f64(wp), f64(g), f64(Rout), f64(w), f64(k1),
                                    f64(k2), 1.0, 1.0)
            row = {"token": ref["dgate"].sum(1, keepdims=True), "channel": ref["dgate"].sum(0)}.get(gate, ref["dgate"])
        assert same_kind(dR, ref["dR"]) and same_kind(dY, ref["dY"])
        assert g is None or same_kind(dg, row)


# ----------------------------------------------------------------------------- streams and graphs


def _adapter_set(seed, d_in, d_out, nad=3, rmax=32):
    ad = AdapterSet(nad, rmax, d_in, d_out, rank=[rmax, 7, rmax // 2][:nad], alpha=[1.0, -0.5, 2.0][:nad], seed=seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ad.Bt.copy_(torch.randn(ad.Bt.shape, generator=g, device=DEV) * 0.1)

    def batch(lengths, ids):
        n = sum(lengths)
        rand = lambda d: torch.randn((n, d), generator=g, device=DEV)  # noqa: E731
        return rand(d_in).to(torch.bfloat16), request_table(lengths, ids), rand(d_out), rand(d_out).to(torch.bfloat16)
    return ad, batch


def _pass(ad, b):
    X, req, Y0, dY = b
    Y, V = ad.forward(X, req, Y0, keep=True)
    return (Y, V) + ad.backward(dY, X, req, V)


def test_one_adapter_set_on_two_streams():
    ad, batch = _adapter_set(201, 4096, 2048)
    work = [batch([300, 0, 500, 17], [0, 1, 2, -1]), batch([1] * 40, [0, 1, 2, -1] * 10)]
    want = [_pass(ad, b) for b in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = []
    for turn in range(10):
        for s, b in zip(streams, work):
            with torch.cuda.stream(s):
                got.append(_pass(ad, b))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2])), i


def test_graph_of_an_adapter_set_outlives_longer_calls():
    ad, batch = _adapter_set(202, 1024, 512)
    small, large = batch([1] * 8, [0, 1, 2, -1] * 2), batch([900, 300, 1300], [2, 0, 1])
    want, want_large = _pass(ad, small), _pass(ad, large)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _pass(ad, small)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _pass(ad, small)
    for turn in range(4):
        got = _pass(ad, large)
        # blocks of every size that a workspace given back could be handed out as
        canaries = [torch.full((1 << k,), turn, dtype=torch.uint8, device=DEV) for k in range(9, 24)]
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), turn
        assert all(torch.equal(a, b) for a, b in zip(got, want_large)), turn
        assert all((c == turn).all() for c in canaries), turn


def test_one_layer_with_adapters_on_two_streams_and_in_a_graph():
    ad, batch = _adapter_set(203, 1024, 512)
    Wt = (np.random.default_rng(203).standard_normal((512, 1024)) / 32).astype(np.float32)
    L = W4A4Layer("mxfp4", "hadamard", Wt)
    work = [batch([30, 0, 200, 17], [0, 1, 2, -1])[:2], batch([1] * 40, [0, 1, 2, -1] * 10)[:2]]
    want = [L.forward(X, adapters=ad, requests=req) for X, req in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = []
    for turn in range(10):
        for s, (X, req) in zip(streams, work):
            with torch.cuda.stream(s):
                got.append(L.forward(X, adapters=ad, requests=req))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))
    (X, req), (X2, req2) = work[1], work[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = L.forward(X, adapters=ad, requests=req)
    for turn in range(4):
        large = L.forward(X2, adapters=ad, requests=req2)
        canaries = [torch.full((1 << k,), turn, dtype=torch.uint8, device=DEV) for k in range(9, 22)]
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[1]) and torch.equal(large, want[0]), turn
        assert all((c == turn).all() for c in canaries), turn


# ----------------------------------------------------------------------------- adapters: many of them


@pytest.mark.parametrize("n,nseg,nad,kind", [(3000, 200, 150, "ragged"), (300, 300, 70, "single"), (700, 65, 64, "ragged"),
                                             (2500, 2500, 300, "single"), (257, 129, 65, "ragged")])
def test_adapter_backward_of_many_adapters_and_requests(n, nseg, nad, kind):
    # more than 64 adapters and requests; adapters without tokens, of rank 0, with many requests and with one
    c = Case(301, n, 64, 72, nseg, nad, 16, kind=kind)
    dY = dev(c.r.standard_normal((n, 72)), "bf16")
    _, V = c.forward()
    dX, dA, dB = new(n, 64), new(nad, 16, 64), new(nad, 16, 72)
    ws = torch.full((W.wush_adapter_backward_ws_bytes(n, 64, 72, nseg, nad, 16),), 0xFF, dtype=torch.uint8, device=DEV)
    W.wush_adapter_backward(dY, c.X, *c.dev, V, None, dX, dA, dB, ws=ws)
    torch.cuda.synchronize()
    ref, mag = bo.adapter_backward(f64(dY), f64(c.X), *c.plain(), f64(V), None)
    near(dX, ref[0], mag[0], 72 + 16, "dX")
    near(dA, ref[1], mag[1], 72 + n, "dA")
    near(dB, ref[2], mag[2], n, "dBt")


def test_time_of_many_adapters_and_requests():
    # 4096 requests of a token over 1024 adapters: 64 turns of 64 requests, some microseconds each, and small products.
    # Work that grew with requests times adapters took above 3 ms for a quarter of these adapters.
    n, nad = 4096, 1024
    c = Case(302, n, 64, 64, n, nad, 16, kind="single")
    dY, V, dA, dB = dev(c.r.standard_normal((n, 64)), "bf16"), new(n, 16).zero_(), new(nad, 16, 64), new(nad, 16, 64)
    ws = torch.empty(W.wush_adapter_backward_ws_bytes(n, 64, 64, n, nad, 16), dtype=torch.uint8, device=DEV)
    best = np.inf
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        W.wush_adapter_backward(dY, c.X, *c.dev, V, None, None, dA, dB, ws=ws)
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    assert best < 2.0, best


def test_adapter_backward_of_few_among_many_adapters():
    # lists of several chunks between adapters without tokens: their partial sums lie side by side
    n, nad, d_in, d_out = 6000, 100, 64, 72
    c = Case(303, n, d_in, d_out, 7, nad, 16, ranks=[16] * nad)
    c.off, c.ids = [0, 1800, 1900, 4300, 4301, 4600, 5999, 6000], [99, 0, 5, 6, -1, 70, 64]
    c.dev = tuple(torch.tensor(a, dtype=torch.int32, device=DEV) for a in (c.off, c.ids)) + c.dev[2:]
    dY = dev(c.r.standard_normal((n, d_out)), "bf16")
    _, V = c.forward()
    dA, dB = new(nad, 16, d_in), new(nad, 16, d_out)
    need = W.wush_adapter_backward_ws_bytes(n, d_in, d_out, 7, nad, 16)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    W.wush_adapter_backward(dY, c.X, *c.dev, V, None, None, dA, dB, ws=ws[:need])
    torch.cuda.synchronize()
    assert (ws[need:] == 0xFF).all()
    ref, mag = bo.adapter_backward(f64(dY), f64(c.X), *c.plain(), f64(V), None)
    near(dA, ref[1], mag[1], d_out + n, "dA")
    near(dB, ref[2], mag[2], n, "dBt")


@pytest.mark.parametrize("xdt", ["bf16", "f32"])
@pytest.mark.parametrize("rmax", [16, 32, 64, 128])
@pytest.mark.parametrize("n,nseg", [(100, 4), (25, 1), (320, 9), (50, 3), (600, 5)])
def test_adapter_forward_of_every_token_tile(n, nseg, rmax, xdt):
    # requests of some 16 to 32 tokens, and longer ones; every number of row tiles of the factor, whole and partly used,
    # and pieces of k that end inside one, at the last column and past several
    for d_in in (64, 96, 1032):
        c = Case(304, n, d_in, 40, nseg, 4, rmax, xdt, ranks=[rmax, rmax // 2 + 1, rmax // 4 + 1, rmax - 1])
        c.check(*c.forward(), c.Y0)


# ----------------------------------------------------------------------------- block norm: wide rows, many rows


LEFT_OUT = ["nothing", "dRout", "dR", "w_post", "w_pre", "Y"]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("n,d", [(530, 8200), (300, 16392)])
def test_wide_norm_gradients_of_many_rows(n, d, types):
    # a workgroup walks over several rows; every gate, and every tensor left out in turn
    for i, gate in enumerate(["none", "channel", "token", "element"]):
        r, Y, wp, g, R, w = _norm_inputs(102 + i, n, d, types, gate)
        _norm_grads(r, Y, wp, g, R, w, types, 0.75, 1.25, d)
    left = LEFT_OUT[1:] if types == TYPES[3] else LEFT_OUT[1 + TYPES.index(types) % 5:][:1]
    for out in left:
        r, Y, wp, g, R, w = _norm_inputs(110, n, d, types, "token")
        _norm_grads(r, None if out == "Y" else Y, None if out in ("Y", "w_post") else wp, None if out == "Y" else g, R,
                    None if out == "w_pre" else w, types, 0.75, 1.25, d, dr=out != "dRout", want_dR=out != "dR")


@pytest.mark.parametrize("d", [12296, 16384, 20488, 24576])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
def test_widest_norm_gradients(gate, d):
    types = ("f32", "bf16", "bf16")
    r, Y, wp, g, R, w = _norm_inputs(120, 270, d, types, gate)
    _norm_grads(r, Y, wp, g, R, w, types, 1.0, 0.5, d)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("n,d", [(600, 520), (3, 12296), (3, 17408)])
def test_norm_with_several_pieces_a_thread(n, d, types):
    for gate in ("none", "channel", "token", "element"):
        _, Y, wp, g, R, w = _norm_inputs(130, n, d, types, gate)
        Rout, U, k1, k2 = new(n, d, dt=DT[types[1]]), new(n, d, dt=DT[types[2]]), new(n), new(n)
        W.wush_block_norm(Y, wp, g, R, w, Rout, U, k1, k2, branch_scale=0.7, res_scale=0.9)
        torch.cuda.synchronize()
        _norm_check(Y, wp, g, R, w, np.float32(0.7), np.float32(0.9), np.float32(1e-6), Rout, U, k1, k2, d)


# ----------------------------------------------------------------------------- outputs beyond the last-level cache
# Outputs above 256 MB are written past the caches.  The same rows in two calls below that must give the same bits, and
# the tests of small sizes hold those to the 64-bit form.


def _rand(g, n, d, dt="f32"):
    return torch.randn((n, d), generator=g, device=DEV).to(DT[dt])


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("types,n,d", [(("f32", "f32", "f32"), 2100, 16384), (("bf16", "f32", "f32"), 2100, 16392),
                                       (("f32", "bf16", "bf16"), 4200, 16384), (("bf16", "bf16", "bf16"), 4200, 16392),
                                       (("bf16", "f32", "bf16"), 2800, 16384), (("f32", "f32", "bf16"), 2800, 16392)])
def test_norm_outputs_beyond_the_cache(types, n, d):
    g, h = _gen(401), n // 2
    Y, R, w = _rand(g, n, d, types[0]), _rand(g, n, d, types[1]), 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
    outs = [[torch.full((n, d), 7.0, dtype=DT[t], device=DEV) for t in types[1:]] for _ in range(2)]
    assert n * d * sum(t[0].element_size() for t in zip(outs[0])) > 256 << 20
    W.wush_block_norm(Y, w, None, R, w, *outs[0])
    for a in (slice(0, h), slice(h, n)):
        W.wush_block_norm(Y[a], w, None, R[a], w, outs[1][0][a], outs[1][1][a])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("hdt", ["f32", "bf16"])
@pytest.mark.parametrize("xdt", ["f32", "bf16"])
def test_gated_activation_outputs_beyond_the_cache(xdt, hdt):
    g, d = _gen(402), 17408
    n = 4200 if xdt == hdt == "f32" else 8200
    x, dH = _rand(g, n, 2 * d, xdt), _rand(g, n, d, hdt)

    def both(rows):
        m = dH[rows].shape[0]
        H = torch.full((m, d), 7.0, dtype=DT[hdt], device=DEV)
        c = [torch.full((m, d // k), 99, dtype=t, device=DEV) for _ in range(2) for k, t in ((1, torch.int8), (32, torch.uint8))]
        W.wush_act8_swiglu(x[rows, :d], x[rows, d:], H, *c)
        H2 = torch.full_like(H, 7.0)
        W.wush_act8_swiglu(x[rows, :d], x[rows, d:], H2)
        dx = torch.full((m, 2 * d), 7.0, dtype=DT[xdt], device=DEV)
        W.wush_act8_swiglu_bwd(dH[rows], *c, dx[:, :d], dx[:, d:])
        back = torch.full((m, d), 7.0, dtype=DT[xdt], device=DEV)
        W.wush_act8_unpack(c[0], c[1], back)
        torch.cuda.synchronize()
        return [H, H2, dx, back] + c
    whole = both(slice(0, n))
    assert whole[0].numel() * whole[0].element_size() > 256 << 20
    for a in range(0, n, n // 4):
        rows = slice(a, min(n, a + n // 4))
        assert all(torch.equal(w[rows], p) for w, p in zip(whole, both(rows))), a


@pytest.mark.parametrize("rmax", [16, 32, 64, 128])
@pytest.mark.parametrize("ydt", ["f32", "bf16"])
def test_adapter_outputs_beyond_the_cache(ydt, rmax):
    # every request's rows at its first, middle and last tokens against the 64-bit form; with and without a base
    n, d_in, d_out = (4100, 264, 17408) if ydt == "f32" else (8200, 264, 17408)
    c = Case(403, n, d_in, d_out, 9, 4, rmax, ydt=ydt, ranks=[rmax, rmax // 2 + 1, 7, 0])
    assert c.Y0.numel() * c.Y0.element_size() > 256 << 20
    rows = sorted({t for a, b in zip(c.off, c.off[1:]) if a < b for t in (a, min(a + 63, b - 1), (a + b) // 2, b - 1)})
    # a request of one token for each of these rows
    ids = [c.ids[next(s for s in range(len(c.ids)) if c.off[s] <= t < c.off[s + 1])] for t in rows]
    for base in (c.Y0, None):
        Y, V = c.forward(Y0=base)
        plain = (list(range(len(rows) + 1)), ids) + c.plain()[2:]
        ref, mag = bo.adapter_forward(f64(c.X[rows]), *plain, None if base is None else f64(base[rows]), d_out)
        near(Y[rows], ref[0], mag[0], d_in + rmax, "Y")
        near(V[rows], ref[1], mag[1], d_in, "V")
        assert torch.isfinite(Y).all()


# ----------------------------------------------------------------------------- the fine-tuning example


def test_example_gradients_of_both_adapter_sets_against_the_formulas():
    # the example's backward pass against the 64-bit forms, from what its forward pass kept.  dY, dH and dGU are rounded
    # to bf16 between the steps, and dY W before it is added: four roundings of at most 2^-9 of a value each, which the
    # sums carry on; their norm is within 4 * 2^-9 of the result's, twice that with the terms' cancellation
    from finetune_mlp import MlpBlock
    g, n, d, h = _gen(501), 200, 256, 512
    block = MlpBlock(d, h, nad=2)
    R, c = _rand(g, n, d, "bf16"), _rand(g, n, d, "bf16")
    lengths, ids = [70, 30, 100], [0, -1, 1]
    req, off = request_table(lengths, ids), [0, 70, 100, 200]
    for ad in (block.ad_gu, block.ad_dn):
        ad.Bt.copy_(torch.randn(ad.Bt.shape, generator=g, device=DEV) * 0.1)
    _, kept = block.forward(R, req, train=True)
    grads = block.backward(c, req, kept)
    torch.cuda.synchronize()
    (u8, us), V1, (gc, gs, uc, uss), (h8, hs), V2, Y, Rout, k1, k2 = kept
    val = lambda q, s: bo.act8_values(q.cpu().numpy(), s.cpu().numpy())  # noqa: E731

    def adapters(ad, dY, X, V, dX0):
        return bo.adapter_backward(dY, X, off, ids, f64(ad.A), f64(ad.Bt), [16, 16], [1.0, 1.0], f64(V), dX0)[0]
    dY = bo.block_norm_bwd(f64(c), None, f64(Y), f64(block.w_post), f64(block.scale), f64(Rout), f64(block.w_out), f64(k1),
                           f64(k2), 1.0, 1.0)["dY"]
    dH, dA2, dB2 = adapters(block.ad_dn, dY, val(h8, hs), V2, dY @ f64(block.Wdn))
    dG, dU = bo.swiglu_bwd(dH, val(gc, gs), val(uc, uss))
    _, dA1, dB1 = adapters(block.ad_gu, np.concatenate([dG, dU], axis=1), val(u8, us), V1, None)
    for got, ref in zip((t for pair in grads for t in pair), (dA1, dB1, dA2, dB2)):
        assert np.linalg.norm(f64(got) - ref) <= 8 * 2.0 ** -9 * np.linalg.norm(ref)


# ----------------------------------------------------------------------------- adapters: infinities


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_adapter_gradients_reached_by_an_infinity(dt):
    # not finite where the infinity reaches, bit by bit the same elsewhere
    c = Case(305, 90, 264, 136, 3, 3, 16, dt, ranks=[16, 9, 16])
    c.off, c.ids = [0, 30, 60, 90], [0, 1, 2]
    c.dev = tuple(torch.tensor(a, dtype=torch.int32, device=DEV) for a in (c.off, c.ids)) + c.dev[2:]
    dY = dev(c.r.standard_normal((90, 136)), dt)
    _, V = c.forward()

    def grads(X, dY):
        dX, dA, dB = new(90, 264), new(3, 16, 264), new(3, 16, 136)
        W.wush_adapter_backward(dY, X, *c.dev, V, None, dX, dA, dB)
        torch.cuda.synchronize()
        return dX, dA, dB
    want = grads(c.X, dY)
    X = c.X.clone()
    X[40, 11] = float("inf")                      # a token of adapter 1: column 11 of its dA
    dX, dA, dB = grads(X, dY)
    assert torch.equal(dX, want[0]) and torch.equal(dB, want[2])
    assert not torch.isfinite(dA[1, :9, 11]).any()
    dA[1, :9, 11] = want[1][1, :9, 11]
    assert torch.equal(dA, want[1])
    bad = dY.clone()
    bad[70, 5] = float("-inf")                    # one of adapter 2: its row of dX, all of dA, column 5 of dBt
    dX, dA, dB = grads(c.X, bad)
    assert not torch.isfinite(dX[70]).any() and not torch.isfinite(dA[2]).any() and not torch.isfinite(dB[2, :, 5]).any()
    dX[70], dA[2], dB[2, :, 5] = want[0][70], want[1][2], want[2][2, :, 5]
    assert all(torch.equal(a, b) for a, b in zip((dX, dA, dB), want))


# ----------------------------------------------------------------------------- adapters: very many requests


@pytest.mark.parametrize("nseg", [65, 4096, 4097, 9000])
def test_adapter_of_very_many_requests(nseg):
    # requests of no token, one and several, more than one and two counts of 64 find
    r = np.random.default_rng(306)
    lengths = r.choice([0, 0, 1, 1, 1, 2, 5, 17], nseg)
    n, nad = int(lengths.sum()), 5
    c = Case(306, n, 64, 40, 2, nad, 16, ranks=[16, 16, 9, 0, 16])
    c.off, c.ids = [0] + [int(v) for v in np.cumsum(lengths)], [int(v) for v in r.integers(-1, nad, nseg)]
    c.dev = tuple(torch.tensor(a, dtype=torch.int32, device=DEV) for a in (c.off, c.ids)) + c.dev[2:]
    Y, V = c.forward()
    c.check(Y, V, c.Y0)
    dY = dev(c.r.standard_normal((n, 40)), "bf16")
    dX, dA, dB = new(n, 64), new(nad, 16, 64), new(nad, 16, 40)
    W.wush_adapter_backward(dY, c.X, *c.dev, V, None, dX, dA, dB)
    torch.cuda.synchronize()
    ref, mag = bo.adapter_backward(f64(dY), f64(c.X), *c.plain(), f64(V), None)
    near(dX, ref[0], mag[0], 40 + 16, "dX")
    near(dA, ref[1], mag[1], 40 + n, "dA")
    near(dB, ref[2], mag[2], n, "dBt")


def test_time_of_very_many_requests():
    # 65536 requests of a token: work that grows with the requests, some 130000 short workgroups, takes about a
    # millisecond; where each workgroup looked at all requests it took 22
    n = 65536
    A = torch.zeros((8, 16, 64), dtype=torch.bfloat16, device=DEV)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    args = (i32(range(n + 1)), i32(np.arange(n) % 8), A, A, i32([16] * 8), torch.ones(8, device=DEV))
    X, Y = torch.zeros((n, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((n, 64), device=DEV)
    ws = torch.empty(W.wush_adapter_ws_bytes(n, 64, n, 16), dtype=torch.uint8, device=DEV)
    best = np.inf
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        W.wush_adapter_forward(X, *args, Y, Y, ws=ws)
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    assert best < 5.0, best
