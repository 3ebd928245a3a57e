"""Block norm, act8 and adapters on the GPU at their edges: infinities, wide rows in numbers, many adapters, outputs
beyond the last-level cache, streams and graphs.

Bounds are those of test_gpu_block_ops: (K + 32) 2^-24 times the result computed from magnitudes, and 2^-8 of its value
for bf16 results.
"""

import numpy as np
import pytest
import torch

import aware_block_transforms_amd as W
from aware_block_transforms_amd.layer import AdapterSet, W4A4Layer, request_table
from oracle import block_ops as bo
from gpu_util import DEV
from test_gpu_block_ops import Case, _norm_inputs, dev, f64, near, new

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
