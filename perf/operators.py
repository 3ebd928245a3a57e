"""Measured cases of the operators around a frozen W4A4 projection.

Three operators, each in the directions that a program calls:

  block norm   the norm after a block, its gate and residual scale, the residual sum and the norm before the next
               block (``wush_block_norm``), and its gradients (``wush_block_norm_bwd``)
  act8         activations kept in 8 bits for the backward pass: the gated MLP activation that stores its two inputs
               (``wush_act8_swiglu``) and its gradient from what was stored (``wush_act8_swiglu_bwd``); plain storing
               and reading back (``wush_act8_pack``, ``wush_act8_unpack``)
  adapters     low-rank adapters of many requests beside the shared projection (``wush_adapter_forward``), and the
               gradients of the adapters and of their input (``wush_adapter_backward``), the input either whole or as
               an act8 checkpoint

``run`` computes the plain form where ``own`` is false (torch, 32 bits) and calls the library where it is true.
"""

import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 32          # act8: values under one scale
EPS = 1e-6

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2, "act8": 1 + 1 / GROUP}


# ----------------------------------------------------------------------------- cases


def listed():
    return [
        # one token of one request between two blocks of a serving model: only latency counts
        dict(name="norm-token", op="norm_fwd", n=1, d=4096, ydt="f32", rdt="bf16", udt="bf16", gate="none"),
        # a long prefill between two blocks, the matmul's fp32 output in, bf16 for the next transform out
        dict(name="norm-prefill", op="norm_fwd", n=16384, d=5120, ydt="f32", rdt="bf16", udt="bf16", gate="channel"),
        # the same place in a training step of a 4096-wide model
        dict(name="norm-train", op="norm_bwd", n=4096, d=4096, ydt="f32", rdt="bf16", udt="bf16", gate="channel"),
        # a ragged batch with a gate for each value, everything in fp32, an odd width
        dict(name="norm-train-odd", op="norm_bwd", n=1021, d=2600, ydt="f32", rdt="f32", udt="f32", gate="element"),
        # a short fine-tuning batch through a 12288-wide gated MLP: forward with checkpoints, then backward
        dict(name="act8-mlp-short", op="act8_mlp", n=61, d=12288, gdt="bf16", hdt="bf16"),
        # the largest activation of a 17408-wide MLP at 16384 tokens, kept in 8 bits and used by the backward pass
        dict(name="act8-mlp-train", op="act8_mlp", n=16384, d=17408, gdt="f32", hdt="bf16"),
        # a projection's input kept in 8 bits and read back, a ragged token count
        dict(name="act8-store", op="act8_store", n=4099, d=5120, xdt="bf16", ydt="bf16"),
        # one token with one of eight adapters on a square projection: only latency counts
        dict(name="adapter-token", op="adapter_fwd", n=1, d_in=4096, d_out=4096, nreq=1, nad=8, rmax=16, layout=1,
             xdt="bf16", ydt="f32", save=False),
        # a decode step: 64 requests of one token each, 32 adapters of ragged rank, some requests without one
        dict(name="adapter-decode", op="adapter_fwd", n=64, d_in=4096, d_out=12288, nreq=64, nad=32, rmax=64,
             layout=2, xdt="bf16", ydt="f32", save=False),
        # a prefill of nine ragged requests on the up projection, the last rank unused rows included
        dict(name="adapter-prefill", op="adapter_fwd", n=16384, d_in=5120, d_out=17408, nreq=9, nad=6, rmax=64,
             layout=3, xdt="bf16", ydt="f32", save=False),
        # training two adapters on ragged sequences of a 4096-wide model's up projection
        dict(name="adapter-train", op="adapter_bwd", n=4096, d_in=4096, d_out=12288, nreq=5, nad=2, rmax=32,
             layout=4, xdt="bf16", gdt="bf16", ydt="bf16"),
        # training adapters of the down projection, whose wide input was kept in 8 bits
        dict(name="adapter-train-act8", op="adapter_bwd", n=16384, d_in=17408, d_out=5120, nreq=12, nad=4, rmax=64,
             layout=5, xdt="act8", gdt="bf16", ydt="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "act8_mlp", "act8_store", "adapter_fwd", "adapter_fwd", "adapter_bwd",
                     "adapter_bwd"])
    fl = ["f32", "bf16"]
    if op in ("norm_fwd", "norm_bwd"):
        d = 8 * _log(rng, 16, 2176)
        n = min(_log(rng, 1, 16384), max(1, 16384 * 5120 // d))
        rdt = rng.choice(fl)
        return dict(op=op, n=n, d=d, ydt=rng.choice(fl), rdt=rdt, udt=rng.choice(fl) if rdt == "f32" else "bf16",
                    gate=rng.choice(["none", "channel", "token", "element"]))
    if op == "act8_mlp":
        return dict(op=op, n=_log(rng, 1, 16384), d=32 * _log(rng, 4, 544), gdt=rng.choice(fl), hdt=rng.choice(fl))
    if op == "act8_store":
        return dict(op=op, n=_log(rng, 1, 16384), d=32 * _log(rng, 4, 544), xdt=rng.choice(fl), ydt=rng.choice(fl))
    d_in, d_out = 32 * _log(rng, 8, 544), 8 * _log(rng, 32, 2176)
    n = _log(rng, 1, 16384)
    nreq = min(n, _log(rng, 1, 128))
    nad = _log(rng, 1, 32)
    rmax = rng.choice([16, 32, 64, 128] if n < 4096 else [16, 32, 64])
    # the plain form multiplies every token by every adapter
    while n * (d_in + d_out) * nad * rmax > 16384 * (5120 + 17408) * 8 * 64:
        nad, n = max(1, nad // 2), n if nad > 1 else n // 2
    nreq = min(n, nreq)
    case = dict(op=op, n=n, d_in=d_in, d_out=d_out, nreq=nreq, nad=nad, rmax=rmax, layout=rng.randrange(1 << 20),
                xdt=rng.choice(fl), ydt=rng.choice(fl))
    if op == "adapter_fwd":
        case["save"] = rng.random() < 0.5
    else:
        case["xdt"] = rng.choice(["f32", "bf16", "act8"])
        case["gdt"] = rng.choice(fl)
    return case


# ----------------------------------------------------------------------------- inputs


def _requests(case):
    """(offsets [nreq + 1], adapter of each request or -1, rank of each adapter), from the case alone."""
    r = random.Random(case["layout"])
    n, nreq, nad, rmax = case["n"], case["nreq"], case["nad"], case["rmax"]
    if n == nreq:
        off = list(range(n + 1))
    else:
        # ragged requests; now and then one is empty
        off = [0] + sorted(r.randrange(n + 1) for _ in range(nreq - 1)) + [n]
    ids = [r.randrange(nad) if nreq == 1 or r.random() < 0.9 else -1 for _ in range(nreq)]
    ranks = [r.choice([rmax, rmax, rmax // 2, rmax // 2 + 1, 8]) for _ in range(nad)]
    return off, ids, ranks


def _covered(case):
    """Tokens under an adapter, the sum of their ranks, and the ranks of the adapters in use."""
    off, ids, ranks = _requests(case)
    lens = [b - a for a, b in zip(off, off[1:])]
    used = sorted({i for i, m in zip(ids, lens) if i >= 0 and m})
    return (sum(m for m, i in zip(lens, ids) if i >= 0), sum(m * ranks[i] for m, i in zip(lens, ids) if i >= 0),
            sum(ranks[i] for i in used))


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale)


def _acts(g, n, d):
    """Activations: normal values, one channel in 512 larger by a factor of 20 to 100."""
    x = _normal(g, (n, d))
    k = max(1, d // 512)
    ch = torch.randperm(d, generator=g, device=DEV)[:k]
    x[:, ch] *= 20.0 * 5.0 ** torch.rand(k, generator=g, device=DEV)
    return x


def _pow2(e):
    """2^e in 32 bits, for whole e in [-126, 127]."""
    return e.to(torch.int32).add(127).bitwise_left_shift(23).view(torch.float32)


def _act8(x):
    """(codes int8, scale bytes) of an act8 checkpoint: q = rint(x 2^(6-e)) in [-127, 127], e = floor(log2 max|x|)."""
    n, d = x.shape
    v = x.float().reshape(n, d // GROUP, GROUP)
    e = torch.frexp(v.abs().amax(-1, keepdim=True))[1].sub(1).clamp(-120, 127)
    e = torch.where(v.abs().amax(-1, keepdim=True) > 0, e, torch.full_like(e, -120))
    q = torch.round(v * _pow2(6 - e)).clamp(-127, 127)
    return q.to(torch.int8).reshape(n, d), (e + 127).to(torch.uint8).reshape(n, d // GROUP)


def _value8(codes, scales):
    n, d = codes.shape
    e = scales.to(torch.int32).sub(127 + 6)
    return (codes.float().reshape(n, d // GROUP, GROUP) * _pow2(e).unsqueeze(-1)).reshape(n, d)


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], dict(case)
    if op in ("norm_fwd", "norm_bwd"):
        n, d = case["n"], case["d"]
        s["y"] = _acts(g, n, d).to(DT[case["ydt"]])
        s["r"] = _normal(g, (n, d), 3.0).to(DT[case["rdt"]])
        s["w_post"] = 1.0 + _normal(g, (d,), 0.1)
        s["w_pre"] = 1.0 + _normal(g, (d,), 0.1)
        s["gate"] = {"none": lambda: None,
                     "channel": lambda: 0.5 + _normal(g, (d,), 0.2),
                     "token": lambda: torch.rand((n, 1), generator=g, device=DEV),
                     "element": lambda: torch.sigmoid(_normal(g, (n, d))).to(DT[case["ydt"]])}[case["gate"]]()
        s["branch"], s["res"] = 0.7, 0.9
        if op == "norm_bwd":
            r, _, s["rstd_post"], s["rstd_pre"] = _norm_fwd(s)
            s["rout"] = r.to(DT[case["rdt"]])
            s["du"] = _normal(g, (n, d), 0.5).to(DT[case["udt"]])
            s["drout"] = _normal(g, (n, d)).to(DT[case["rdt"]])
            del s["r"]
    elif op == "act8_mlp":
        n, d = case["n"], case["d"]
        # the two halves of one fused projection's output
        gu = torch.empty((n, 2 * d), dtype=DT[case["gdt"]], device=DEV)
        gu[:, :d] = _acts(g, n, d)
        gu[:, d:] = _acts(g, n, d)
        s["g"], s["u"] = gu[:, :d], gu[:, d:]
        s["dh"] = _normal(g, (n, d), 0.1).to(DT[case["hdt"]])
    elif op == "act8_store":
        s["x"] = _acts(g, case["n"], case["d"]).to(DT[case["xdt"]])
    else:
        n, d_in, d_out, nad, rmax = (case[k] for k in ("n", "d_in", "d_out", "nad", "rmax"))
        off, ids, ranks = _requests(case)
        s["off"] = torch.tensor(off, dtype=torch.int32, device=DEV)
        s["ids"] = torch.tensor(ids, dtype=torch.int32, device=DEV)
        s["rank"] = torch.tensor(ranks, dtype=torch.int32, device=DEV)
        s["alpha"] = 0.5 + torch.rand(nad, generator=g, device=DEV)
        s["A"] = _normal(g, (nad, rmax, d_in), d_in ** -0.5).to(torch.bfloat16)
        s["Bt"] = _normal(g, (nad, rmax, d_out), 0.1).to(torch.bfloat16)
        x = _acts(g, n, d_in)
        if case["xdt"] == "act8":
            s["x"], s["xs"] = _act8(x.to(torch.bfloat16))
        else:
            s["x"], s["xs"] = x.to(DT[case["xdt"]]), None
        del x
        if op == "adapter_fwd":
            s["y0"] = _normal(g, (n, d_out)).to(DT[case["ydt"]])
        else:
            s["v"] = _low(s["x"] if s["xs"] is None else _value8(s["x"], s["xs"]), s["A"], s)
            s["dy"] = _normal(g, (n, d_out), 0.1).to(DT[case["gdt"]])
            s["dx0"] = _normal(g, (n, d_in), 0.1).to(DT[case["ydt"]])
    return s


# ----------------------------------------------------------------------------- plain forms (32 bits)


def _norm_fwd(s):
    y = s["y"].float()
    rp = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    a = y * rp * s["w_post"]
    if s["gate"] is not None:
        a = a * s["gate"].float()
    r = s["res"] * s["r"].float() + s["branch"] * a
    rn = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    return r, r * rn * s["w_pre"], rp.reshape(-1), rn.reshape(-1)


def _norm_bwd(s):
    y, r, du = s["y"].float(), s["rout"].float(), s["du"].float()
    rp, rn = s["rstd_post"].unsqueeze(-1), s["rstd_pre"].unsqueeze(-1)
    xr = r * rn
    q = du * s["w_pre"]
    dr = s["drout"].float() + rn * (q - xr * (q * xr).mean(-1, keepdim=True))
    dw_pre = (du * xr).sum(0)
    xy = y * rp
    a = xy * s["w_post"]
    da, dgate = s["branch"] * dr, None
    if s["gate"] is not None:
        dgate = da * a
        if s["case_gate"] == "channel":
            dgate = dgate.sum(0)
        elif s["case_gate"] == "token":
            dgate = dgate.sum(-1, keepdim=True)
        else:
            dgate = dgate.to(s["gate"].dtype)
        da = da * s["gate"].float()
    dw_post = (da * xy).sum(0)
    p = da * s["w_post"]
    dy = rp * (p - xy * (p * xy).mean(-1, keepdim=True))
    return (dy.to(s["y"].dtype), (s["res"] * dr).to(s["rout"].dtype), dgate, dw_post, dw_pre)


def _owner(s):
    """Adapter of every token, -1 for none."""
    t = torch.arange(s["n"], dtype=torch.int32, device=DEV)
    return s["ids"][torch.searchsorted(s["off"][1:].contiguous(), t, right=True)]


def _mask(s):
    """[n][nad][rmax]: whose token, and which of its rows count; times the adapter's factor."""
    own_by = _owner(s).unsqueeze(-1) == torch.arange(s["nad"], device=DEV)
    rows = torch.arange(s["rmax"], device=DEV) < s["rank"].unsqueeze(-1)
    return own_by.unsqueeze(-1) * (rows * s["alpha"].unsqueeze(-1))


def _all_low(x, w, s):
    """Every token by every adapter's rows, those of other adapters zero: [n][nad * rmax]."""
    v = x.float() @ w.float().reshape(s["nad"] * s["rmax"], -1).t()
    return v * _mask(s).reshape(s["n"], -1)


def _low(x, w, s):
    return _all_low(x, w, s).reshape(s["n"], s["nad"], s["rmax"]).sum(1)


def _spread(v, s):
    """[n][rmax] to [n][nad * rmax], zero but in the place of the token's adapter."""
    own_by = (_owner(s).unsqueeze(-1) == torch.arange(s["nad"], device=DEV)).unsqueeze(-1)
    return (v.unsqueeze(1) * own_by).reshape(s["n"], -1)


def _plain(s):
    op = s["op"]
    if op == "norm_fwd":
        r, u, rp, rn = _norm_fwd(s)
        return r.to(DT[s["rdt"]]), u.to(DT[s["udt"]]), rp, rn
    if op == "norm_bwd":
        return _norm_bwd({**s, "case_gate": "none" if s["gate"] is None else _kind(s)})
    if op == "act8_mlp":
        gf, uf = s["g"].float(), s["u"].float()
        h = (gf / (1 + torch.exp(-gf)) * uf).to(DT[s["hdt"]])
        gh, uh = _value8(*_act8(gf)), _value8(*_act8(uf))
        sg = 1 / (1 + torch.exp(-gh))
        dh = s["dh"].float()
        dg = dh * uh * sg * (1 + gh * (1 - sg))
        return h, dg.to(DT[s["gdt"]]), (dh * gh * sg).to(DT[s["gdt"]])
    if op == "act8_store":
        return _value8(*_act8(s["x"])).to(DT[s["ydt"]])
    nad, rmax = s["nad"], s["rmax"]
    if op == "adapter_fwd":
        va = _all_low(s["x"], s["A"], s)
        y = (s["y0"].float() + va @ s["Bt"].float().reshape(nad * rmax, -1)).to(DT[s["ydt"]])
        return (y, va.reshape(s["n"], nad, rmax).sum(1)) if s["save"] else y
    x = s["x"].float() if s["xs"] is None else _value8(s["x"], s["xs"])
    dy = s["dy"].float()
    dva = _all_low(dy, s["Bt"], s)
    dx = (s["dx0"].float() + dva @ s["A"].float().reshape(nad * rmax, -1)).to(DT[s["ydt"]])
    da = (dva.t() @ x).reshape(nad, rmax, -1)
    dbt = (_spread(s["v"], s).t() @ dy).reshape(nad, rmax, -1)
    return dx, da, dbt


def _kind(s):
    shape = tuple(s["gate"].shape)
    return "channel" if len(shape) == 1 else "token" if shape[1] == 1 and s["d"] > 1 else "element"


# ----------------------------------------------------------------------------- the library's calls


def _library(s):
    import aware_block_transforms_amd as W
    op = s["op"]
    new = lambda *shape, dt=torch.float32: torch.empty(shape, dtype=dt, device=DEV)  # noqa: E731
    if op == "norm_fwd":
        n, d = s["n"], s["d"]
        r, u, rp, rn = new(n, d, dt=DT[s["rdt"]]), new(n, d, dt=DT[s["udt"]]), new(n), new(n)
        W.wush_block_norm(s["y"], s["w_post"], s["gate"], s["r"], s["w_pre"], r, u, rstd_post=rp, rstd_pre=rn,
                          branch_scale=s["branch"], res_scale=s["res"], eps=EPS)
        return r, u, rp, rn
    if op == "norm_bwd":
        n, d = s["n"], s["d"]
        dy, dr = torch.empty_like(s["y"]), torch.empty_like(s["rout"])
        dgate = None if s["gate"] is None else torch.empty_like(s["gate"])
        dw_post, dw_pre = new(d), new(d)
        ws = new(W.wush_block_norm_bwd_ws_bytes(n, d), dt=torch.uint8)
        W.wush_block_norm_bwd(s["du"], s["drout"], s["y"], s["w_post"], s["gate"], s["rout"], s["w_pre"],
                              s["rstd_post"], s["rstd_pre"], dy, dr, dgate, dw_post, dw_pre,
                              branch_scale=s["branch"], res_scale=s["res"], ws=ws)
        return dy, dr, dgate, dw_post, dw_pre
    if op == "act8_mlp":
        n, d = s["n"], s["d"]
        h = new(n, d, dt=DT[s["hdt"]])
        gc, uc = new(n, d, dt=torch.int8), new(n, d, dt=torch.int8)
        gs, us = new(n, d // GROUP, dt=torch.uint8), new(n, d // GROUP, dt=torch.uint8)
        W.wush_act8_swiglu(s["g"], s["u"], h, gc, gs, uc, us)
        dg, du = new(n, d, dt=DT[s["gdt"]]), new(n, d, dt=DT[s["gdt"]])
        W.wush_act8_swiglu_bwd(s["dh"], gc, gs, uc, us, dg, du)
        return h, dg, du
    if op == "act8_store":
        n, d = s["n"], s["d"]
        c, sc, y = new(n, d, dt=torch.int8), new(n, d // GROUP, dt=torch.uint8), new(n, d, dt=DT[s["ydt"]])
        W.wush_act8_pack(s["x"], c, sc)
        W.wush_act8_unpack(c, sc, y)
        return y
    n, d_in, d_out, nad, rmax, nreq = (s[k] for k in ("n", "d_in", "d_out", "nad", "rmax", "nreq"))
    if op == "adapter_fwd":
        y, v = torch.empty_like(s["y0"]), new(n, rmax) if s["save"] else None
        ws = new(W.wush_adapter_ws_bytes(n, d_in, nreq, rmax), dt=torch.uint8)
        W.wush_adapter_forward(s["x"], s["off"], s["ids"], s["A"], s["Bt"], s["rank"], s["alpha"], s["y0"], y, V=v,
                               ws=ws)
        return (y, v) if s["save"] else y
    dx, da, dbt = torch.empty_like(s["dx0"]), new(nad, rmax, d_in), new(nad, rmax, d_out)
    ws = new(W.wush_adapter_backward_ws_bytes(n, d_in, d_out, nreq, nad, rmax), dt=torch.uint8)
    W.wush_adapter_backward(s["dy"], s["x"], s["off"], s["ids"], s["A"], s["Bt"], s["rank"], s["alpha"], s["v"],
                            s["dx0"], dx, da, dbt, x_scales=s["xs"], ws=ws)
    return dx, da, dbt


def run(state):
    return _library(state) if own else _plain(state)


# ----------------------------------------------------------------------------- what a pass cannot do without


def work(case):
    op, n = case["op"], case["n"]
    if op in ("norm_fwd", "norm_bwd"):
        e, d = n * case["d"], case["d"]
        y, r, u = BYTES[case["ydt"]], BYTES[case["rdt"]], BYTES[case["udt"]]
        gate = {"none": 0, "channel": 4 * d, "token": 4 * n, "element": e * y}[case["gate"]]
        if op == "norm_fwd":
            return {"bytes": e * (y + 2 * r + u) + gate + 8 * d + 8 * n, "flops": 11 * e}
        return {"bytes": e * (u + 3 * r + 2 * y) + 2 * gate + 16 * d + 8 * n, "flops": 24 * e}
    if op == "act8_mlp":
        # read both halves, write h; store and read both checkpoints; read dh, write both gradients
        e = n * case["d"]
        return {"bytes": e * (4 * BYTES[case["gdt"]] + 2 * BYTES[case["hdt"]] + 4 * BYTES["act8"]), "flops": 28 * e}
    if op == "act8_store":
        e = n * case["d"]
        return {"bytes": e * (BYTES[case["xdt"]] + BYTES[case["ydt"]] + 2 * BYTES["act8"]), "flops": 5 * e}
    d_in, d_out, nad, rmax = case["d_in"], case["d_out"], case["nad"], case["rmax"]
    tokens, ranks, rows = _covered(case)
    y, x = BYTES[case["ydt"]], BYTES[case["xdt"]]
    if op == "adapter_fwd":
        return {"bytes": tokens * d_in * x + rows * (d_in + d_out) * 2 + 2 * n * d_out * y
                + (4 * n * rmax if case["save"] else 0), "flops": 2 * ranks * (d_in + d_out)}
    return {"bytes": tokens * (d_in * x + d_out * BYTES[case["gdt"]] + 4 * rmax) + rows * (d_in + d_out) * 2
            + 2 * n * d_in * y + nad * rmax * (d_in + d_out) * 4, "flops": 4 * ranks * (d_in + d_out)}


# ----------------------------------------------------------------------------- 64 bits, from the definitions


def _rows(total, width):
    """Row ranges small enough for 64-bit temporaries."""
    step = max(1, (1 << 26) // max(1, width))
    return [slice(a, min(total, a + step)) for a in range(0, total, step)]


def _exact_norm_fwd(s):
    outs = []
    for c in _rows(s["n"], s["d"]):
        y, r = s["y"][c].double(), s["r"][c].double()
        rp = (y.square().sum(1) / s["d"] + EPS).pow(-0.5)
        branch = torch.einsum("td,t,d->td", y, rp, s["w_post"].double())
        if s["gate"] is not None:
            branch *= (s["gate"] if s["gate"].dim() == 1 else s["gate"][c]).double()
        ro = r * s["res"] + branch * s["branch"]
        rn = (ro.square().sum(1) / s["d"] + EPS).pow(-0.5)
        outs.append((ro, torch.einsum("td,t,d->td", ro, rn, s["w_pre"].double()), rp, rn))
    return tuple(torch.cat(o) for o in zip(*outs))


def _exact_norm_bwd(s):
    # the gradient of a mean-square norm z = v k w, k = rstd: dv = k (w dz) - v k^3 <w dz, v> / d
    d, w_post, w_pre = s["d"], s["w_post"].double(), s["w_pre"].double()
    dys, drs, dgs = [], [], []
    dw_post, dw_pre, dgc = (torch.zeros(d, dtype=torch.float64, device=DEV) for _ in range(3))
    kind = "none" if s["gate"] is None else _kind(s)
    for c in _rows(s["n"], d):
        k1, k2 = s["rstd_post"][c].double().unsqueeze(1), s["rstd_pre"][c].double().unsqueeze(1)
        y, v, du = s["y"][c].double(), s["rout"][c].double(), s["du"][c].double()
        dz = du * w_pre
        total = s["drout"][c].double() + k2 * dz - v * (k2 ** 3 / d) * (dz * v).sum(1, keepdim=True)
        dw_pre += (du * v * k2).sum(0)
        drs.append(total * s["res"])
        db = total * s["branch"]
        gate = None if kind == "none" else s["gate"].double() if kind == "channel" else s["gate"][c].double()
        if gate is not None:
            dg = db * (y * k1 * w_post)
            if kind == "channel":
                dgc += dg.sum(0)
            else:
                dgs.append(dg.sum(1, keepdim=True) if kind == "token" else dg)
            db = db * gate
        dw_post += (db * y * k1).sum(0)
        dp = db * w_post
        dys.append(k1 * dp - y * (k1 ** 3 / d) * (dp * y).sum(1, keepdim=True))
    dgate = None if kind == "none" else dgc if kind == "channel" else torch.cat(dgs)
    return torch.cat(dys), torch.cat(drs), dgate, dw_post, dw_pre


def _exact_kept(x):
    """What an act8 checkpoint of x stands for: x to the nearest of 255 multiples of 2^(e-6), ties to the even one."""
    v = x.double().reshape(x.shape[0], -1, GROUP)
    top = v.abs().max(-1, keepdim=True).values
    # the exponent field of the 64-bit value is floor(log2) + 1023
    e = (top.view(torch.int64) >> 52).sub(1023).clamp(-120, 127)
    unit = (e + (1023 - 6) << 52).view(torch.float64)
    return (torch.clamp(torch.round(v / unit), -127, 127) * unit).reshape(x.shape)


def _exact_act8_mlp(s):
    outs = []
    for c in _rows(s["n"], s["d"]):
        g, u, dh = s["g"][c].double(), s["u"][c].double(), s["dh"][c].double()
        gk, uk = _exact_kept(g), _exact_kept(u)
        p = torch.sigmoid(gk)
        outs.append((g * torch.sigmoid(g) * u, dh * uk * (p + gk * p * torch.sigmoid(-gk)), dh * gk * p))
    return tuple(torch.cat(o) for o in zip(*outs))


def _exact_adapters(s):
    """Request by request, from the definition."""
    off, ids, ranks = _requests(s)
    n, rmax = s["n"], s["rmax"]
    x = s["x"] if s["xs"] is None else None

    def inputs(a, b):
        if x is not None:
            return x[a:b].double()
        unit = torch.exp2(s["xs"][a:b].double() - 133).repeat_interleave(GROUP, dim=1)
        return s["x"][a:b].double() * unit

    if s["op"] == "adapter_fwd":
        y, v = s["y0"].double(), torch.zeros((n, rmax), dtype=torch.float64, device=DEV)
    else:
        y = s["dx0"].double()
        da = torch.zeros(s["A"].shape, dtype=torch.float64, device=DEV)
        dbt = torch.zeros(s["Bt"].shape, dtype=torch.float64, device=DEV)
    for a, b, i in zip(off, off[1:], ids):
        if i < 0 or a == b:
            continue
        k, f = ranks[i], s["alpha"][i].double()
        wa, wb = s["A"][i, :k].double(), s["Bt"][i, :k].double()
        if s["op"] == "adapter_fwd":
            low = f * (inputs(a, b) @ wa.t())
            v[a:b, :k] = low
            y[a:b] += low @ wb
        else:
            dy = s["dy"][a:b].double()
            low = f * (dy @ wb.t())
            y[a:b] += low @ wa
            da[i, :k] += low.t() @ inputs(a, b)
            dbt[i, :k] += s["v"][a:b, :k].double().t() @ dy
    if s["op"] == "adapter_fwd":
        return (y, v) if s["save"] else y
    return y, da, dbt


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        return _exact_norm_fwd(s)
    if op == "norm_bwd":
        return _exact_norm_bwd(s)
    if op == "act8_mlp":
        return _exact_act8_mlp(s)
    if op == "act8_store":
        return _exact_kept(s["x"])
    return _exact_adapters(s)
