"""Plain 64-bit forms of the operators around a frozen projection (numpy).

Block norm and its gradient, act8 checkpoints and the gated activation that
uses them, adapters and their gradients.  Every function that sums also gives
the sum of the terms' magnitudes, from which the tests derive their bounds.
"""

import numpy as np


def _f(a):
    return None if a is None else np.asarray(a, np.float64)


# ----------------------------------------------------------------------------- block norm


def block_norm(Y, w_post, gate, R, w_pre, branch, res, eps):
    """(Rout, U, rstd_post, rstd_pre); U and rstd values None where there is no norm.  gate broadcasts over [n][d]."""
    Y, w_post, gate, R, w_pre = map(_f, (Y, w_post, gate, R, w_pre))
    k1 = k2 = U = None
    out = res * R
    if Y is not None:
        b = Y
        if w_post is not None:
            k1 = 1.0 / np.sqrt(np.mean(Y * Y, axis=1) + eps)
            b = b * k1[:, None] * w_post
        if gate is not None:
            b = b * gate
        out = out + branch * b
    if w_pre is not None:
        k2 = 1.0 / np.sqrt(np.mean(out * out, axis=1) + eps)
        U = out * k2[:, None] * w_pre
    return out, U, k1, k2


def _norm_grad(x, k, w, dz):
    """z = x k w, k = rstd(x): gradient of x, and the terms of that of w."""
    xh = x * k[:, None]
    q = dz * w
    return k[:, None] * (q - xh * np.mean(q * xh, axis=1, keepdims=True)), dz * xh


def block_norm_bwd(dU, dRout, Y, w_post, gate, Rout, w_pre, k1, k2, branch, res):
    """dict of dY, dR, dgate (full [n][d] terms), dw_post and dw_pre (terms [n][d]), from the stored Rout and rstd."""
    dU, dRout, Y, w_post, gate, Rout, w_pre, k1, k2 = map(_f, (dU, dRout, Y, w_post, gate, Rout, w_pre, k1, k2))
    out = {}
    t = 0.0 if dRout is None else dRout
    if w_pre is not None:
        dx, out["dw_pre"] = _norm_grad(Rout, k2, w_pre, dU)
        t = t + dx
    out["dR"] = res * t
    if Y is not None:
        h = branch * t
        z = Y if w_post is None else Y * k1[:, None] * w_post
        out["dgate"] = h * z
        db = h if gate is None else h * gate
        if w_post is None:
            out["dY"] = db + np.zeros_like(Y)
        else:
            out["dY"], out["dw_post"] = _norm_grad(Y, k1, w_post, db)
    return out


# ----------------------------------------------------------------------------- act8


def act8_pack(X):
    """(codes int8, scale bytes) of float32 X [n][d], d a multiple of 32."""
    X = np.asarray(X, np.float32)
    n, d = X.shape
    v = X.astype(np.float64).reshape(n, d // 32, 32)
    with np.errstate(invalid="ignore"):
        a = np.abs(v).max(axis=2)
    bad = ~np.isfinite(v).all(axis=2)
    a = np.where(bad | (a == 0), 2.0 ** -120, a)
    e = np.clip(np.frexp(a)[1] - 1, -120, 127)
    with np.errstate(invalid="ignore"):
        q = np.clip(np.rint(np.ldexp(v, (6 - e)[:, :, None])), -127, 127)
    q = np.where(bad[:, :, None], 0, q).astype(np.int8)
    return q.reshape(n, d), np.where(bad, 255, e + 127).astype(np.uint8)


def act8_values(codes, scales):
    """What a checkpoint stands for, in 64 bits (exactly)."""
    n, d = codes.shape
    e = scales.astype(np.int64) - 127
    v = np.ldexp(codes.astype(np.float64).reshape(n, d // 32, 32), (e - 6)[:, :, None])
    return np.where((scales == 255)[:, :, None], np.nan, v).reshape(n, d)


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def swiglu(G, U):
    G, U = _f(G), _f(U)
    return G * sigmoid(G) * U


def swiglu_bwd(dH, g, u):
    """(dG, dU) at the values g, u."""
    dH, g, u = map(_f, (dH, g, u))
    s = sigmoid(g)
    return dH * u * s * (1.0 + g * (1.0 - s)), dH * g * s


# ----------------------------------------------------------------------------- adapters


def adapter_forward(X, off, ids, A, Bt, rank, alpha, Y0, d_out):
    """((Y, V), (their magnitudes)): a loop over the requests."""
    X, A, Bt, Y0 = map(_f, (X, A, Bt, Y0))
    n, nad, rmax = X.shape[0], A.shape[0], A.shape[1]
    V, Vm = np.zeros((n, rmax)), np.zeros((n, rmax))
    Y = np.zeros((n, d_out)) if Y0 is None else Y0.copy()
    Ym = np.abs(Y)
    for s in range(len(ids)):
        b, e, i = off[s], off[s + 1], ids[s]
        if b == e or not 0 <= i < nad or rank[i] == 0:
            continue
        k = rank[i]
        V[b:e, :k] = alpha[i] * (X[b:e] @ A[i, :k].T)
        Vm[b:e, :k] = abs(alpha[i]) * (np.abs(X[b:e]) @ np.abs(A[i, :k].T))
        Y[b:e] += V[b:e, :k] @ Bt[i, :k]
        Ym[b:e] += Vm[b:e, :k] @ np.abs(Bt[i, :k])
    return (Y, V), (Ym, Vm)


def adapter_backward(dY, X, off, ids, A, Bt, rank, alpha, V, dX0):
    """((dX, dA, dBt), (their magnitudes))."""
    dY, X, A, Bt, V, dX0 = map(_f, (dY, X, A, Bt, V, dX0))
    nad = A.shape[0]
    dX = np.zeros_like(X) if dX0 is None else dX0.copy()
    dXm = np.abs(dX)
    dA, dB = np.zeros_like(A), np.zeros_like(Bt)
    dAm, dBm = np.zeros_like(A), np.zeros_like(Bt)
    for s in range(len(ids)):
        b, e, i = off[s], off[s + 1], ids[s]
        if b == e or not 0 <= i < nad or rank[i] == 0:
            continue
        k = rank[i]
        dV = alpha[i] * (dY[b:e] @ Bt[i, :k].T)
        dVm = abs(alpha[i]) * (np.abs(dY[b:e]) @ np.abs(Bt[i, :k].T))
        dX[b:e] += dV @ A[i, :k]
        dXm[b:e] += dVm @ np.abs(A[i, :k])
        dA[i, :k] += dV.T @ X[b:e]
        dAm[i, :k] += dVm.T @ np.abs(X[b:e])
        dB[i, :k] += V[b:e, :k].T @ dY[b:e]
        dBm[i, :k] += np.abs(V[b:e, :k]).T @ np.abs(dY[b:e])
    return (dX, dA, dB), (dXm, dAm, dBm)
