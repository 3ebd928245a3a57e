"""Allocation helpers around the libwush calls for one quantized linear layer and the adapters beside it.

``AdapterSet`` holds low-rank adapters of one projection.  ``W4A4Layer`` holds the device-resident pieces of one layer (transform
matrices, packed weight codes and scales) and exposes the online path
(transform + quantize activations, then the W4A4 matmul) as two library
calls.  Tensors come from torch's caching allocator; every byte of
arithmetic runs inside libwush.so.
"""

import numpy as np
import torch

from . import _lib as W


def codes_shape(rows, d_in):
    return (rows, d_in // 2)


def scales_dtype(fmt):
    return torch.int16 if fmt == "int4" else torch.uint8


def _scratch(need, device):
    """A call's workspace.  It belongs to the call alone: torch's allocator takes it from the current stream's blocks, or
    from the pool of the graph being captured, so calls on several streams, and replays, never meet in one."""
    return torch.empty(max(need, 16), dtype=torch.uint8, device=device)


class W4A4Layer:
    """Weights Wt [d_out][d_in] (nn.Linear layout) quantized with a per-block transform."""

    def __init__(self, fmt, kind, Wt, Sx=None, device="cuda", build_host=True, Tx=None, Tw=None):
        """Wt: host float32 [d_out][d_in]; Sx: host float32 [d_in/bs][bs][bs] moments.

        The transform pair is built on the host by wush_build_transforms unless
        Tx / Tw (host float32 [nblk][bs][bs]) are given.
        """
        self.fmt, self.kind = fmt, kind
        self.bs = W.BLOCK[fmt]
        Wt = np.ascontiguousarray(Wt, dtype=np.float32)
        self.d_out, self.d_in = Wt.shape
        nblk = self.d_in // self.bs
        if Tx is None:
            Tx = np.empty((nblk, self.bs, self.bs), np.float32)
            Tw = np.empty_like(Tx)
            if kind in ("wus", "wush") and Sx is None:
                raise ValueError("WUS/WUSH need activation moments Sx")
            W.wush_build_transforms(kind, self.bs, Wt, None if Sx is None else np.ascontiguousarray(Sx, np.float32),
                                    Tx, Tw)
        self.Tx_host, self.Tw_host = Tx, Tw
        self.identity = kind == "identity"
        self.Tx = None if self.identity else torch.from_numpy(np.ascontiguousarray(Tx)).to(device)
        self.Tw = None if self.identity else torch.from_numpy(np.ascontiguousarray(Tw)).to(device)
        Wd = torch.from_numpy(Wt).to(device)
        self.w_codes = torch.empty(codes_shape(self.d_out, self.d_in), dtype=torch.uint8, device=device)
        self.w_scales = torch.empty((self.d_out, nblk), dtype=scales_dtype(fmt), device=device)
        self.w_g = W.wush_pack_weights(fmt, Wd, self.Tw, self.w_codes, self.w_scales)
        del Wd
        self.x_g = 1.0

    def calibrate(self, X):
        """NVFP4 only: per-tensor activation scale from calibration activations (device tensor)."""
        if self.fmt == "nvfp4":
            self.x_g = W.wush_nvfp4_global_scale(X, self.Tx)
        return self.x_g

    def alloc_activation_codes(self, n, device="cuda"):
        nblk = self.d_in // self.bs
        return (torch.empty(codes_shape(n, self.d_in), dtype=torch.uint8, device=device),
                torch.empty((n, nblk), dtype=scales_dtype(self.fmt), device=device))

    def quantize(self, X, codes, scales):
        W.wush_transform_quant(self.fmt, X, self.Tx, codes, scales, g=self.x_g)

    def matmul(self, codes, scales, Y):
        n = codes.shape[0]
        need = W.wush_w4a4_gemm_ws_bytes(self.fmt, n, self.d_out, self.d_in)
        W.wush_w4a4_gemm(self.fmt, codes, scales, self.w_codes, self.w_scales, Y, a_g=self.x_g, b_g=self.w_g,
                         ws=_scratch(need, codes.device) if need else None)

    def forward(self, X, out=None, adapters=None, requests=None):
        """X W^T from the quantized operands; with an AdapterSet and the requests that X is made of, their adapters
        are added to it in place."""
        n = X.shape[0]
        codes, scales = self.alloc_activation_codes(n, X.device)
        self.quantize(X, codes, scales)
        Y = out if out is not None else torch.empty((n, self.d_out), dtype=torch.float32, device=X.device)
        self.matmul(codes, scales, Y)
        if adapters is not None:
            adapters.forward(X, requests, Y, out=Y)
        return Y


def request_table(lengths, adapters, device="cuda"):
    """(offsets, adapter ids) on the device: request i has lengths[i] tokens and adapter adapters[i], -1 for none."""
    off = np.concatenate(([0], np.cumsum(np.asarray(lengths, np.int64)))).astype(np.int32)
    return torch.from_numpy(off).to(device), torch.tensor(adapters, dtype=torch.int32, device=device)


class AdapterSet:
    """Low-rank adapters beside one projection d_in -> d_out.

    ``A`` [nad][rmax][d_in] and ``Bt`` [nad][rmax][d_out] are bfloat16 (Bt is the transpose of the usual B and starts at
    zero), ``rank`` and ``alpha`` per adapter.  A request table (see ``request_table``) says whose tokens are whose.  Calls
    run on the current stream and keep nothing in the set: one set serves several streams and captured graphs at a time.
    """

    def __init__(self, nad, rmax, d_in, d_out, rank=None, alpha=1.0, device="cuda", seed=0):
        self.nad, self.rmax, self.d_in, self.d_out = nad, rmax, d_in, d_out
        r = np.random.default_rng([seed, nad, d_in])
        A = (r.standard_normal((nad, rmax, d_in)) / np.sqrt(d_in)).astype(np.float32)
        self.A = torch.from_numpy(A).to(device).to(torch.bfloat16)
        self.Bt = torch.zeros((nad, rmax, d_out), dtype=torch.bfloat16, device=device)
        self.rank = torch.tensor([rmax] * nad if rank is None else list(rank), dtype=torch.int32, device=device)
        self.alpha = torch.tensor([float(alpha)] * nad if np.isscalar(alpha) else list(alpha), dtype=torch.float32,
                                  device=device)

    def forward(self, X, requests, Y0, out=None, keep=False):
        """Y = Y0 + alpha X A^T Bt, per request; with ``keep`` also V, which the backward pass needs."""
        off, ids = requests
        n = X.shape[0]
        Y = out if out is not None else torch.empty_like(Y0)
        V = torch.empty((n, self.rmax), dtype=torch.float32, device=X.device) if keep else None
        ws = _scratch(W.wush_adapter_ws_bytes(n, self.d_in, ids.shape[0], self.rmax), X.device)
        W.wush_adapter_forward(X, off, ids, self.A, self.Bt, self.rank, self.alpha, Y0, Y, V=V, ws=ws)
        return (Y, V) if keep else Y

    def backward(self, dY, X, requests, V, dX0=None, x_scales=None, dx_dtype=torch.bfloat16):
        """(dX, dA, dBt); X may be the codes of an act8 checkpoint, with their scales in ``x_scales``."""
        off, ids = requests
        n, dev = dY.shape[0], dY.device
        dX = torch.empty((n, self.d_in), dtype=dx_dtype if dX0 is None else dX0.dtype, device=dev)
        dA = torch.empty((self.nad, self.rmax, self.d_in), dtype=torch.float32, device=dev)
        dBt = torch.empty((self.nad, self.rmax, self.d_out), dtype=torch.float32, device=dev)
        ws = _scratch(W.wush_adapter_backward_ws_bytes(n, self.d_in, self.d_out, ids.shape[0], self.nad, self.rmax), dev)
        W.wush_adapter_backward(dY, X, off, ids, self.A, self.Bt, self.rank, self.alpha, V, dX0, dX, dA, dBt,
                                x_scales=x_scales, ws=ws)
        return dX, dA, dBt


def act8_store(X):
    """(codes, scales) of an act8 checkpoint of X."""
    n, d = X.shape
    codes = torch.empty((n, d), dtype=torch.int8, device=X.device)
    scales = torch.empty((n, d // 32), dtype=torch.uint8, device=X.device)
    W.wush_act8_pack(X, codes, scales)
    return codes, scales
