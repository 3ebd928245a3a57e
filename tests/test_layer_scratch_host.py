"""Workspaces of the layer helpers: every call has its own, without a GPU (the library's calls are recorded)."""

import torch

from aware_block_transforms_amd import layer


def test_calls_of_one_adapter_set_share_no_workspace(monkeypatch):
    # two streams may have a call each in flight, and a captured graph keeps the workspace of its own
    held = []
    monkeypatch.setattr(layer.W, "wush_adapter_forward", lambda *a, ws, **k: held.append(ws))
    monkeypatch.setattr(layer.W, "wush_adapter_backward", lambda *a, ws, **k: held.append(ws))
    ad = layer.AdapterSet(2, 16, 64, 96, device="cpu")
    req = layer.request_table([3, 5], [0, 1], device="cpu")
    X, Y0, V = torch.zeros(8, 64), torch.zeros(8, 96), torch.zeros(8, 16)
    for _ in range(2):
        ad.forward(X, req, Y0)
        ad.forward(X, req, Y0, keep=True)
        ad.backward(Y0, X, req, V)
    assert len(held) == 6 and len({t.data_ptr() for t in held}) == 6
    n, d_in, d_out, nseg, nad, rmax = 8, 64, 96, 2, 2, 16
    for i, t in enumerate(held):
        need = layer.W.wush_adapter_backward_ws_bytes(n, d_in, d_out, nseg, nad, rmax) if i % 3 == 2 else \
            layer.W.wush_adapter_ws_bytes(n, d_in, nseg, rmax)
        assert t.numel() >= need
    assert not any(torch.is_tensor(v) and v.data_ptr() in {t.data_ptr() for t in held} for v in vars(ad).values())


def test_calls_of_one_layer_share_no_workspace(monkeypatch):
    held = []
    monkeypatch.setattr(layer.W, "wush_w4a4_gemm", lambda *a, ws, **k: held.append(ws))
    L = object.__new__(layer.W4A4Layer)          # packing weights needs a GPU
    vars(L).update(fmt="mxfp4", bs=32, d_in=256, d_out=128, x_g=1.0, w_g=1.0, w_codes=None, w_scales=None)
    codes, scales = L.alloc_activation_codes(64, "cpu")
    for _ in range(3):
        L.matmul(codes, scales, torch.zeros(64, 128))
    need = layer.W.wush_w4a4_gemm_ws_bytes("mxfp4", 64, 128, 256)
    assert need > 0 and all(t.numel() >= need for t in held)
    assert len(held) == 3 and len({t.data_ptr() for t in held}) == 3
