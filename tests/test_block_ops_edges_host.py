"""Block norm, act8 and adapters without a GPU: refusals at the edges of what the kernels assume."""

import pytest

import aware_block_transforms_amd as W
from test_block_ops_host import L, ODD, P, norm_bwd


@pytest.mark.parametrize("kw", [dict(dwp=ODD), dict(dw=ODD), dict(kind=1, gate=P, dgate=ODD)])
def test_block_norm_bwd_refuses_unaligned_sums(kw):
    # the column sums are written 16 bytes at a time
    assert norm_bwd(**kw) == W.WUSH_E_ARG
    assert b"16-byte aligned" in L.wush_last_error()


@pytest.mark.parametrize("d", [2 ** 31 - 32, 2 ** 31 - 480])
def test_act8_refuses_rows_whose_columns_pass_31_bits(d):
    # the last piece of 512 columns of such a row ends past 2^31 - 1
    shape = W.WUSH_E_SHAPE
    assert L.wush_act8_pack(1, 1, d, P, P, P, None) == shape
    assert L.wush_act8_unpack(1, 1, d, P, P, P, None) == shape
    assert L.wush_act8_swiglu(1, 1, 1, d, P, P, d, P, P, P, P, P, None) == shape
    assert L.wush_act8_swiglu_bwd(1, 1, 1, d, P, P, P, P, P, P, P, d, None) == shape
    assert L.wush_act8_pack(1, 0, 2 ** 31 - 512, None, None, None, None) == W.WUSH_OK


def test_adapter_workspace_grows_with_adapters_by_their_lists_alone():
    # sums in parts are kept for adapters of several chunks only, and those are bounded by the launch
    need = [L.wush_adapter_backward_ws_bytes(16384, 5120, 17408, 12, nad, 64) for nad in (100, 1000)]
    assert 0 < need[1] - need[0] < 1 << 20, need
    assert need[1] < 1 << 28
