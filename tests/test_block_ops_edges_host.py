"""Block norm, act8 and adapters without a GPU: refusals at the edges of what the kernels assume."""

import pytest

import aware_block_transforms_amd as W
from test_block_ops_host import L, ODD, P, norm_bwd


@pytest.mark.parametrize("kw", [dict(dwp=ODD), dict(dw=ODD), dict(kind=1, gate=P, dgate=ODD)])
def test_block_norm_bwd_refuses_unaligned_sums(kw):
    # the column sums are written 16 bytes at a time
    assert norm_bwd(**kw) == W.WUSH_E_ARG
    assert b"16-byte aligned" in L.wush_last_error()
