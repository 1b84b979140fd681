"""Bounded waits of the block operators: with the test knob DCN_CORE_TEST_STALL=1 the
first load of every CTA is never issued, the waits give up after about a second, the
kernel sets the device error word and returns; dcn_core_sync_status reports
DCN_ERR_TIMEOUT and clears the word, and the next call works normally."""
import os

import numpy as np
import pytest
import torch

import deformable_convolution_core_b200 as dcn
from oracle import block as ob
from tests.block_testutil import dev

pytestmark = pytest.mark.gpu


def check(run, output):
    run()
    dcn.dcn_core_sync_status()
    want = output().clone()
    old = os.environ.get("DCN_CORE_TEST_STALL")
    os.environ["DCN_CORE_TEST_STALL"] = "1"
    try:
        run()
        with pytest.raises(dcn.DcnError) as e:
            dcn.dcn_core_sync_status()
        assert e.value.status == dcn.DCN_ERR_TIMEOUT
    finally:
        if old is None:
            os.environ.pop("DCN_CORE_TEST_STALL", None)
        else:
            os.environ["DCN_CORE_TEST_STALL"] = old
    run()
    dcn.dcn_core_sync_status()
    assert torch.equal(output(), want)


@pytest.mark.parametrize("M,K,N", [(300, 640, 200), (100, 5120, 200), (19000, 256, 300)])
def test_linear(M, K, N):
    rng = np.random.default_rng(M)
    a = dev(rng.integers(0, 120, (M, ob.pitch(K)), dtype=np.uint8))
    w = dev(rng.integers(0, 120, (N, ob.pitch(K)), dtype=np.uint8))
    sa, sw = torch.rand(ob.blocks(K), M, device="cuda"), torch.rand(ob.blocks(K), ob.blocks(N), device="cuda")
    out = torch.empty(M, N, device="cuda")
    n = dcn.dcn_core_linear_fp8_workspace(M, K, N)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    check(lambda: dcn.dcn_core_linear_fp8(a, sa, M, K, w, sw, N, None, out, "f32", ws, n), lambda: out)


@pytest.mark.parametrize("M,C,dtype", [(5000, 160, "bf16"), (700, 1280, "f32"), (900, 773, "f32")])
def test_block_norm_backward(M, C, dtype):
    """C = 1280 and 773: rows of several warps, whose barriers every thread still meets."""
    rng = np.random.default_rng(C)
    r, y, dr, dh = (dev(rng.standard_normal((M, C)).astype(np.float32), dtype) for _ in range(4))
    st = torch.ones(2, M, device="cuda")
    dx, dy = torch.empty_like(r), torch.empty_like(r)
    g = torch.empty(C, device="cuda")
    p = dcn.make_block_norm(M, C, dtype, post_norm="rms", pre_norm="layer")
    n = dcn.dcn_core_block_norm_backward_workspace(p)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    check(lambda: dcn.dcn_core_block_norm_backward(p, r, y, None, None, None, None, st, st, dr, dh, dx, dy,
                                                   grad_pre_gamma=g, workspace=ws, workspace_bytes=n), lambda: dy)
