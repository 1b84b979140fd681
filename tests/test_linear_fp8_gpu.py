"""Linear layer on block-scaled e4m3 operands: forward and backward against the
float64 oracle, element by element.

Bound of an fp32 result: the products are exact; the sum of K terms in fp32, in
any order, is off by at most K * 2^-24 of the sum of the absolute terms to first
order.  The gate is 4 K * 2^-24 of that sum (the projection's gate: tensor-core
sums may truncate instead of rounding), plus 8 * 2^-24 for the scales' product,
the scaled addition and the bias; results of other types add one rounding."""
import numpy as np
import pytest
import torch

import deformable_convolution_core_b200 as dcn
from oracle import block as ob
from tests.block_testutil import Guarded, TORCH, U, assert_within, dev, host

pytestmark = pytest.mark.gpu


def random_operand(rng, rows, cols, block_rows):
    """Random codes of every value but NaN, NaN codes behind each row's end (they
    must not be used), scales over some binades."""
    q = rng.integers(0, 256, (rows, ob.pitch(cols)), dtype=np.uint8)
    q[(q & 127) == 127] = 56
    q[:, cols:] = 127
    r = -(-rows // block_rows)
    s = np.exp2(rng.uniform(-12, -6, (ob.blocks(cols), r))).astype(np.float32)
    return q, s


def bound_of(K, mag):
    return (4 * K + 8) * U * mag


def forward(a, sa, w, sw, M, K, N, bias, out_dtype, stream=None):
    out = Guarded((M, N), TORCH[out_dtype])
    nbytes = dcn.dcn_core_linear_fp8_workspace(M, K, N)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda") if nbytes else None
    args = [dev(v) for v in (a, sa, w, sw, bias)]
    torch.cuda.synchronize()
    dcn.dcn_core_linear_fp8(args[0], args[1], M, K, args[2], args[3], N, args[4], out.t, out_dtype,
                            ws, nbytes, stream)
    torch.cuda.synchronize()
    dcn.dcn_core_sync_status()
    assert out.untouched()
    return out.t


SIZES = [  # rows, inner, columns
    (1, 16, 8), (1, 1, 1), (1, 160, 640), (3, 37, 5), (8, 5120, 75), (8, 1300, 1000), (7, 20000, 24), (9, 64, 40),
    (16, 128, 128), (17, 300, 200), (31, 5120, 130),
    (32, 640, 160), (33, 16, 8), (40, 1, 1), (64, 31, 17), (100, 5120, 200), (128, 128, 128),
    (129, 160, 640), (200, 336, 450), (300, 1280, 333), (1000, 640, 161), (2000, 200, 257),
    (19000, 136, 200), (19100, 129, 391)]


@pytest.mark.parametrize("out_dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_linear_matches_the_oracle(M, K, N, out_dtype):
    rng = np.random.default_rng(M * 7 + K * 3 + N)
    a, sa = random_operand(rng, M, K, 1)
    w, sw = random_operand(rng, N, K, 128)
    bias = None if M % 2 else rng.standard_normal(N).astype(np.float32)
    got = forward(a, sa, w, sw, M, K, N, bias, out_dtype)
    ref, mag = ob.linear_fp8(a, sa, w, sw, K, bias)
    assert_within(host(got), ref, bound_of(K, mag), out_dtype, f"{M}x{K}x{N}")


@pytest.mark.parametrize("M", [5, 200])
def test_nan_block_reaches_its_row_only(M):
    rng = np.random.default_rng(M)
    a, sa = random_operand(rng, M, 300, 1)
    w, sw = random_operand(rng, 150, 300, 128)
    a[3, 128:256], sa[1, 3] = 127, np.nan
    w[140:, 256:300], sw[2, 1] = 127, np.nan
    got = host(forward(a, sa, w, sw, M, 300, 150, None, "f32"))
    nan = np.zeros((M, 150), dtype=bool)
    nan[3], nan[:, 128:] = True, True
    assert np.array_equal(np.isnan(got), nan)


def test_same_bits_every_time():
    rng = np.random.default_rng(9)
    for M, K, N in [(7, 1280, 320), (100, 5120, 200), (1000, 640, 160)]:
        a, sa = random_operand(rng, M, K, 1)
        w, sw = random_operand(rng, N, K, 128)
        first = forward(a, sa, w, sw, M, K, N, None, "f32")
        for _ in range(3):
            assert torch.equal(first, forward(a, sa, w, sw, M, K, N, None, "f32"))


def test_zero_scales_give_the_bias():
    a, sa = random_operand(np.random.default_rng(1), 200, 256, 1)
    w, sw = random_operand(np.random.default_rng(2), 64, 256, 128)
    bias = np.arange(64, dtype=np.float32)
    got = host(forward(a, np.zeros_like(sa), w, sw, 200, 256, 64, bias, "f16"))
    assert np.array_equal(got, np.tile(bias, (200, 1)))


def test_operand_of_more_than_2_31_values():
    M, K, N = 4_200_000, 528, 24
    rng = np.random.default_rng(3)
    w, sw = random_operand(rng, N, K, 128)
    g = torch.Generator("cuda").manual_seed(1)
    a = torch.randint(0, 120, (M, K), dtype=torch.uint8, device="cuda", generator=g)
    sa = torch.rand(ob.blocks(K), M, device="cuda", generator=g) * 2.0 ** -8
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    assert dcn.dcn_core_linear_fp8_workspace(M, K, N) == 0
    dcn.dcn_core_linear_fp8(a, sa, M, K, dev(w), dev(sw), N, None, out, "bf16")
    dcn.dcn_core_sync_status()
    for r in (0, 2_034_000, 4_067_300, M - 100):  # the last ones behind 2^31
        rows = slice(r, r + 100)
        ref, mag = ob.linear_fp8(host(a[rows]), host(sa[:, rows]), w, sw, K)
        assert_within(host(out[rows]), ref, bound_of(K, mag), "bf16", f"rows {r}")


def test_output_of_more_than_2_31_values():
    M, K, N = 1_100_000, 16, 2048
    rng = np.random.default_rng(4)
    w, sw = random_operand(rng, N, K, 128)
    g = torch.Generator("cuda").manual_seed(2)
    a = torch.randint(0, 120, (M, K), dtype=torch.uint8, device="cuda", generator=g)
    sa = torch.rand(1, M, device="cuda", generator=g)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    dcn.dcn_core_linear_fp8(a, sa, M, K, dev(w), dev(sw), N, None, out, "bf16")
    dcn.dcn_core_sync_status()
    for r in (0, 1_048_500, M - 100):
        rows = slice(r, r + 100)
        ref, mag = ob.linear_fp8(host(a[rows]), host(sa[:, rows]), w, sw, K)
        assert_within(host(out[rows]), ref, bound_of(K, mag), "bf16", f"rows {r}")


# ---------------------------------------------------------------------------
def backward(x, w, dy, M, K, N, dtype, want=(True, True, True)):
    """x (M, K), w (N, K) as fp32 arrays, dy a device tensor; the operands come
    from the library's quantiser as a program takes them."""
    xd, wd = dev(x, "f32"), dev(w, "f32")
    xt = torch.empty(K, ob.pitch(M), dtype=torch.uint8, device="cuda")
    xts = torch.empty(ob.blocks(M), K, device="cuda")
    dcn.dcn_core_quantize_fp8(xd, M, K, "f32", 1, None, None, xt, xts)
    wt = torch.empty(K, ob.pitch(N), dtype=torch.uint8, device="cuda")
    wts = torch.empty(ob.blocks(N), ob.blocks(K), device="cuda")
    dcn.dcn_core_quantize_fp8(wd, N, K, "f32", 128, None, None, wt, wts)
    gi = Guarded((M, K), TORCH[dtype]) if want[0] else None
    gw = Guarded((N, K), torch.float32) if want[1] else None
    gb = Guarded((N,), torch.float32) if want[2] else None
    nbytes = dcn.dcn_core_linear_fp8_backward_workspace(M, K, N)
    ws = Guarded((nbytes,), torch.uint8)
    dcn.dcn_core_linear_fp8_backward(dy, dtype, M, K, N, wt if want[0] else None, wts if want[0] else None,
                                     xt if want[1] else None, xts if want[1] else None,
                                     gi.t if gi else None, gw.t if gw else None, gb.t if gb else None,
                                     ws.t, nbytes)
    torch.cuda.synchronize()
    dcn.dcn_core_sync_status()
    assert all(g is None or g.untouched() for g in (gi, gw, gb, ws))
    return [None if g is None else host(g.t) for g in (gi, gw, gb)], (host(wt), host(wts), host(xt), host(xts))


def check_backward(dy, got, ops, M, K, N, dtype):
    gi, gw, gb = got
    wt, wts, xt, xts = ops
    dyh = host(dy)
    if gi is not None:
        q, s = ob.quantize(dyh)
        ref, mag = ob.linear_fp8(q, s, wt, wts, N)
        assert_within(gi, ref, bound_of(N, mag), dtype, "grad_input")
    if gw is not None:
        q, s = ob.quantize(np.ascontiguousarray(dyh.T))
        a, b = ob.values(q, s, M), ob.values(xt, xts, M)
        assert_within(gw, a @ b.T, bound_of(M, np.abs(a) @ np.abs(b).T), "f32", "grad_weight")
    if gb is not None:
        # an fp32 sum of M terms
        assert_within(gb, dyh.sum(0), M * U * np.abs(dyh).sum(0), "f32", "grad_bias")


BACK_SIZES = [(1, 16, 8), (5, 160, 64), (33, 17, 130), (200, 336, 45), (1003, 168, 331), (4000, 64, 96),
              (130, 1280, 640), (3000, 640, 200)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,N", BACK_SIZES)
def test_linear_backward_matches_the_oracle(M, K, N, dtype):
    rng = np.random.default_rng(M + K + N)
    x, w = rng.standard_normal((M, K)), rng.standard_normal((N, K)) / np.sqrt(K)
    dy = dev(1e-2 * rng.standard_normal((M, N)), dtype)
    got, ops = backward(x, w, dy, M, K, N, dtype)
    check_backward(dy, got, ops, M, K, N, dtype)


@pytest.mark.parametrize("want", [(True, False, False), (False, True, False), (False, False, True)])
def test_each_gradient_alone(want):
    M, K, N = 300, 160, 72
    rng = np.random.default_rng(8)
    dy = dev(rng.standard_normal((M, N)), "bf16")
    got, ops = backward(rng.standard_normal((M, K)), rng.standard_normal((N, K)), dy, M, K, N, "bf16", want)
    check_backward(dy, got, ops, M, K, N, "bf16")


def test_backward_is_the_derivative_of_the_forward():
    """The forward is linear in the values its operands stand for: a change of one
    input value by its scale times a code step moves the output by the step times
    the weight row, which grad_input sums.  <dy, out(a + d) - out(a)> = <grad_input, d>
    up to the quantisation of dy, so dy has few bits."""
    rng = np.random.default_rng(12)
    M, K, N = 200, 256, 128
    a, sa = random_operand(rng, M, K, 1)
    b = a.copy()
    b[::3, ::5] = 56  # the code of 1
    w, sw = random_operand(rng, N, K, 128)
    dy = np.where(rng.random((M, N)) < 0.5, -1.0, 1.0)  # exact in e4m3
    wv = dev(ob.values(w, sw, K, 128).astype(np.float32))
    wt = torch.empty(K, ob.pitch(N), dtype=torch.uint8, device="cuda")
    wts = torch.empty(ob.blocks(N), ob.blocks(K), device="cuda")
    dcn.dcn_core_quantize_fp8(wv, N, K, "f32", 128, None, None, wt, wts)
    w2, sw2 = ob.quantize(host(wv), 128)  # the same values in the quantiser's own scales
    out = [host(forward(v, sa, w2, sw2, M, K, N, None, "f32")) for v in (a, b)]
    gi = torch.empty(M, K, device="cuda")
    nbytes = dcn.dcn_core_linear_fp8_backward_workspace(M, K, N)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    dcn.dcn_core_linear_fp8_backward(dev(dy), "f32", M, K, N, wt, wts, None, None, gi, None, None, ws, nbytes)
    dcn.dcn_core_sync_status()
    d = ob.values(b, sa, K) - ob.values(a, sa, K)
    av, bv, w2v = ob.values(a, sa, K), ob.values(b, sa, K), ob.values(w2, sw2, K, 128)
    noise = bound_of(K, (np.abs(av) + np.abs(bv)) @ np.abs(w2v).T).sum()
    noise += (bound_of(N, np.abs(dy) @ np.abs(w2v)) * np.abs(d)).sum()
    assert abs((dy * (out[1] - out[0])).sum() - (host(gi) * d).sum()) <= noise


def test_missing_and_short_workspaces_are_refused():
    M, K, N = 100, 5120, 200
    need = dcn.dcn_core_linear_fp8_workspace(M, K, N)
    assert need > 0
    rng = np.random.default_rng(1)
    a, sa = random_operand(rng, M, K, 1)
    w, sw = random_operand(rng, N, K, 128)
    args = [dev(a), dev(sa), M, K, dev(w), dev(sw), N, None, torch.empty(M, N, device="cuda"), "f32"]
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for w_, n in ((None, 0), (ws, need - 16)):
        with pytest.raises(dcn.DcnError) as e:
            dcn.dcn_core_linear_fp8(*args, w_, n)
        assert e.value.status == dcn.DCN_ERR_INVALID_ARG
    dcn.dcn_core_sync_status()
