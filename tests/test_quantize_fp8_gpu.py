"""Block-scaled e4m3 quantiser on the GPU.  Codes and scales are defined by fp32
operations, so they have to equal the oracle's bit for bit."""
import numpy as np
import pytest
import torch

import deformable_convolution_core_b200 as dcn
from oracle import block as ob
from tests.block_testutil import Guarded, TORCH, dev, host

pytestmark = pytest.mark.gpu


def bits(scales):
    return np.ascontiguousarray(scales, dtype=np.float32).view(np.uint32)


def same_scales(got, ref):
    g, r = np.asarray(got, np.float32), np.asarray(ref, np.float32)
    return np.array_equal(np.isnan(g), np.isnan(r)) and np.array_equal(bits(g)[~np.isnan(g)], bits(r)[~np.isnan(r)])


def run(x, dtype, block_rows, rows_out=True, trans_out=True, stream=None):
    rows, cols = x.shape
    kb, mb = ob.blocks(cols), ob.blocks(rows)
    whole = block_rows == 128
    g = {}
    if rows_out:
        g["q"] = Guarded((rows, ob.pitch(cols)), torch.uint8)
        g["s"] = Guarded((kb, mb if whole else rows), torch.float32)
    if trans_out:
        g["qt"] = Guarded((cols, ob.pitch(rows)), torch.uint8)
        g["st"] = Guarded((mb, kb if whole else cols), torch.float32)
    t = {k: v.t for k, v in g.items()}
    dcn.dcn_core_quantize_fp8(x, rows, cols, dtype, block_rows, t.get("q"), t.get("s"), t.get("qt"),
                              t.get("st"), stream)
    torch.cuda.synchronize()
    dcn.dcn_core_sync_status()
    assert all(v.untouched() for v in g.values())
    return {k: host(v) for k, v in t.items()}


def check(xh, got, block_rows):
    if "q" in got:
        q, s = ob.quantize(xh, block_rows)
        assert np.array_equal(got["q"], q) and same_scales(got["s"], s)
    if "qt" in got:
        q, s = ob.quantize(np.ascontiguousarray(xh.T), block_rows)
        assert np.array_equal(got["qt"], q) and same_scales(got["st"], s)


SHAPES = [(1, 1), (1, 160), (2, 8), (5, 129), (127, 128), (128, 128), (129, 127), (300, 160),
          (64, 1280), (257, 344), (1000, 24), (130, 1001)]


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_codes_and_scales_equal_the_oracle(rows, cols, dtype, block_rows):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-6, 6, (rows, 1)))
    xd = dev(x, dtype)
    check(host(xd), run(xd, dtype, block_rows), block_rows)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows_out,trans_out", [(True, False), (False, True)])
def test_either_output_alone(rows_out, trans_out, block_rows):
    x = dev(np.random.default_rng(1).standard_normal((200, 168)), "bf16")
    check(host(x), run(x, "bf16", block_rows, rows_out, trans_out), block_rows)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_the_whole_range_of_the_type(dtype):
    """Every binade of the type, ties of the code grid, subnormals, zeros and the largest values."""
    info = torch.finfo(TORCH[dtype])
    rng = np.random.default_rng(2)
    x = rng.standard_normal((64, 256)) * np.exp2(rng.uniform(np.log2(info.tiny), np.log2(info.max) - 3, (64, 256)))
    x[:8, :128] = np.repeat(ob.e4m3_values()[120:128].clip(max=448)[:8, None], 128, 1)  # exact codes
    x[8, :127] = (ob.e4m3_values()[:127] + np.append(ob.e4m3_values()[1:127], 448)) / 2  # ties
    x[8, 127] = 448
    x[9], x[10, :128], x[11, :] = 0, info.max, info.tiny / 4
    x = np.nan_to_num(x)
    xd = dev(x.astype(np.float32), dtype)
    for block_rows in (1, 128):
        check(host(xd), run(xd, dtype, block_rows), block_rows)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_nan_and_infinity_stay_in_their_block(block_rows):
    x = np.random.default_rng(3).standard_normal((300, 272)).astype(np.float32)
    x[5, 7], x[140, 200], x[299, 271], x[10, 130] = np.nan, np.inf, -np.inf, np.nan
    xd = dev(x, "bf16")
    check(host(xd), run(xd, "bf16", block_rows), block_rows)


def test_more_than_2_31_values():
    rows, cols = 4_200_000, 520
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 600_000):  # distinct values all over
        x[i:i + 600_000].normal_(generator=torch.Generator("cuda").manual_seed(i))
    q = torch.empty(rows, ob.pitch(cols), dtype=torch.uint8, device="cuda")
    s = torch.empty(ob.blocks(cols), rows, device="cuda")
    qt = torch.empty(cols, ob.pitch(rows), dtype=torch.uint8, device="cuda")
    st = torch.empty(ob.blocks(rows), cols, device="cuda")
    dcn.dcn_core_quantize_fp8(x, rows, cols, "bf16", 1, q, s, qt, st)
    dcn.dcn_core_sync_status()
    for r0 in (0, 2_065_000, rows - 128):  # blocks of rows, the last ones behind 2^31
        r0 = r0 // 128 * 128
        part = x[r0:r0 + 128]
        cq, cs = ob.quantize(host(part))
        n = part.shape[0]
        assert np.array_equal(host(q[r0:r0 + n]), cq) and same_scales(host(s[:, r0:r0 + n]), cs)
        cq, cs = ob.quantize(np.ascontiguousarray(host(part).T))
        assert np.array_equal(host(qt[:, r0:r0 + n]), cq[:, :n])
        assert same_scales(host(st[r0 // 128:r0 // 128 + 1]), cs)


def test_on_another_stream():
    x = dev(np.random.default_rng(4).standard_normal((500, 320)), "f16")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = run(x, "f16", 1, stream=s)
    check(host(x), got, 1)
