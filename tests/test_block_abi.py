"""Refusals of the block operators: the library's before any launch (raw
addresses, nothing is dereferenced) and the binding's of tensors that do not fit.
Runs without a GPU."""
import os
import re

import pytest
import torch

import deformable_convolution_core_b200 as dcn
from deformable_convolution_core_b200 import build as dcn_build
from tests.conftest import ROOT

FAKE = 1 << 20  # aligned; never dereferenced here
INVALID, UNSUPPORTED = dcn.DCN_ERR_INVALID_ARG, dcn.DCN_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    dcn_build.build()
    return dcn.load_library()


def refused(status, call, *args):
    with pytest.raises(dcn.DcnError) as e:
        call(*args)
    assert e.value.status == status


def changed(good, **change):
    """The positional arguments of `good` (an ordered dict) with some replaced."""
    assert set(change) <= set(good)
    return list({**good, **change}.values())


def test_struct_mirrors_the_header():
    text = open(os.path.join(ROOT, "include", "dcn_core.h")).read()
    body = re.search(r"typedef struct \{([^{}]*)\} dcn_block_norm;", text, re.S).group(1)
    names = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        names += [n.strip() for n in decl.split(None, 1)[1].split(",")]
    assert names == [n for n, _ in dcn.DcnBlockNorm._fields_]


def test_every_declared_entry_point_is_in_the_binding():
    text = open(os.path.join(ROOT, "include", "dcn_core.h")).read()
    names = set(re.findall(r"DCN_API\s+[\w\s\*]+?\b(\w+)\s*\(", text))
    assert names == set(dcn.EXPORTED_SYMBOLS)
    for n in names:
        assert callable(getattr(dcn, n))


def test_pitch():
    assert [dcn.dcn_core_fp8_pitch(n) for n in (0, -3, 1, 16, 17, 160, 2**31 - 1)] == [
        0, 0, 16, 16, 32, 160, 2**31]


QUANT = dict(input=FAKE, rows=4, cols=40, dtype="bf16", block_rows=1, q=FAKE, scales=FAKE, q_t=FAKE,
             scales_t=FAKE, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(input=None), INVALID), (dict(rows=0), INVALID), (dict(cols=0), INVALID),
    (dict(cols=-5), INVALID), (dict(dtype=3), INVALID), (dict(block_rows=64), INVALID),
    (dict(block_rows=0), INVALID), (dict(q=None), INVALID), (dict(scales=None), INVALID),
    (dict(q_t=None), INVALID), (dict(scales_t=None), INVALID),
    (dict(q=None, scales=None, q_t=None, scales_t=None), INVALID),
    (dict(rows=2**31 - 1), UNSUPPORTED), (dict(cols=2**31 - 65535), UNSUPPORTED),
    (dict(input=FAKE + 8), UNSUPPORTED), (dict(q=FAKE + 1), UNSUPPORTED),
    (dict(q_t=FAKE + 4), UNSUPPORTED), (dict(scales=FAKE + 2), UNSUPPORTED),
])
def test_quantize_refuses(change, status):
    refused(status, dcn.dcn_core_quantize_fp8, *changed(QUANT, **change))


LINEAR = dict(input=FAKE, input_scales=FAKE, M=200, K=64, weight=FAKE, weight_scales=FAKE, Nout=32,
              bias=FAKE, output=FAKE, out_dtype="bf16", workspace=None, workspace_bytes=0, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(input=None), INVALID), (dict(input_scales=None), INVALID), (dict(weight=None), INVALID),
    (dict(weight_scales=None), INVALID), (dict(output=None), INVALID), (dict(M=0), INVALID),
    (dict(K=0), INVALID), (dict(Nout=-1), INVALID), (dict(out_dtype=9), INVALID),
    (dict(M=2**31 - 1), UNSUPPORTED), (dict(K=2**31 - 1), UNSUPPORTED),
    (dict(Nout=2**31 - 65535), UNSUPPORTED),
    (dict(input=FAKE + 4), UNSUPPORTED), (dict(weight=FAKE + 8), UNSUPPORTED),
    (dict(output=FAKE + 2), UNSUPPORTED), (dict(bias=FAKE + 2), UNSUPPORTED),
    (dict(workspace=FAKE + 4), UNSUPPORTED), (dict(input_scales=FAKE + 1), UNSUPPORTED),
])
def test_linear_refuses(change, status):
    refused(status, dcn.dcn_core_linear_fp8, *changed(LINEAR, **change))


BACK = dict(grad_out=FAKE, dtype="bf16", M=200, K=64, Nout=32, weight_t=FAKE, weight_t_scales=FAKE,
            input_t=FAKE, input_t_scales=FAKE, grad_input=FAKE, grad_weight=FAKE, grad_bias=FAKE,
            workspace=FAKE, workspace_bytes=1 << 30, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(grad_out=None), INVALID), (dict(M=0), INVALID), (dict(K=0), INVALID),
    (dict(Nout=0), INVALID), (dict(dtype=-1), INVALID), (dict(weight_t=None), INVALID),
    (dict(weight_t_scales=None), INVALID), (dict(input_t=None), INVALID),
    (dict(input_t_scales=None), INVALID), (dict(workspace=None), INVALID),
    (dict(grad_input=None, grad_weight=None, grad_bias=None), INVALID),
    (dict(M=2**31 - 1), UNSUPPORTED), (dict(K=2**31 - 1), UNSUPPORTED),
    (dict(grad_out=FAKE + 8), UNSUPPORTED), (dict(grad_weight=FAKE + 4), UNSUPPORTED),
    (dict(workspace=FAKE + 8), UNSUPPORTED), (dict(grad_bias=FAKE + 2), UNSUPPORTED),
])
def test_linear_backward_refuses(change, status):
    refused(status, dcn.dcn_core_linear_fp8_backward, *changed(BACK, **change))


def norm(**kw):
    return dcn.make_block_norm(**{**dict(M=6, C=40, post_norm="layer", pre_norm="rms"), **kw})


NORM = dict(norm=None, residual=FAKE, branch=FAKE, gate=FAKE, post_gamma=FAKE, post_beta=FAKE,
            pre_gamma=FAKE, pre_beta=FAKE, residual_out=FAKE, normed=FAKE, normed_scales=None,
            post_stats=FAKE, pre_stats=FAKE, stream=0)
NORM_BACK = dict(norm=None, residual_out=FAKE, branch=FAKE, gate=FAKE, post_gamma=FAKE,
                 post_beta=FAKE, pre_gamma=FAKE, post_stats=FAKE, pre_stats=FAKE,
                 grad_residual_out=FAKE, grad_normed=FAKE, grad_residual=FAKE, grad_branch=FAKE,
                 grad_gate=FAKE, grad_post_gamma=FAKE, grad_post_beta=FAKE, grad_pre_gamma=FAKE,
                 grad_pre_beta=FAKE, workspace=FAKE, workspace_bytes=1 << 30, stream=0)

BAD_NORMS = [
    (dict(M=0), INVALID), (dict(C=0), INVALID), (dict(rows_per_gate=-1), INVALID),
    (dict(stream_dtype=5), INVALID), (dict(branch_dtype=5), INVALID), (dict(post_norm=3), INVALID),
    (dict(pre_norm=-1), INVALID), (dict(post_eps=-1e-6), INVALID),
    (dict(pre_eps=float("inf")), INVALID), (dict(pre_eps=float("nan")), INVALID),
    (dict(residual_scale=float("nan")), INVALID), (dict(C=5121), UNSUPPORTED),
    (dict(stream_dtype="bf16", branch_dtype="f32"), UNSUPPORTED),
    (dict(stream_dtype="bf16", branch_dtype="f16"), UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", BAD_NORMS)
def test_both_norm_passes_refuse_the_description(change, status):
    p = norm(**change)
    refused(status, dcn.dcn_core_block_norm, *changed(NORM, norm=p))
    refused(status, dcn.dcn_core_block_norm_backward, *changed(NORM_BACK, norm=p))
    assert dcn.dcn_core_block_norm_backward_workspace(p) == 0


@pytest.mark.parametrize("desc,change,status", [
    ({}, dict(residual=None), INVALID),
    ({}, dict(residual_out=None, normed=None, pre_stats=None), INVALID),  # nothing to write
    ({}, dict(branch=None), INVALID),                                     # a post norm of nothing
    (dict(post_norm="none"), dict(branch=None, post_gamma=None, post_beta=None, post_stats=None),
     INVALID),                                                            # a gate of nothing
    (dict(post_norm="none"), dict(post_beta=None, post_stats=None), INVALID),
    (dict(post_norm="none"), dict(post_gamma=None, post_beta=None), INVALID),
    (dict(pre_norm="none"), {}, INVALID),
    (dict(pre_norm="none"), dict(pre_gamma=None, pre_beta=None, pre_stats=None), INVALID),
    ({}, dict(normed=None, normed_scales=FAKE), INVALID),
    ({}, dict(residual=FAKE + 8), UNSUPPORTED), ({}, dict(gate=FAKE + 4), UNSUPPORTED),
    ({}, dict(normed=FAKE + 2), UNSUPPORTED), ({}, dict(pre_stats=FAKE + 1), UNSUPPORTED),
])
def test_block_norm_refuses(desc, change, status):
    refused(status, dcn.dcn_core_block_norm, *changed(NORM, norm=norm(**desc), **change))


@pytest.mark.parametrize("desc,change,status", [
    ({}, dict(residual_out=None), INVALID), ({}, dict(pre_stats=None), INVALID),
    ({}, dict(grad_normed=None), INVALID), ({}, dict(post_stats=None), INVALID),
    ({}, dict(grad_branch=None), INVALID), ({}, dict(gate=None), INVALID),
    ({}, dict(branch=None), INVALID),
    (dict(pre_norm="none"), dict(pre_gamma=None, pre_stats=None, grad_pre_gamma=None,
                                 grad_pre_beta=None), INVALID),            # grad_normed of nothing
    (dict(pre_norm="none"), dict(pre_gamma=None, pre_stats=None, grad_normed=None,
                                 grad_pre_beta=None), INVALID),
    (dict(pre_norm="none"), dict(pre_gamma=None, pre_stats=None, grad_normed=None,
                                 grad_pre_gamma=None, grad_pre_beta=None, grad_residual_out=None),
     INVALID),                                                             # no gradient comes in
    (dict(post_norm="none"), dict(post_gamma=None, post_beta=None, post_stats=None), INVALID),
    ({}, dict(grad_gate=FAKE + 4), UNSUPPORTED), ({}, dict(grad_branch=FAKE + 8), UNSUPPORTED),
    ({}, dict(workspace=FAKE + 4), UNSUPPORTED), ({}, dict(post_stats=FAKE + 2), UNSUPPORTED),
])
def test_block_norm_backward_refuses(desc, change, status):
    refused(status, dcn.dcn_core_block_norm_backward,
            *changed(NORM_BACK, norm=norm(**desc), **change))


def test_binding_refuses_tensors_that_do_not_fit():
    host = torch.zeros(4, 40, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not on the current CUDA device"):
        dcn.dcn_core_quantize_fp8(*changed(QUANT, input=host))
    with pytest.raises(ValueError, match="contiguous"):
        dcn.dcn_core_quantize_fp8(*changed(QUANT, input=torch.zeros(40, 4).t()))
    with pytest.raises(TypeError):
        dcn.dcn_core_linear_fp8(*changed(LINEAR, input="codes"))
    with pytest.raises(ValueError, match="workspace"):
        dcn.dcn_core_linear_fp8(*changed(LINEAR, workspace=torch.zeros(8), workspace_bytes=64))
