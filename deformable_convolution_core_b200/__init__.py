"""Python binding of the B200 deformable-convolution core (DCNv3 / DCNv4).

Argument marshalling only: every step of the operator runs in the CUDA
kernels of ``libdcncore.so`` behind the C ABI declared in
``include/dcn_core.h``.  The functions below carry the same names as the C
entry points.  Tensors may be given as torch tensors (their device pointer is
passed) or as raw integer addresses; streams as ``torch.cuda.Stream``, a raw
handle or None (the current torch stream).

There is no fallback: if the library is missing or a call fails, an
exception is raised.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# DCN_CORE_LIBRARY selects another build of the library, e.g. the
# bounds-checked libdcncore_checked.so.
LIB_PATH = os.environ.get("DCN_CORE_LIBRARY") or os.path.join(_HERE, "libdcncore.so")

# DCN_CORE_ABI_VERSION of include/dcn_core.h that DcnProblem mirrors.
ABI_VERSION = 5
DCN_OK, DCN_ERR_INVALID_ARG, DCN_ERR_UNSUPPORTED, DCN_ERR_CUDA, DCN_ERR_TIMEOUT = 0, 1, 2, 3, 4
DCN_ERR_OUT_OF_BOUNDS = 5  # only from the bounds-checked build
# Scratch the allocation-free backward owns per GPU (DCN_CORE_NOALLOC_SCRATCH_BYTES).
DCN_CORE_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024
DCN_F32, DCN_BF16, DCN_F16 = 0, 1, 2
# storage-type names accepted wherever a dtype is given as a string
DTYPES = {"f32": DCN_F32, "float32": DCN_F32, "bf16": DCN_BF16, "bfloat16": DCN_BF16,
          "f16": DCN_F16, "float16": DCN_F16}

# dcn_norm of include/dcn_core.h and the names accepted for it.
DCN_NORM_NONE, DCN_NORM_LAYER, DCN_NORM_RMS = 0, 1, 2
NORMS = {"none": DCN_NORM_NONE, "layer": DCN_NORM_LAYER, "rms": DCN_NORM_RMS}

# Every entry point of include/dcn_core.h.
EXPORTED_SYMBOLS = (
    "dcn_core_output_hw",
    "dcn_core_forward",
    "dcn_core_forward_host",
    "dcn_core_backward_workspace",
    "dcn_core_backward",
    "dcn_core_backward_host",
    "dcn_core_backward_noalloc",
    "dcn_core_backward_deterministic_workspace",
    "dcn_core_backward_deterministic",
    "dcn_core_offset_mask_guide",
    "dcn_core_offset_mask_projection",
    "dcn_core_linear_bf16",
    "dcn_core_offset_mask_guide_projection",
    "dcn_core_fp8_pitch",
    "dcn_core_quantize_fp8",
    "dcn_core_linear_fp8_workspace",
    "dcn_core_linear_fp8",
    "dcn_core_linear_fp8_backward_workspace",
    "dcn_core_linear_fp8_backward",
    "dcn_core_block_norm",
    "dcn_core_block_norm_backward_workspace",
    "dcn_core_block_norm_backward",
    "dcn_core_sync_status",
    "dcn_status_string",
    "dcn_core_abi_version",
)


class DcnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {dcn_status_string(status)} (status {status})")


class DcnProblem(ctypes.Structure):
    """Mirror of ``dcn_problem`` in include/dcn_core.h."""
    _fields_ = [("N", ctypes.c_int), ("H", ctypes.c_int), ("W", ctypes.c_int),
                ("G", ctypes.c_int), ("Cg", ctypes.c_int), ("K", ctypes.c_int),
                ("stride", ctypes.c_int), ("pad", ctypes.c_int), ("dilation", ctypes.c_int),
                ("offset_scale", ctypes.c_float), ("softmax", ctypes.c_int),
                ("dtype", ctypes.c_int), ("remove_center", ctypes.c_int),
                ("separate_axes", ctypes.c_int), ("stride_w", ctypes.c_int),
                ("pad_w", ctypes.c_int), ("dilation_w", ctypes.c_int)]

    def __repr__(self):
        return "DcnProblem(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


def make_problem(N, H, W, G, Cg, K=3, stride=1, pad=1, dilation=1, offset_scale=1.0,
                 softmax=1, dtype="f32", remove_center=0, stride_w=None, pad_w=None,
                 dilation_w=None) -> DcnProblem:
    """stride, pad and dilation apply to both axes unless a width value
    (stride_w, pad_w, dilation_w) is given; then they are the height axis's."""
    if isinstance(dtype, str):
        dtype = DTYPES[dtype]
    separate = stride_w is not None or pad_w is not None or dilation_w is not None
    sw = stride if stride_w is None else stride_w
    pw = pad if pad_w is None else pad_w
    dw = dilation if dilation_w is None else dilation_w
    return DcnProblem(int(N), int(H), int(W), int(G), int(Cg), int(K), int(stride), int(pad),
                      int(dilation), float(offset_scale), int(softmax), int(dtype),
                      int(remove_center), int(separate), int(sw), int(pw), int(dw))


def problem_for(wl) -> DcnProblem:
    """DcnProblem of a workload description (any object with the fields of
    gen.workloads.Workload)."""
    return make_problem(wl.N, wl.H, wl.W, wl.G, wl.Cg, wl.K, wl.stride, wl.pad, wl.dilation,
                        wl.offset_scale, wl.softmax, wl.dtype,
                        getattr(wl, "remove_center", 0))


class DcnBlockNorm(ctypes.Structure):
    """Mirror of ``dcn_block_norm`` in include/dcn_core.h."""
    _fields_ = [("M", ctypes.c_int), ("C", ctypes.c_int), ("rows_per_gate", ctypes.c_int),
                ("stream_dtype", ctypes.c_int), ("branch_dtype", ctypes.c_int),
                ("post_norm", ctypes.c_int), ("pre_norm", ctypes.c_int),
                ("post_eps", ctypes.c_float), ("pre_eps", ctypes.c_float),
                ("residual_scale", ctypes.c_float)]

    def __repr__(self):
        return "DcnBlockNorm(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


def make_block_norm(M, C, stream_dtype="bf16", branch_dtype=None, post_norm="none",
                    pre_norm="layer", rows_per_gate=0, post_eps=1e-6, pre_eps=1e-6,
                    residual_scale=1.0) -> DcnBlockNorm:
    """branch_dtype defaults to the stream's type; rows_per_gate = 0 is one gate
    vector for all rows."""
    if isinstance(stream_dtype, str):
        stream_dtype = DTYPES[stream_dtype]
    if branch_dtype is None:
        branch_dtype = stream_dtype
    elif isinstance(branch_dtype, str):
        branch_dtype = DTYPES[branch_dtype]
    post_norm = NORMS[post_norm] if isinstance(post_norm, str) else post_norm
    pre_norm = NORMS[pre_norm] if isinstance(pre_norm, str) else pre_norm
    return DcnBlockNorm(int(M), int(C), int(rows_per_gate), int(stream_dtype), int(branch_dtype),
                        int(post_norm), int(pre_norm), float(post_eps), float(pre_eps),
                        float(residual_scale))


def taps(problem: DcnProblem) -> int:
    """Taps per (pixel, group): K*K, or K*K - 1 with remove_center."""
    return problem.K * problem.K - (1 if problem.remove_center else 0)


_lib = None


def library_path() -> str:
    return LIB_PATH


def load_library():
    """Load libdcncore.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m deformable_convolution_core_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, pp = ctypes.c_void_p, ctypes.POINTER(DcnProblem)
    ip = ctypes.POINTER(ctypes.c_int)
    st = ctypes.c_int
    lib.dcn_core_output_hw.argtypes = [pp, ip, ip]
    lib.dcn_core_output_hw.restype = st
    lib.dcn_core_forward.argtypes = [pp, vp, vp, vp, vp, vp]
    lib.dcn_core_forward.restype = st
    lib.dcn_core_forward_host.argtypes = [pp] + [vp] * 9
    lib.dcn_core_forward_host.restype = st
    lib.dcn_core_backward_workspace.argtypes = [pp]
    lib.dcn_core_backward_workspace.restype = ctypes.c_size_t
    lib.dcn_core_backward.argtypes = [pp] + [vp] * 8 + [ctypes.c_size_t, vp]
    lib.dcn_core_backward.restype = st
    lib.dcn_core_backward_host.argtypes = [pp] + [vp] * 12 + [ctypes.c_size_t, vp]
    lib.dcn_core_backward_host.restype = st
    lib.dcn_core_backward_noalloc.argtypes = [pp] + [vp] * 8
    lib.dcn_core_backward_noalloc.restype = st
    lib.dcn_core_backward_deterministic_workspace.argtypes = [pp]
    lib.dcn_core_backward_deterministic_workspace.restype = ctypes.c_size_t
    lib.dcn_core_backward_deterministic.argtypes = [pp] + [vp] * 8 + [ctypes.c_size_t, vp]
    lib.dcn_core_backward_deterministic.restype = st
    lib.dcn_core_offset_mask_guide.argtypes = [pp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp]
    lib.dcn_core_offset_mask_guide.restype = st
    lib.dcn_core_offset_mask_projection.argtypes = [pp, vp, ctypes.c_int, vp, vp, vp, vp, vp]
    lib.dcn_core_offset_mask_projection.restype = st
    lib.dcn_core_offset_mask_guide_projection.argtypes = [pp, vp, vp, vp, vp, vp, ctypes.c_float,
                                                          vp, vp, vp, vp, vp]
    lib.dcn_core_offset_mask_guide_projection.restype = st
    lib.dcn_core_linear_bf16.argtypes = [vp, ctypes.c_int, ctypes.c_int, vp, ctypes.c_int, vp, vp,
                                         ctypes.c_int, vp]
    lib.dcn_core_linear_bf16.restype = st
    ci, sz, npp = ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(DcnBlockNorm)
    lib.dcn_core_fp8_pitch.argtypes = [ci]
    lib.dcn_core_fp8_pitch.restype = sz
    lib.dcn_core_quantize_fp8.argtypes = [vp, ci, ci, ci, ci, vp, vp, vp, vp, vp]
    lib.dcn_core_quantize_fp8.restype = st
    lib.dcn_core_linear_fp8_workspace.argtypes = [ci, ci, ci]
    lib.dcn_core_linear_fp8_workspace.restype = sz
    lib.dcn_core_linear_fp8.argtypes = [vp, vp, ci, ci, vp, vp, ci, vp, vp, ci, vp, sz, vp]
    lib.dcn_core_linear_fp8.restype = st
    lib.dcn_core_linear_fp8_backward_workspace.argtypes = [ci, ci, ci]
    lib.dcn_core_linear_fp8_backward_workspace.restype = sz
    lib.dcn_core_linear_fp8_backward.argtypes = [vp, ci, ci, ci, ci] + [vp] * 8 + [sz, vp]
    lib.dcn_core_linear_fp8_backward.restype = st
    lib.dcn_core_block_norm.argtypes = [npp] + [vp] * 13
    lib.dcn_core_block_norm.restype = st
    lib.dcn_core_block_norm_backward_workspace.argtypes = [npp]
    lib.dcn_core_block_norm_backward_workspace.restype = sz
    lib.dcn_core_block_norm_backward.argtypes = [npp] + [vp] * 18 + [sz, vp]
    lib.dcn_core_block_norm_backward.restype = st
    lib.dcn_core_sync_status.argtypes = [vp]
    lib.dcn_core_sync_status.restype = st
    lib.dcn_status_string.argtypes = [st]
    lib.dcn_status_string.restype = ctypes.c_char_p
    lib.dcn_core_abi_version.argtypes = []
    lib.dcn_core_abi_version.restype = ctypes.c_int
    if lib.dcn_core_abi_version() != ABI_VERSION:
        raise ImportError(f"{LIB_PATH} has ABI version {lib.dcn_core_abi_version()}, this binding "
                          f"expects {ABI_VERSION}: rebuild it")
    _lib = lib
    return lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        if not t.is_contiguous():
            raise ValueError("tensors passed to the C ABI must be contiguous")
        return t.data_ptr()
    raise TypeError(f"cannot pass {type(t)} as a pointer")


def _stream(s) -> int | None:
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int, where: str):
    if status != DCN_OK:
        raise DcnError(status, where)


def dcn_status_string(status: int) -> str:
    return load_library().dcn_status_string(int(status)).decode()


def dcn_core_abi_version() -> int:
    return int(load_library().dcn_core_abi_version())


def dcn_core_output_hw(problem: DcnProblem) -> tuple[int, int]:
    ho, wo = ctypes.c_int(0), ctypes.c_int(0)
    _check(load_library().dcn_core_output_hw(ctypes.byref(problem), ctypes.byref(ho),
                                             ctypes.byref(wo)), "dcn_core_output_hw")
    return ho.value, wo.value


def dcn_core_forward(problem: DcnProblem, input, offset, mask, output, stream=None) -> None:
    _check(load_library().dcn_core_forward(ctypes.byref(problem), _ptr(input), _ptr(offset),
                                           _ptr(mask), _ptr(output), _stream(stream)),
           "dcn_core_forward")


def dcn_core_forward_host(problem: DcnProblem, h_input, h_offset, h_mask, h_output, d_input,
                          d_offset, d_mask, d_output, stream=None) -> None:
    _check(load_library().dcn_core_forward_host(
        ctypes.byref(problem), _ptr(h_input), _ptr(h_offset), _ptr(h_mask), _ptr(h_output),
        _ptr(d_input), _ptr(d_offset), _ptr(d_mask), _ptr(d_output), _stream(stream)),
        "dcn_core_forward_host")


def dcn_core_backward_workspace(problem: DcnProblem) -> int:
    return int(load_library().dcn_core_backward_workspace(ctypes.byref(problem)))


def dcn_core_backward(problem: DcnProblem, input, offset, mask, grad_out, grad_input,
                      grad_offset, grad_mask, workspace=None, workspace_bytes=0,
                      stream=None) -> None:
    _check(load_library().dcn_core_backward(
        ctypes.byref(problem), _ptr(input), _ptr(offset), _ptr(mask), _ptr(grad_out),
        _ptr(grad_input), _ptr(grad_offset), _ptr(grad_mask), _ptr(workspace),
        int(workspace_bytes), _stream(stream)), "dcn_core_backward")


def dcn_core_backward_host(problem: DcnProblem, input, offset, mask, h_grad_out, h_grad_input,
                           h_grad_offset, h_grad_mask, d_grad_out, d_grad_input, d_grad_offset,
                           d_grad_mask, workspace=None, workspace_bytes=0, stream=None) -> None:
    """Backward with grad_out and the three gradients on (pinned) host
    buffers; input, offset and mask are the device tensors of the forward."""
    _check(load_library().dcn_core_backward_host(
        ctypes.byref(problem), _ptr(input), _ptr(offset), _ptr(mask), _ptr(h_grad_out),
        _ptr(h_grad_input), _ptr(h_grad_offset), _ptr(h_grad_mask), _ptr(d_grad_out),
        _ptr(d_grad_input), _ptr(d_grad_offset), _ptr(d_grad_mask), _ptr(workspace),
        int(workspace_bytes), _stream(stream)), "dcn_core_backward_host")


def dcn_core_backward_noalloc(problem: DcnProblem, input, offset, mask, grad_out, grad_input,
                              grad_offset, grad_mask, stream=None) -> None:
    """Backward without a workspace, for callers that cannot allocate device
    memory (see include/dcn_core.h).  For bf16 or fp16 storage the fp32 grad_input
    accumulator must fit the library's fixed DCN_CORE_NOALLOC_SCRATCH_BYTES
    array; calls that may overlap on the GPU must be serialised."""
    status = load_library().dcn_core_backward_noalloc(
        ctypes.byref(problem), _ptr(input), _ptr(offset), _ptr(mask), _ptr(grad_out),
        _ptr(grad_input), _ptr(grad_offset), _ptr(grad_mask), _stream(stream))
    if status == DCN_ERR_UNSUPPORTED and problem.dtype != DCN_F32:
        need = problem.N * problem.H * problem.W * problem.G * problem.Cg * 4
        if need > DCN_CORE_NOALLOC_SCRATCH_BYTES:
            raise DcnError(status, f"dcn_core_backward_noalloc: the fp32 accumulator of 2-byte storage needs {need} "
                                   f"bytes, more than the {DCN_CORE_NOALLOC_SCRATCH_BYTES} bytes "
                                   "of scratch this entry point owns")
    _check(status, "dcn_core_backward_noalloc")


def dcn_core_backward_deterministic_workspace(problem: DcnProblem) -> int:
    return int(load_library().dcn_core_backward_deterministic_workspace(ctypes.byref(problem)))


def dcn_core_backward_deterministic(problem: DcnProblem, input, offset, mask, grad_out,
                                    grad_input, grad_offset, grad_mask, workspace,
                                    workspace_bytes, stream=None) -> None:
    """Bitwise-reproducible backward (see include/dcn_core.h): grad_input is
    accumulated exactly in 64-bit fixed point inside `workspace`."""
    _check(load_library().dcn_core_backward_deterministic(
        ctypes.byref(problem), _ptr(input), _ptr(offset), _ptr(mask), _ptr(grad_out),
        _ptr(grad_input), _ptr(grad_offset), _ptr(grad_mask), _ptr(workspace),
        int(workspace_bytes), _stream(stream)), "dcn_core_backward_deterministic")


def dcn_core_offset_mask_guide(problem: DcnProblem, input, dw_weight, dw_bias, ln_gamma,
                               ln_beta, ln_eps: float, query, stream=None) -> None:
    """Depthwise 3x3 + LayerNorm + GELU of the block's input into the bf16
    query of the offset / mask projection (see include/dcn_core.h)."""
    _check(load_library().dcn_core_offset_mask_guide(
        ctypes.byref(problem), _ptr(input), _ptr(dw_weight), _ptr(dw_bias), _ptr(ln_gamma),
        _ptr(ln_beta), float(ln_eps), _ptr(query), _stream(stream)), "dcn_core_offset_mask_guide")


def dcn_core_offset_mask_projection(problem: DcnProblem, query, Cq: int, weight, bias, offset,
                                    mask, stream=None) -> None:
    """offset / mask = query @ weight.T + bias on the tensor cores (see
    include/dcn_core.h).  query (N, Ho, Wo, Cq) and weight (G*KK*3, Cq) are
    bf16; bias (G*KK*3) fp32 or None; offset and mask are written in the
    problem's storage type and the layouts dcn_core_forward reads."""
    _check(load_library().dcn_core_offset_mask_projection(
        ctypes.byref(problem), _ptr(query), int(Cq), _ptr(weight), _ptr(bias), _ptr(offset),
        _ptr(mask), _stream(stream)), "dcn_core_offset_mask_projection")


def dcn_core_offset_mask_guide_projection(problem: DcnProblem, input, dw_weight, dw_bias,
                                          ln_gamma, ln_beta, ln_eps: float, weight, bias, offset,
                                          mask, stream=None) -> None:
    """Guide features and offset / mask projection in one kernel (the query
    stays on chip; see include/dcn_core.h): the result of
    dcn_core_offset_mask_guide followed by dcn_core_offset_mask_projection."""
    _check(load_library().dcn_core_offset_mask_guide_projection(
        ctypes.byref(problem), _ptr(input), _ptr(dw_weight), _ptr(dw_bias), _ptr(ln_gamma),
        _ptr(ln_beta), float(ln_eps), _ptr(weight), _ptr(bias), _ptr(offset), _ptr(mask),
        _stream(stream)), "dcn_core_offset_mask_guide_projection")


def dcn_core_linear_bf16(input, M: int, K: int, weight, Nout: int, bias, output,
                         out_dtype="f32", stream=None) -> None:
    """output (M, Nout) = input (M, K) @ weight (Nout, K).T + bias on the tensor
    cores; bf16 operands, fp32 accumulation, output in out_dtype."""
    if isinstance(out_dtype, str):
        out_dtype = DTYPES[out_dtype]
    _check(load_library().dcn_core_linear_bf16(
        _ptr(input), int(M), int(K), _ptr(weight), int(Nout), _ptr(bias), _ptr(output),
        int(out_dtype), _stream(stream)), "dcn_core_linear_bf16")


# Torch types by dcn_dtype, and those a buffer of e4m3 codes may have: filled when the
# first tensor comes (the binding itself does not need torch).
_TORCH: dict = {}


def _torch_types() -> dict:
    if not _TORCH:
        import torch
        _TORCH.update({DCN_F32: (torch.float32,), DCN_BF16: (torch.bfloat16,),
                       DCN_F16: (torch.float16,), "codes": (torch.float8_e4m3fn, torch.uint8),
                       "device": getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                       "stream": torch.cuda.current_stream,
                       "raw_stream": getattr(torch._C, "_cuda_getCurrentRawStream", None)})
    return _TORCH


def _bad_arg(t, name: str, numel: int, dtypes):
    if not hasattr(t, "data_ptr"):
        raise TypeError(f"{name}: cannot pass {type(t)} as a pointer")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors passed to the C ABI must be contiguous")
    if not t.is_cuda or t.get_device() != _torch_types()["device"]():
        raise ValueError(f"{name}: the tensor is on {t.device}, not on the current CUDA device")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")


def _here() -> int | None:
    """The current CUDA device, or None without one."""
    try:
        return _torch_types()["device"]()
    except (AssertionError, RuntimeError):
        return None


# The tensors of one call of the block operators are checked and converted one by one:
# each must be contiguous, on the current device, of the named type and of exactly the
# number of elements that the sizes give (another size means that two tensors were
# mixed up).  None and raw addresses go through as they are.  A plain function: a call
# has up to 19 of them, and a short kernel ends before their checks do.
def _arg(t, name: str, numel: int, kind, device) -> int | None:
    if t is None:
        return None
    try:
        if (t.get_device() == device and t.dtype in _TORCH[kind] and t.numel() == numel
                and t.is_contiguous()):
            return t.data_ptr()
    except (AttributeError, TypeError, KeyError):
        if type(t) is int:
            return t
    _bad_arg(t, name, numel, _TORCH.get(kind, ()))


def _arg_workspace(t, nbytes: int, device) -> int | None:
    if t is None or type(t) is int:
        return t
    if t.nbytes < nbytes:
        raise ValueError(f"workspace: {nbytes} bytes named, the tensor has {t.nbytes}")
    if not t.is_contiguous() or t.get_device() != device:
        _bad_arg(t, "workspace", t.numel(), None)
    return t.data_ptr()


def _arg_stream(s, device) -> int | None:
    if s is not None:
        return s if type(s) is int else s.cuda_stream
    raw = _TORCH["raw_stream"]
    if raw is None or device is None:
        return _TORCH["stream"]().cuda_stream
    return raw(device)


def _ceil(a: int, b: int) -> int:
    return -(-a // b)


def dcn_core_fp8_pitch(cols: int) -> int:
    """Row pitch in bytes of an e4m3 matrix: 16 * ceil(cols / 16)."""
    return int(load_library().dcn_core_fp8_pitch(int(cols)))


def dcn_core_quantize_fp8(input, rows: int, cols: int, dtype, block_rows: int, q, scales, q_t=None,
                          scales_t=None, stream=None) -> None:
    """Block-scaled e4m3 of a (rows, cols) matrix, and of its transpose from the
    same read (see include/dcn_core.h).  q (rows, pitch(cols)) with scales
    (ceil(cols/128), rows) or, with block_rows = 128, (ceil(cols/128),
    ceil(rows/128)); q_t (cols, pitch(rows)) with scales_t likewise; either pair
    may be None."""
    if isinstance(dtype, str):
        dtype = DTYPES[dtype]
    rows, cols = int(rows), int(cols)
    kb, mb = _ceil(cols, 128), _ceil(rows, 128)
    whole = block_rows == 128
    here = _here()
    _check(load_library().dcn_core_quantize_fp8(
        _arg(input, "input", rows * cols, dtype, here), dtype, rows, cols, block_rows,
        _arg(q, "q", rows * _ceil(cols, 16) * 16, "codes", here),
        _arg(scales, "scales", kb * (mb if whole else rows), DCN_F32, here),
        _arg(q_t, "q_t", cols * _ceil(rows, 16) * 16, "codes", here),
        _arg(scales_t, "scales_t", mb * (kb if whole else cols), DCN_F32, here),
        _arg_stream(stream, here)),
        "dcn_core_quantize_fp8")


def dcn_core_linear_fp8_workspace(M: int, K: int, Nout: int) -> int:
    return int(load_library().dcn_core_linear_fp8_workspace(int(M), int(K), int(Nout)))


def dcn_core_linear_fp8(input, input_scales, M: int, K: int, weight, weight_scales, Nout: int, bias,
                        output, out_dtype="bf16", workspace=None, workspace_bytes=0,
                        stream=None) -> None:
    """output (M, Nout) = input (M, K) @ weight (Nout, K).T + bias on block-scaled
    e4m3 operands (see include/dcn_core.h): the input in blocks of 1 x 128, the
    weight in blocks of 128 x 128, output in out_dtype."""
    if isinstance(out_dtype, str):
        out_dtype = DTYPES[out_dtype]
    M, K, Nout = int(M), int(K), int(Nout)
    kb, pitch = _ceil(K, 128), _ceil(K, 16) * 16
    here = _here()
    _check(load_library().dcn_core_linear_fp8(
        _arg(input, "input", M * pitch, "codes", here),
        _arg(input_scales, "input_scales", kb * M, DCN_F32, here),
        M, K, _arg(weight, "weight", Nout * pitch, "codes", here),
        _arg(weight_scales, "weight_scales", kb * _ceil(Nout, 128), DCN_F32, here), Nout,
        _arg(bias, "bias", Nout, DCN_F32, here), _arg(output, "output", M * Nout, out_dtype, here),
        out_dtype,
        _arg_workspace(workspace, workspace_bytes, here),
        workspace_bytes, _arg_stream(stream, here)),
        "dcn_core_linear_fp8")


def dcn_core_linear_fp8_backward_workspace(M: int, K: int, Nout: int) -> int:
    return int(load_library().dcn_core_linear_fp8_backward_workspace(int(M), int(K), int(Nout)))


def dcn_core_linear_fp8_backward(grad_out, dtype, M: int, K: int, Nout: int, weight_t,
                                 weight_t_scales, input_t, input_t_scales, grad_input,
                                 grad_weight, grad_bias, workspace, workspace_bytes,
                                 stream=None) -> None:
    """Gradients of dcn_core_linear_fp8 (see include/dcn_core.h).  weight_t and
    input_t are the transposes dcn_core_quantize_fp8 writes (block_rows 128 and
    1); grad_input has grad_out's type, grad_weight and grad_bias are fp32; a
    gradient given as None is not computed."""
    if isinstance(dtype, str):
        dtype = DTYPES[dtype]
    M, K, Nout = int(M), int(K), int(Nout)
    nb, mb = _ceil(Nout, 128), _ceil(M, 128)
    here = _here()
    _check(load_library().dcn_core_linear_fp8_backward(
        _arg(grad_out, "grad_out", M * Nout, dtype, here), dtype, M, K, Nout,
        _arg(weight_t, "weight_t", K * _ceil(Nout, 16) * 16, "codes", here),
        _arg(weight_t_scales, "weight_t_scales", nb * _ceil(K, 128), DCN_F32, here),
        _arg(input_t, "input_t", K * _ceil(M, 16) * 16, "codes", here),
        _arg(input_t_scales, "input_t_scales", mb * K, DCN_F32, here),
        _arg(grad_input, "grad_input", M * K, dtype, here),
        _arg(grad_weight, "grad_weight", Nout * K, DCN_F32, here),
        _arg(grad_bias, "grad_bias", Nout, DCN_F32, here),
        _arg_workspace(workspace, workspace_bytes, here),
        workspace_bytes, _arg_stream(stream, here)), "dcn_core_linear_fp8_backward")


def dcn_core_block_norm(norm: DcnBlockNorm, residual, branch, gate, post_gamma, post_beta,
                        pre_gamma, pre_beta, residual_out, normed, normed_scales=None,
                        post_stats=None, pre_stats=None, stream=None) -> None:
    """Post norm, gate, residual scale and the next pre norm in one pass (see
    include/dcn_core.h).  With normed_scales given, normed takes e4m3 codes
    (M, pitch(C)): the input of dcn_core_linear_fp8."""
    M, C, sd, bd = norm.M, norm.C, norm.stream_dtype, norm.branch_dtype
    gates = _ceil(M, norm.rows_per_gate) if norm.rows_per_gate > 0 else 1
    fp8 = normed_scales is not None
    here = _here()
    _check(load_library().dcn_core_block_norm(
        ctypes.byref(norm), _arg(residual, "residual", M * C, sd, here),
        _arg(branch, "branch", M * C, bd, here),
        _arg(gate, "gate", gates * C, DCN_F32, here),
        _arg(post_gamma, "post_gamma", C, DCN_F32, here),
        _arg(post_beta, "post_beta", C, DCN_F32, here),
        _arg(pre_gamma, "pre_gamma", C, DCN_F32, here),
        _arg(pre_beta, "pre_beta", C, DCN_F32, here),
        _arg(residual_out, "residual_out", M * C, sd, here),
        _arg(normed, "normed", M * (_ceil(C, 16) * 16 if fp8 else C), "codes" if fp8 else bd, here),
        _arg(normed_scales, "normed_scales", _ceil(C, 128) * M, DCN_F32, here),
        _arg(post_stats, "post_stats", 2 * M, DCN_F32, here),
        _arg(pre_stats, "pre_stats", 2 * M, DCN_F32, here),
        _arg_stream(stream, here)), "dcn_core_block_norm")


def dcn_core_block_norm_backward_workspace(norm: DcnBlockNorm) -> int:
    return int(load_library().dcn_core_block_norm_backward_workspace(ctypes.byref(norm)))


def dcn_core_block_norm_backward(norm: DcnBlockNorm, residual_out, branch, gate, post_gamma,
                                 post_beta, pre_gamma, post_stats, pre_stats, grad_residual_out,
                                 grad_normed, grad_residual, grad_branch, grad_gate=None,
                                 grad_post_gamma=None, grad_post_beta=None, grad_pre_gamma=None,
                                 grad_pre_beta=None, workspace=None, workspace_bytes=0,
                                 stream=None) -> None:
    """Gradients of dcn_core_block_norm (see include/dcn_core.h); a gradient given
    as None is not computed."""
    M, C, sd, bd = norm.M, norm.C, norm.stream_dtype, norm.branch_dtype
    gates = _ceil(M, norm.rows_per_gate) if norm.rows_per_gate > 0 else 1
    here = _here()
    _check(load_library().dcn_core_block_norm_backward(
        ctypes.byref(norm), _arg(residual_out, "residual_out", M * C, sd, here),
        _arg(branch, "branch", M * C, bd, here), _arg(gate, "gate", gates * C, DCN_F32, here),
        _arg(post_gamma, "post_gamma", C, DCN_F32, here),
        _arg(post_beta, "post_beta", C, DCN_F32, here),
        _arg(pre_gamma, "pre_gamma", C, DCN_F32, here),
        _arg(post_stats, "post_stats", 2 * M, DCN_F32, here),
        _arg(pre_stats, "pre_stats", 2 * M, DCN_F32, here),
        _arg(grad_residual_out, "grad_residual_out", M * C, sd, here),
        _arg(grad_normed, "grad_normed", M * C, bd, here),
        _arg(grad_residual, "grad_residual", M * C, sd, here),
        _arg(grad_branch, "grad_branch", M * C, bd, here),
        _arg(grad_gate, "grad_gate", gates * C, DCN_F32, here),
        _arg(grad_post_gamma, "grad_post_gamma", C, DCN_F32, here),
        _arg(grad_post_beta, "grad_post_beta", C, DCN_F32, here),
        _arg(grad_pre_gamma, "grad_pre_gamma", C, DCN_F32, here),
        _arg(grad_pre_beta, "grad_pre_beta", C, DCN_F32, here),
        _arg_workspace(workspace, workspace_bytes, here),
        workspace_bytes, _arg_stream(stream, here)),
        "dcn_core_block_norm_backward")


def dcn_core_sync_status(stream=None) -> None:
    _check(load_library().dcn_core_sync_status(_stream(stream)), "dcn_core_sync_status")


__all__ = ["DcnProblem", "DcnBlockNorm", "DcnError", "make_problem", "make_block_norm", "problem_for", "taps", "load_library",
           "library_path", "EXPORTED_SYMBOLS", *EXPORTED_SYMBOLS, "ABI_VERSION",
           "DCN_CORE_NOALLOC_SCRATCH_BYTES",
           "DCN_OK", "DCN_ERR_INVALID_ARG", "DCN_ERR_UNSUPPORTED", "DCN_ERR_CUDA",
           "DCN_ERR_TIMEOUT", "DCN_ERR_OUT_OF_BOUNDS", "DCN_F32", "DCN_BF16", "DCN_F16",
           "DTYPES", "DCN_NORM_NONE", "DCN_NORM_LAYER", "DCN_NORM_RMS", "NORMS"]
