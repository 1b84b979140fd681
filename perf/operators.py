"""The block operators around the deformable-convolution core, case by case.

Each case is one pass through one operator of the block: the norms on either
side of a branch with its gate and residual scale (forward, to the storage type
or to block-scaled e4m3, and backward), the quantiser to block-scaled e4m3, and
the linear layer on such operands (forward and backward).  ``run`` computes it
in plain torch operations, or, where ``own`` is true, with the library's entry
points.  ``exact`` is the same operator in 64 bits, written apart.

Definitions that all three share:
  * e4m3 blocks: over the 128 values of a block (1 x 128 of a row, or 128 x 128),
    a = max(max|x|, 7 * 2^-58), scale = fl32(a / 448), inv = fl32(448 / a),
    q = e4m3(fl32(x * inv)), rounded to nearest even.  A value stands for q * scale.
  * codes are stored with a row pitch of 16 * ceil(columns / 16), zeros behind the
    last column; scales as (blocks along the row, rows or blocks of 128 rows).
  * norms and sums are taken of unrounded 32-bit values; every output is rounded once.
"""
import math

import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_E4M3 = torch.float8_e4m3fn
_FLOOR = 7.0 * 2.0 ** -58


def listed():
    """The InternImage-L stages are 96^2 x 160, 48^2 x 320, 24^2 x 640 and
    12^2 x 1280 channels with 64 images; the MLP of a block is four times as wide."""
    return [
        # serving one token: the norm that closes a branch and opens the next one
        dict(name="norm: one row", op="norm", rows=1, channels=1280, stream="bf16", branch="bf16",
             post="layer", pre="layer", gates=1, fp8=True, train=False),
        # training, stage 1: layer scale, residual and the next LayerNorm, with what the backward keeps
        dict(name="norm: stage 1", op="norm", rows=64 * 96 * 96, channels=160, stream="bf16",
             branch="bf16", post="none", pre="layer", gates=1, fp8=False, train=True),
        # serving, stage 4: a 32-bit residual stream, the next operand straight to e4m3
        dict(name="norm: stage 4 to e4m3", op="norm", rows=64 * 12 * 12, channels=1280,
             stream="f32", branch="bf16", post="layer", pre="rms", gates=1, fp8=True, train=False),
        # training, stage 2: norms on both sides, one gate for each image (stochastic depth)
        dict(name="norm backward: stage 2", op="norm_backward", rows=64 * 48 * 48, channels=320,
             stream="bf16", branch="bf16", post="layer", pre="layer", gates=64),
        # an odd width and row count in 32 bits
        dict(name="norm backward: odd sizes", op="norm_backward", rows=4001, channels=773,
             stream="f32", branch="f32", post="rms", pre="rms", gates=1),
        # training, stage 3: the activations once along the rows and once transposed
        dict(name="quantise: stage 3", op="quantise", rows=64 * 24 * 24, cols=640, dtype="bf16",
             block_rows=1, both=True),
        # a weight of stage 4, laid out for the forward and the backward product
        dict(name="quantise: weight", op="quantise", rows=5120, cols=1280, dtype="f32",
             block_rows=128, both=True),
        # serving one token through the second layer of the stage-4 MLP
        dict(name="linear: one row", op="linear", rows=1, inner=5120, cols=1280, out="bf16",
             bias=True),
        # the first layer of the stage-1 MLP: many rows, a short inner length that ends inside a block
        dict(name="linear: stage 1", op="linear", rows=64 * 96 * 96, inner=160, cols=640,
             out="bf16", bias=True),
        # the first layer of the stage-4 MLP: the most arithmetic
        dict(name="linear: stage 4", op="linear", rows=64 * 12 * 12, inner=1280, cols=5120,
             out="bf16", bias=True),
        # training, the first layer of the stage-3 MLP
        dict(name="linear backward: stage 3", op="linear_backward", rows=64 * 24 * 24, inner=640,
             cols=2560, dtype="bf16"),
        # ragged in every dimension
        dict(name="linear backward: ragged", op="linear_backward", rows=1003, inner=168, cols=331,
             dtype="f32"),
    ]


def _size(rng, lo, hi):
    """A whole number whose logarithm is spread evenly; odd values stay odd."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """Channels: mostly multiples of 16, sometimes any number."""
    n = _size(rng, lo, hi)
    return n if rng.random() < 0.3 else max(16, n // 16 * 16)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "quantise", "linear", "linear", "linear_backward"])
    if op in ("norm", "norm_backward"):
        channels = _width(rng, 32, 5120)
        rows = _size(rng, 1, min(590000, 47_000_000 // channels))
        stream, branch = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16"),
                                     ("f32", "f16")])
        c = dict(op=op, rows=rows, channels=channels, stream=stream, branch=branch,
                 post=rng.choice(["none", "layer", "rms"]), pre=rng.choice(["layer", "rms"]),
                 gates=rng.choice([0, 1, min(rows, rng.randint(2, 64))]))
        if op == "norm":
            c["fp8"] = rng.random() < 0.5
            c["train"] = rng.random() < 0.5
        return c
    if op == "quantise":
        cols = _width(rng, 32, 5120)
        return dict(op=op, rows=_size(rng, 1, min(590000, 23_000_000 // cols)), cols=cols,
                    dtype=rng.choice(["f32", "bf16", "f16"]), block_rows=rng.choice([1, 128]),
                    both=rng.random() < 0.5)
    inner, cols = _width(rng, 32, 5120), _width(rng, 32, 5120)
    if op == "linear":
        most = min(590000, 60_000_000_000 // (inner * cols), 380_000_000 // cols)
        return dict(op=op, rows=_size(rng, 1, most), inner=inner, cols=cols,
                    out=rng.choice(["f32", "bf16", "f16"]), bias=rng.random() < 0.5)
    most = min(150000, 30_000_000_000 // (inner * cols), 95_000_000 // cols)
    return dict(op=op, rows=_size(rng, 1, most), inner=inner, cols=cols,
                dtype=rng.choice(["f32", "bf16", "f16"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pitch(cols):
    return (cols + 15) // 16 * 16


def _blocks(n):
    return (n + 127) // 128


def _activations(g, rows, cols, dtype):
    """Channels of differing size and centre, as a network's activations have them."""
    width = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    centre = 0.3 * torch.randn(cols, generator=g, device="cuda")
    return torch.randn(rows, cols, generator=g, device="cuda").mul_(width).add_(centre).to(_T[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": dict(case)}

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    def param(n, mean, std):
        return mean + std * torch.randn(n, generator=g, device="cuda")

    if op in ("norm", "norm_backward"):
        M, C = case["rows"], case["channels"]
        st, bt = _T[case["stream"]], _T[case["branch"]]
        s["x"] = _activations(g, M, C, case["stream"])
        s["y"] = _activations(g, M, C, case["branch"])
        s["post_gamma"] = param(C, 1.0, 0.2) if case["post"] != "none" else None
        s["post_beta"] = param(C, 0.0, 0.2) if case["post"] == "layer" else None
        s["pre_gamma"] = param(C, 1.0, 0.2)
        s["pre_beta"] = param(C, 0.0, 0.2) if case["pre"] == "layer" else None
        n = case["gates"]
        s["per_gate"] = -(-M // n) if n > 1 else 0
        n = -(-M // s["per_gate"]) if s["per_gate"] else n
        s["gate"] = param((n, C), 0.4, 0.2) if n else None
        if s["per_gate"]:  # stochastic depth: some images skip the branch
            s["gate"][torch.rand(n, generator=g, device="cuda") < 0.2] = 0.0
        s["alpha"] = 1.0
        if op == "norm":
            out = {"residual": empty(M, C, dtype=st)}
            if case["fp8"]:
                out["normed"] = empty(M, _pitch(C), dtype=_E4M3)
                out["scales"] = empty(_blocks(C), M)
            else:
                out["normed"] = empty(M, C, dtype=bt)
            if case["train"]:
                if case["post"] != "none":
                    out["post_stats"] = empty(2, M)
                out["pre_stats"] = empty(2, M)
            s["out"] = out
        else:
            fwd = _norm_plain(s["x"], s["y"], s, dict(case, fp8=False, train=True))
            s["r"], s["post_stats"], s["pre_stats"] = (fwd["residual"], fwd.get("post_stats"), fwd["pre_stats"])
            del fwd, s["x"]
            s["grad_residual_out"] = (1e-3 * torch.randn(M, C, generator=g, device="cuda")).to(st)
            s["grad_normed"] = (1e-3 * torch.randn(M, C, generator=g, device="cuda")).to(bt)
            out = {"residual": empty(M, C, dtype=st), "branch": empty(M, C, dtype=bt)}
            for k in ("gate", "post_gamma", "post_beta", "pre_gamma", "pre_beta"):
                if s[k] is not None:
                    out[k] = torch.empty_like(s[k])
            s["out"] = out
        return s
    if op == "quantise":
        M, K = case["rows"], case["cols"]
        s["x"] = _activations(g, M, K, case["dtype"])
        b = case["block_rows"]
        s["out"] = {"q": empty(M, _pitch(K), dtype=_E4M3),
                    "scales": empty(_blocks(K), _blocks(M) if b > 1 else M)}
        if case["both"]:
            s["out"]["q_t"] = empty(K, _pitch(M), dtype=_E4M3)
            s["out"]["scales_t"] = empty(_blocks(M), _blocks(K) if b > 1 else K)
        return s
    M, K, N = case["rows"], case["inner"], case["cols"]
    weight = torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)
    if op == "linear":
        s["a"], s["a_scales"] = _quantise_plain(_activations(g, M, K, "bf16"), 1)
        s["w"], s["w_scales"] = _quantise_plain(weight, 128)
        s["bias"] = param(N, 0.0, 0.2) if case["bias"] else None
        s["out"] = empty(M, N, dtype=_T[case["out"]])
        return s
    s["w_t"], s["w_t_scales"] = _quantise_plain(weight.t().contiguous(), 128)
    s["x_t"], s["x_t_scales"] = _quantise_plain(_activations(g, M, K, "bf16").t().contiguous(), 1)
    s["grad"] = (1e-3 * torch.randn(M, N, generator=g, device="cuda")).to(_T[case["dtype"]])
    s["out"] = {"input": empty(M, K, dtype=_T[case["dtype"]]), "weight": empty(N, K), "bias": empty(N)}
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _quantise_plain(x, block_rows):
    """(codes with their pitch, scales) of a 2-D tensor."""
    rows, cols = x.shape
    kb, rb = _blocks(cols), -(-rows // block_rows)
    v = torch.zeros(rb * block_rows, kb * 128, device=x.device)
    v[:rows, :cols] = x
    v = v.view(rb, block_rows, kb, 128)
    a = v.abs().amax(dim=(1, 3)).clamp_(min=_FLOOR)
    top = torch.full_like(a, 448.0)  # a tensor: a division by a number is a product with its reciprocal
    q = (v * (top / a)[:, None, :, None]).to(_E4M3).view(rb * block_rows, kb * 128)
    q = q[:rows, : _pitch(cols)].contiguous()
    return q, (a / top).t().contiguous()


def _values_plain(q, scales, block_rows, cols):
    """What the codes stand for, in 32 bits."""
    rows = q.shape[0]
    s = scales.repeat_interleave(block_rows, dim=1)[:, :rows].t()
    v = q[:, :cols].float()
    return v * s.repeat_interleave(128, dim=1)[:, :cols]


def _stats_plain(v, kind, eps=1e-6):
    """(mean, 1 / deviation) of each row, as columns."""
    if kind == "rms":
        return torch.zeros_like(v[:, :1]), torch.rsqrt((v * v).mean(1, keepdim=True) + eps)
    mean = v.mean(1, keepdim=True)
    d = v - mean
    return mean, torch.rsqrt((d * d).mean(1, keepdim=True) + eps)


def _affine(v, gamma, beta):
    v = v if gamma is None else v * gamma
    return v if beta is None else v + beta


def _gate_rows(s, rows):
    """The gate vector of each row (or one for all), in 32 bits."""
    if s["gate"] is None:
        return None
    return s["gate"].repeat_interleave(s["per_gate"], dim=0)[:rows] if s["per_gate"] else s["gate"]


def _norm_plain(x, y, s, case):
    out = {}
    p = y.float()
    if case["post"] != "none":
        mean, rstd = _stats_plain(p, case["post"])
        p = _affine((p - mean) * rstd, s["post_gamma"], s["post_beta"])
        if case["train"]:
            out["post_stats"] = torch.stack([mean[:, 0], rstd[:, 0]])
    gate = _gate_rows(s, x.shape[0])
    r = s["alpha"] * x.float() + (p if gate is None else gate * p)
    out["residual"] = r.to(x.dtype)
    mean, rstd = _stats_plain(r, case["pre"])
    if case["train"]:
        out["pre_stats"] = torch.stack([mean[:, 0], rstd[:, 0]])
    h = _affine((r - mean) * rstd, s["pre_gamma"], s["pre_beta"])
    if case["fp8"]:
        out["normed"], out["scales"] = _quantise_plain(h, 1)
    else:
        out["normed"] = h.to(y.dtype)
    return out


def _norm_vector_back(grad, unit, rstd, kind):
    """The gradient of a row's normalisation: `unit` the normalised row."""
    g = grad - unit * (grad * unit).mean(1, keepdim=True)
    if kind == "layer":
        g = g - grad.mean(1, keepdim=True)
    return g * rstd


def _norm_backward_plain(s, case):
    out = {}
    M = case["rows"]
    dh = s["grad_normed"].float()
    mean, rstd = s["pre_stats"][0][:, None], s["pre_stats"][1][:, None]
    unit = (s["r"].float() - mean) * rstd
    out["pre_gamma"] = (dh * unit).sum(0)
    if s["pre_beta"] is not None:
        out["pre_beta"] = dh.sum(0)
    dr = s["grad_residual_out"].float() + _norm_vector_back(dh * s["pre_gamma"], unit, rstd, case["pre"])
    del unit, dh
    out["residual"] = (s["alpha"] * dr).to(s["r"].dtype)
    y = s["y"].float()
    if case["post"] != "none":
        mean, rstd = s["post_stats"][0][:, None], s["post_stats"][1][:, None]
        y = (y - mean) * rstd
    p = _affine(y, s["post_gamma"], s["post_beta"])
    gate = _gate_rows(s, M)
    if gate is not None:
        if s["per_gate"]:
            n = s["gate"].shape[0]
            v = torch.zeros(n * s["per_gate"], p.shape[1], device=p.device)
            v[:M] = dr * p
            out["gate"] = v.view(n, s["per_gate"], -1).sum(1)
        else:
            out["gate"] = (dr * p).sum(0, keepdim=True)
        dr = dr * gate
    if s["post_beta"] is not None:
        out["post_beta"] = dr.sum(0)
    if s["post_gamma"] is not None:
        out["post_gamma"] = (dr * y).sum(0)
        dr = dr * s["post_gamma"]
    if case["post"] != "none":
        dr = _norm_vector_back(dr, y, rstd, case["post"])
    out["branch"] = dr.to(s["y"].dtype)
    return out


def _quantise_case(s, case):
    x, b = s["x"], case["block_rows"]
    q, scales = _quantise_plain(x, b)
    out = {"q": q, "scales": scales}
    if case["both"]:
        out["q_t"], out["scales_t"] = _quantise_plain(x.t(), b)
    return out


def _linear_plain(s, case):
    K = case["inner"]
    v = _values_plain(s["a"], s["a_scales"], 1, K) @ _values_plain(s["w"], s["w_scales"], 128, K).t()
    if s["bias"] is not None:
        v += s["bias"]
    return v.to(_T[case["out"]])


def _linear_backward_plain(s, case):
    M, N = case["rows"], case["cols"]
    grad = s["grad"].float()
    q, qs = _quantise_plain(grad, 1)
    dx = _values_plain(q, qs, 1, N) @ _values_plain(s["w_t"], s["w_t_scales"], 128, N).t()
    q, qs = _quantise_plain(grad.t(), 1)
    dw = _values_plain(q, qs, 1, M) @ _values_plain(s["x_t"], s["x_t_scales"], 1, M).t()
    return {"input": dx.to(s["grad"].dtype), "weight": dw, "bias": grad.sum(0)}


# ---------------------------------------------------------------------------
# the library's entry points
# ---------------------------------------------------------------------------
def _workspace(s, need):
    """The workspace a program keeps beside its buffers."""
    if "workspace" not in s:
        s["workspace_bytes"] = need()
        s["workspace"] = (torch.empty(s["workspace_bytes"], dtype=torch.uint8, device="cuda")
                          if s["workspace_bytes"] else None)
    return s["workspace"], s["workspace_bytes"]


def _block_norm(dcn, s, case):
    if "problem" not in s:
        s["problem"] = dcn.make_block_norm(case["rows"], case["channels"], stream_dtype=case["stream"],
                                           branch_dtype=case["branch"], post_norm=case["post"],
                                           pre_norm=case["pre"], rows_per_gate=s["per_gate"],
                                           post_eps=1e-6, pre_eps=1e-6, residual_scale=s["alpha"])
    return s["problem"]


def _run_own(s):
    import deformable_convolution_core_b200 as dcn

    case, out = s["case"], s["out"]
    op = case["op"]
    if op == "norm":
        dcn.dcn_core_block_norm(_block_norm(dcn, s, case), s["x"], s["y"], s["gate"], s["post_gamma"],
                                s["post_beta"], s["pre_gamma"], s["pre_beta"], out["residual"],
                                out["normed"], out.get("scales"), out.get("post_stats"),
                                out.get("pre_stats"))
    elif op == "norm_backward":
        p = _block_norm(dcn, s, case)
        ws, n = _workspace(s, lambda: dcn.dcn_core_block_norm_backward_workspace(p))
        dcn.dcn_core_block_norm_backward(p, s["r"], s["y"], s["gate"], s["post_gamma"], s["post_beta"],
                                         s["pre_gamma"], s["post_stats"], s["pre_stats"],
                                         s["grad_residual_out"], s["grad_normed"], out["residual"],
                                         out["branch"], out.get("gate"), out.get("post_gamma"),
                                         out.get("post_beta"), out.get("pre_gamma"),
                                         out.get("pre_beta"), ws, n)
    elif op == "quantise":
        dcn.dcn_core_quantize_fp8(s["x"], case["rows"], case["cols"], case["dtype"], case["block_rows"],
                                  out["q"], out["scales"], out.get("q_t"), out.get("scales_t"))
    elif op == "linear":
        M, K, N = case["rows"], case["inner"], case["cols"]
        ws, n = _workspace(s, lambda: dcn.dcn_core_linear_fp8_workspace(M, K, N))
        dcn.dcn_core_linear_fp8(s["a"], s["a_scales"], M, K, s["w"], s["w_scales"], N, s["bias"], out,
                                case["out"], ws, n)
    else:
        M, K, N = case["rows"], case["inner"], case["cols"]
        ws, n = _workspace(s, lambda: dcn.dcn_core_linear_fp8_backward_workspace(M, K, N))
        dcn.dcn_core_linear_fp8_backward(s["grad"], case["dtype"], M, K, N, s["w_t"], s["w_t_scales"],
                                         s["x_t"], s["x_t_scales"], out["input"], out["weight"],
                                         out["bias"], ws, n)
    return out


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    op = case["op"]
    if op == "norm":
        return _norm_plain(state["x"], state["y"], state, case)
    if op == "norm_backward":
        return _norm_backward_plain(state, case)
    if op == "quantise":
        return _quantise_case(state, case)
    return _linear_plain(state, case) if op == "linear" else _linear_backward_plain(state, case)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        n = case["rows"] * case["channels"]
        st, bt = _SIZE[case["stream"]], _SIZE[case["branch"]]
        if op == "norm":
            out = n * 1.0 + 4.0 * case["rows"] * _blocks(case["channels"]) if case["fp8"] else n * bt
            return {"bytes": n * (2 * st + bt) + out + (16 * case["rows"] if case["train"] else 0),
                    "flops": 20.0 * n}
        return {"bytes": n * (3 * st + 3 * bt) + 16.0 * case["rows"], "flops": 40.0 * n}
    if op == "quantise":
        M, K = case["rows"], case["cols"]
        b = case["block_rows"]
        out = M * _pitch(K) + 4.0 * _blocks(K) * (_blocks(M) if b > 1 else M)
        if case["both"]:
            out += K * _pitch(M) + 4.0 * _blocks(M) * (_blocks(K) if b > 1 else K)
        return {"bytes": M * K * _SIZE[case["dtype"]] + out, "flops": 4.0 * M * K}
    M, K, N = case["rows"], case["inner"], case["cols"]
    if op == "linear":
        return {"bytes": M * K + 4.0 * M * _blocks(K) + N * K + 4.0 * N + M * N * _SIZE[case["out"]],
                "flops": 2.0 * M * K * N}
    e = _SIZE[case["dtype"]]
    return {"bytes": M * N * e + 2.0 * N * K + M * K * (1 + e) + 4.0 * N * K + 4.0 * N
            + 4.0 * K * _blocks(M),
            "flops": 4.0 * M * K * N}


# ---------------------------------------------------------------------------
# the operators in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_64(v):
    """The nearest e4m3 value, ties to even, of |v| <= 464: three bits after the
    leading one, down to multiples of 2^-9."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(v / step) * step


def _code_blocks_64(x, tall):
    """(codes as 64-bit values, scales (blocks along the row, rows or tall blocks))
    of the definition: the scale and its reciprocal are 32-bit numbers, and so is
    the scaled value that is rounded to a code."""
    M, K = x.shape
    x = torch.nn.functional.pad(x.double(), (0, -K % 128, 0, (-M % 128) if tall else 0))
    t = x.unflatten(1, (-1, 128))
    a = t.abs().max(dim=2).values
    if tall:
        a = a.unflatten(0, (-1, 128)).max(dim=1).values
    a = torch.maximum(a, torch.full_like(a, 7 * 2.0 ** -58))
    inv, scale = (448 / a).float().double(), (a / 448).float().double()
    f = inv.repeat_interleave(128, 0) if tall else inv
    q = _e4m3_64((t * f[:, :, None]).float().double()).flatten(1)
    return q[:M], scale.t().contiguous()


def _pitched_64(q, K):
    return q[:, : -(-K // 16) * 16].contiguous()


def _decoded_64(q, scales, tall, K):
    v = q.double()[:, :K]
    for b in range(scales.shape[0]):
        s = scales[b].double()
        s = s.repeat_interleave(128)[: v.shape[0]] if tall else s
        v[:, 128 * b: 128 * b + 128] *= s[:, None]
    return v


def _moments_64(v, kind):
    mu = v.mean(dim=1) if kind == "layer" else torch.zeros_like(v[:, 0])
    second = ((v - mu[:, None]) ** 2).mean(dim=1)
    return mu, (second + 1e-6) ** -0.5


def _each_row_64(s, M):
    n = s["gate"].shape[0]
    which = torch.arange(M, device="cuda") // (s["per_gate"] or M)
    return which.clamp_(max=n - 1)


def _norm_64(s, case):
    y = s["y"].double()
    M, C = y.shape
    out = {}
    if case["post"] != "none":
        mu, inv = _moments_64(y, case["post"])
        out["post_stats"] = torch.stack([mu, inv])
        y = (y - mu[:, None]) * inv[:, None] * s["post_gamma"].double()
        if s["post_beta"] is not None:
            y = y + s["post_beta"].double()
    if s["gate"] is not None:
        y = y * s["gate"].double()[_each_row_64(s, M)]
    r = s["x"].double() * s["alpha"] + y
    out["residual"] = r
    mu, inv = _moments_64(r, case["pre"])
    out["pre_stats"] = torch.stack([mu, inv])
    h = (r - mu[:, None]) * inv[:, None] * s["pre_gamma"].double()
    if s["pre_beta"] is not None:
        h = h + s["pre_beta"].double()
    out["normed"] = h
    if case["fp8"]:
        q, out["scales"] = _code_blocks_64(h, False)
        out["normed"] = _pitched_64(q, C)
    if not case["train"]:
        out.pop("post_stats", None), out.pop("pre_stats")
    return out


def _norm_backward_64(s, case):
    """By the chain rule on the formula of a norm, n = (v - mean) / deviation:
    dv = (dn - <dn> - n <dn n>) / deviation, without <dn> where no mean is taken."""
    def back(dn, n, inv, kind):
        less = n * (dn * n).mean(dim=1, keepdim=True)
        if kind == "layer":
            less = less + dn.mean(dim=1, keepdim=True)
        return (dn - less) * inv

    out = {}
    M, C = s["y"].shape
    mu, inv = (t[:, None].double() for t in s["pre_stats"])
    n = (s["r"].double() - mu) * inv
    dh = s["grad_normed"].double()
    out["pre_gamma"] = torch.einsum("mc,mc->c", dh, n)
    if s["pre_beta"] is not None:
        out["pre_beta"] = dh.sum(dim=0)
    dr = s["grad_residual_out"].double() + back(dh * s["pre_gamma"].double(), n, inv, case["pre"])
    out["residual"] = dr * s["alpha"]
    n = s["y"].double()
    if case["post"] != "none":
        mu, inv = (t[:, None].double() for t in s["post_stats"])
        n = (n - mu) * inv
    p = n
    if s["post_gamma"] is not None:
        p = p * s["post_gamma"].double()
    if s["post_beta"] is not None:
        p = p + s["post_beta"].double()
    dp = dr
    if s["gate"] is not None:
        which = _each_row_64(s, M)
        out["gate"] = torch.zeros_like(s["gate"], dtype=torch.float64).index_add_(0, which, dr * p)
        dp = dr * s["gate"].double()[which]
    if s["post_beta"] is not None:
        out["post_beta"] = dp.sum(dim=0)
    if s["post_gamma"] is not None:
        out["post_gamma"] = torch.einsum("mc,mc->c", dp, n)
        dp = dp * s["post_gamma"].double()
    out["branch"] = dp if case["post"] == "none" else back(dp, n, inv, case["post"])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    s.pop("out")
    if op == "norm":
        return _norm_64(s, case)
    if op == "norm_backward":
        return _norm_backward_64(s, case)
    if op == "quantise":
        tall, x = case["block_rows"] > 1, s["x"]
        q, scales = _code_blocks_64(x, tall)
        out = {"q": _pitched_64(q, case["cols"]), "scales": scales}
        if case["both"]:
            q, out["scales_t"] = _code_blocks_64(x.t(), tall)
            out["q_t"] = _pitched_64(q, case["rows"])
        return out
    M, K, N = case["rows"], case["inner"], case["cols"]
    if op == "linear":
        v = torch.einsum("mk,nk->mn", _decoded_64(s["a"], s["a_scales"], False, K),
                         _decoded_64(s["w"], s["w_scales"], True, K))
        return v if s["bias"] is None else v + s["bias"].double()
    grad = s["grad"].double()
    q, qs = _code_blocks_64(grad, False)
    dx = torch.einsum("mn,kn->mk", _decoded_64(q, qs, False, N),
                      _decoded_64(s["w_t"], s["w_t_scales"], True, N))
    q, qs = _code_blocks_64(grad.t(), False)
    dw = torch.einsum("nm,km->nk", _decoded_64(q, qs, False, M),
                      _decoded_64(s["x_t"], s["x_t_scales"], False, M))
    return {"input": dx, "weight": dw, "bias": grad.sum(dim=0)}
