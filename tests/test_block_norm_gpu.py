"""Norms around a branch with gate and residual scale: forward and backward
against the float64 oracle, element by element.

Bounds (u = 2^-24).  A row sum takes at most 20 additions in a thread and 8 levels
between threads: 28 u of the mean magnitude, which moves every centred value; the
variance and the reciprocal root add about 14 u + 4 u of the value; the affine part,
the gate and the residual sum add 6 u.  Together less than 64 u of
  S_norm(v, size) = |g| * rstd * (size + <size> + |n| rms(size)) + |b|,
size = |v| for a stored row, and the bound of its input for one that was computed
(an error of the input passes the same formula), which doubles it to 128 u.
Backward: the same formula with d for the gradients; sums over rows run over at most
64 rows in a thread here, 32 slots and 20 + 8 partials: 256 u of the sum of the bounds'
magnitudes covers both the summands' errors (128 u) and the additions."""
import numpy as np
import pytest
import torch

import deformable_convolution_core_b200 as dcn
from oracle import block as ob
from tests.block_testutil import Guarded, TORCH, U, assert_within, dev, host

pytestmark = pytest.mark.gpu


def mean(v):
    return v.mean(axis=1, keepdims=True)


def vec(p, C, dflt):
    return np.full(C, dflt) if p is None else np.abs(np.asarray(p, dtype=np.float64))


def norm_size(v, size, st, g, b):
    """S_norm of the docstring; v the row, st its (mean, rstd)."""
    m, rstd = (np.asarray(s, np.float64)[:, None] for s in st)
    n = np.abs((v - m) * rstd)
    return g * rstd * (size + mean(size) + n * np.sqrt(mean(size ** 2))) + b


class Case:
    def __init__(self, M, C, stream="bf16", branch=None, post="layer", pre="layer", per_gate=0, gate=True,
                 params=True, alpha=1.0, eps=1e-6, has_branch=True, seed=0, offset=0.0, scale=1.0):
        self.M, self.C, self.stream, self.branch = M, C, stream, branch or stream
        self.post, self.pre, self.per_gate, self.alpha, self.eps = post, pre, per_gate, alpha, eps
        rng = np.random.default_rng(seed + M * 31 + C)
        f32 = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
        self.x = dev(scale * f32(M, C) + offset, self.stream)
        self.y = dev(scale * f32(M, C) * np.exp(f32(1, C)) - offset, self.branch) if has_branch else None
        gates = -(-M // per_gate) if per_gate else 1
        self.gate = f32(gates, C) if gate and has_branch else None
        self.gp, self.bp = (f32(C), f32(C)) if post != "none" and params else (None, None)
        self.gq, self.bq = (f32(C), f32(C)) if pre != "none" and params else (None, None)
        self.dr = dev(1e-2 * f32(M, C), self.stream)
        self.dh = dev(1e-2 * f32(M, C), self.branch) if pre != "none" else None
        self.desc = dcn.make_block_norm(M, C, stream, self.branch, post, pre, per_gate, eps, eps, alpha)
        self.kw = dict(post=post, pre=pre, rows_per_gate=per_gate, alpha=alpha)

    def forward(self, fp8=False, in_place=False, stream=None, res=True, stats=True):
        M, C = self.M, self.C
        g = {}
        x = self.x.clone() if in_place else self.x
        if res and not in_place:
            g["r"] = Guarded((M, C), TORCH[self.stream])
        if self.pre != "none":
            g["h"] = Guarded((M, ob.pitch(C)), torch.uint8) if fp8 else Guarded((M, C), TORCH[self.branch])
            if fp8:
                g["scales"] = Guarded((ob.blocks(C), M), torch.float32)
            if stats:
                g["pre_stats"] = Guarded((2, M), torch.float32)
        if self.post != "none" and stats:
            g["post_stats"] = Guarded((2, M), torch.float32)
        t = {k: v.t for k, v in g.items()}
        if in_place:
            t["r"] = x
        p = [dev(v) for v in (self.gate, self.gp, self.bp, self.gq, self.bq)]
        torch.cuda.synchronize()
        dcn.dcn_core_block_norm(self.desc, x, self.y, *p, t.get("r"), t.get("h"), t.get("scales"),
                                t.get("post_stats"), t.get("pre_stats"), stream)
        torch.cuda.synchronize()
        dcn.dcn_core_sync_status()
        assert all(v.untouched() for v in g.values())
        return t

    def sizes(self):
        """(oracle, bound of r / 64 u, bound of h / 128 u)."""
        x, y = host(self.x), host(self.y)
        o = ob.block_norm(x, y, self.gate, self.gp, self.bp, self.gq, self.bq, post_eps=self.eps,
                          pre_eps=self.eps, **self.kw)
        sr = np.abs(self.alpha * x)
        if y is not None:
            sp = np.abs(y)
            if self.post != "none":
                sp = norm_size(y, np.abs(y), o["post_stats"], vec(self.gp, self.C, 1), vec(self.bp, self.C, 0))
            sr = sr + np.abs(ob.gate_rows(self.gate, self.per_gate, self.M, self.C)) * sp
        sh = None
        if self.pre != "none":
            sh = norm_size(o["r"], sr, o["pre_stats"], vec(self.gq, self.C, 1), vec(self.bq, self.C, 0))
        return o, sr, sh

    def check_forward(self, t, fp8=False):
        o, sr, sh = self.sizes()
        if "r" in t:
            assert_within(host(t["r"]), o["r"], 64 * U * sr, self.stream, "residual_out")
        for name, size in (("post_stats", None if self.y is None else np.abs(host(self.y))), ("pre_stats", sr)):
            if name in t:
                got, ref = host(t[name]), o[name]
                assert_within(got[0], ref[0], 64 * U * size.mean(1), "f32", name + " mean")
                # relative error of 1 / deviation: 64 u, and the values' errors over the deviation
                rel = 64 * U * (1 + np.sqrt((size ** 2).mean(1)) * ref[1])
                assert_within(got[1], ref[1], rel * ref[1], "f32", name + " rstd")
        if "h" not in t:
            return
        if not fp8:
            assert_within(host(t["h"]), o["h"], 128 * U * sh, self.branch, "normed")
            return
        # a value stands within half a code step of h: 2^-4 of it or 2^-10 of the scale
        bound = 128 * U * sh
        codes, scales = host(t["h"]), host(t["scales"])
        assert not codes[:, self.C:].any()
        a = np.zeros((self.M, ob.blocks(self.C)))
        e = np.zeros_like(a)
        for k in range(a.shape[1]):
            a[:, k] = np.abs(o["h"][:, k * 128:k * 128 + 128]).max(1)
            e[:, k] = bound[:, k * 128:k * 128 + 128].max(1)
        ref = np.maximum(a, float(ob.FLOOR)) / 448
        assert (np.abs(scales.T - ref) <= e / 448 + 2 * U * ref).all()
        v = ob.values(codes, scales, self.C)
        s = np.repeat(scales.T, 128, axis=1)[:, :self.C]
        half = 2.0 ** -4 * (np.abs(o["h"]) + bound) + 2.0 ** -10 * s
        assert (np.abs(v - o["h"]) <= half * (1 + 2.0 ** -20) + bound).all()

    def backward(self, stream=None, skip=()):
        """Gradients on the oracle's forward, rounded as the forward stores it."""
        o, _, _ = self.sizes()
        M, C = self.M, self.C
        r = dev(o["r"].astype(np.float32), self.stream)
        st = {k: dev(o[k].astype(np.float32)) if k in o else None for k in ("post_stats", "pre_stats")}
        g = {}
        if "residual" not in skip:
            g["residual"] = Guarded((M, C), TORCH[self.stream])
        if self.y is not None:
            g["branch"] = Guarded((M, C), TORCH[self.branch])
        for k, v in (("gate", self.gate), ("post_gamma", self.gp), ("post_beta", self.bp),
                     ("pre_gamma", self.gq), ("pre_beta", self.bq)):
            if v is not None and k not in skip:
                g[k] = Guarded(v.shape, torch.float32)
        t = {k: v.t for k, v in g.items()}
        nbytes = dcn.dcn_core_block_norm_backward_workspace(self.desc)
        ws = Guarded((nbytes,), torch.uint8)
        dr = None if "grad_r" in skip else self.dr
        p = [dev(v) for v in (self.gate, self.gp, self.bp, self.gq)]
        torch.cuda.synchronize()
        dcn.dcn_core_block_norm_backward(
            self.desc, r if self.pre != "none" else None, self.y, *p, st["post_stats"], st["pre_stats"], dr,
            self.dh, t.get("residual"), t.get("branch"), t.get("gate"), t.get("post_gamma"),
            t.get("post_beta"), t.get("pre_gamma"), t.get("pre_beta"), ws.t, nbytes, stream)
        torch.cuda.synchronize()
        dcn.dcn_core_sync_status()
        assert all(v.untouched() for v in g.values()) and ws.untouched()
        self.check_backward(t, host(r), {k: host(v) for k, v in st.items()}, host(dr))
        return t

    def check_backward(self, t, r, st, dr):
        M, C = self.M, self.C
        y, dh = host(self.y), host(self.dh)
        ref = ob.block_norm_backward(r, y, self.gate, self.gp, self.bp, self.gq, st["post_stats"],
                                     st["pre_stats"], dr, dh, **self.kw)
        size = np.zeros((M, C)) if dr is None else np.abs(dr)
        back = lambda d, n, rstd: rstd * (d + mean(d) + n * mean(d * n))  # noqa: E731
        if self.pre != "none":
            m, rstd = (s[:, None] for s in st["pre_stats"])
            n = np.abs((r - m) * rstd)
            size = size + back(np.abs(dh) * vec(self.gq, C, 1), n, rstd)
            sums = dict(pre_gamma=(np.abs(dh) * n).sum(0), pre_beta=np.abs(dh).sum(0))
        else:
            sums = {}
        if "residual" in t:
            assert_within(host(t["residual"]), ref["residual"], 64 * U * abs(self.alpha) * size, self.stream,
                          "grad_residual")
        if y is not None:
            n, rstd = np.abs(y), np.ones((M, 1))
            if self.post != "none":
                m, rstd = (s[:, None] for s in st["post_stats"])
                n = np.abs((y - m) * rstd)
            g = np.abs(ob.gate_rows(self.gate, self.per_gate, M, C))
            p = n * vec(self.gp, C, 1) + vec(self.bp, C, 0)
            if self.gate is not None:
                which = np.arange(M) // self.per_gate if self.per_gate else np.zeros(M, dtype=int)
                sums["gate"] = np.zeros(self.gate.shape)
                np.add.at(sums["gate"], which, size * p)
            d = size * g
            if self.post != "none":
                sums["post_gamma"], sums["post_beta"] = (d * n).sum(0), d.sum(0)
                d = back(d * vec(self.gp, C, 1), n, rstd)
            assert_within(host(t["branch"]), ref["branch"], 128 * U * d, self.branch, "grad_branch")
        for k, s in sums.items():
            if k in t:
                assert_within(host(t[k]), ref[k], 256 * U * s, "f32", "grad_" + k)


SIZES = [(1, 1), (1, 1280), (3, 7), (2, 32), (33, 160), (65, 161), (100, 320), (50, 644), (37, 1280),
         (9, 1283), (5, 2560), (3, 5120), (2, 5119), (300, 40)]
TYPES = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16"), ("f32", "f16")]


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "_".join(t))
@pytest.mark.parametrize("M,C", SIZES)
def test_forward_and_backward_match_the_oracle(M, C, types):
    c = Case(M, C, *types, alpha=0.5)
    c.check_forward(c.forward())
    c.check_forward(c.forward(fp8=True), fp8=True)
    c.backward()


@pytest.mark.parametrize("post", ["none", "layer", "rms"])
@pytest.mark.parametrize("pre", ["none", "layer", "rms"])
@pytest.mark.parametrize("per_gate", [None, 0, 1, 7, 1000])
def test_every_combination_of_norms_and_gates(post, pre, per_gate):
    c = Case(45, 160, post=post, pre=pre, per_gate=per_gate or 0, gate=per_gate is not None)
    c.check_forward(c.forward())
    c.backward()


@pytest.mark.parametrize("M,C,per_gate", [(5000, 160, 144), (5000, 160, 1), (4999, 96, 2500), (2311, 640, 16)])
def test_many_rows_and_gates(M, C, per_gate):
    """More rows than one step of every CTA, gate vectors that end inside CTAs and
    CTAs that end inside gate vectors."""
    c = Case(M, C, per_gate=per_gate, stream="f32")
    c.check_forward(c.forward())
    c.backward()


@pytest.mark.parametrize("pre", ["layer", "rms"])
def test_without_a_branch(pre):
    c = Case(70, 320, post="none", pre=pre, has_branch=False, alpha=1.5)
    c.check_forward(c.forward())
    c.check_forward(c.forward(fp8=True, res=False), fp8=True)
    c.backward()


def test_without_parameters_and_with_some_outputs():
    c = Case(70, 324, params=False, gate=False)
    c.check_forward(c.forward(stats=False))
    c.check_forward(c.forward(res=False, stats=False))
    c.backward()
    c = Case(70, 324, per_gate=9)
    c.backward(skip=("residual", "gate", "post_beta", "pre_gamma"))
    c.backward(skip=("grad_r", "post_gamma", "post_beta", "gate"))
    c.backward(skip=("pre_gamma", "pre_beta"))


def test_in_place_on_the_residual_stream():
    c = Case(333, 160)
    t = c.forward(in_place=True)
    c.check_forward(t)
    assert torch.equal(t["r"], c.forward()["r"])


def test_rows_far_from_zero():
    """A mean a thousand times the deviation: the squares are of centred values."""
    c = Case(20, 640, stream="f32", offset=1000.0, post="layer", pre="layer", eps=0.0)
    c.check_forward(c.forward())


def test_constant_and_zero_rows():
    c = Case(8, 160, stream="f32", gate=False, post="layer", pre="layer", params=False)
    c.x.fill_(2.0)
    c.y.fill_(-3.0)
    t = c.forward()
    assert (t["r"] == 2.0).all() and (t["h"] == 0.0).all()
    c.x.zero_()
    t = c.forward(fp8=True)
    assert (t["h"] == 0).all() and (t["scales"] == 2.0 ** -64).all()


def test_nan_and_infinity_stay_in_their_row():
    c = Case(40, 160, pre="layer", post="rms")
    c.x[3, 5], c.y[7, 9], c.x[39, 159] = float("nan"), float("inf"), float("-inf")
    bad = np.zeros(40, dtype=bool)
    bad[[3, 7, 39]] = True
    t = c.forward()
    assert np.array_equal(np.isnan(host(t["h"])).any(1), bad) and np.isnan(host(t["h"]))[bad].all()
    t = c.forward(fp8=True)
    codes, scales = host(t["h"]), host(t["scales"])
    assert np.array_equal(np.isnan(scales).any(0), bad) and (codes[bad][:, :160] == 127).all()
    assert ((codes[~bad] & 127) != 127).all()


def test_same_bits_every_time():
    c = Case(3000, 320, per_gate=100)
    first = c.backward()
    for _ in range(3):
        again = c.backward()
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_short_workspace_is_refused():
    c = Case(50, 160)
    need = dcn.dcn_core_block_norm_backward_workspace(c.desc)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c.x)
    st = torch.ones(2, 50, device="cuda")
    for w, n in ((None, 0), (ws, need - 4)):
        with pytest.raises(dcn.DcnError) as e:
            dcn.dcn_core_block_norm_backward(c.desc, c.x, c.y, None, None, None, None, st, st, c.dr, c.dh, out,
                                             torch.empty_like(out), workspace=w, workspace_bytes=n)
        assert e.value.status == dcn.DCN_ERR_INVALID_ARG


def test_binding_refuses_other_sizes_and_types():
    c = Case(50, 160)
    out = torch.empty_like(c.x)
    for bad in (torch.empty(49, 160, dtype=torch.bfloat16, device="cuda"), out.float(), out.t()):
        with pytest.raises(ValueError):
            dcn.dcn_core_block_norm(c.desc, c.x, c.y, None, None, None, None, None, bad, out)


def test_more_than_2_31_values():
    M, C = 4_300_000, 512
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.empty(M, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    y = torch.empty(M, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    r, h = torch.empty_like(x), torch.empty_like(x)
    st = torch.empty(2, M, device="cuda")
    desc = dcn.make_block_norm(M, C, "bf16", post_norm="none", pre_norm="layer")
    dcn.dcn_core_block_norm(desc, x, y, None, None, None, None, None, r, h, None, None, st)
    dcn.dcn_core_sync_status()
    dy = torch.empty_like(x)
    nbytes = dcn.dcn_core_block_norm_backward_workspace(desc)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(x)
    dcn.dcn_core_block_norm_backward(desc, r, y, None, None, None, None, None, st, x, y, dx, dy,
                                     workspace=ws, workspace_bytes=nbytes)
    dcn.dcn_core_sync_status()
    for i in (0, 2_097_152, 4_194_304, M - 50):
        s = slice(i, i + 50)
        o = ob.block_norm(host(x[s]), host(y[s]))
        size = np.abs(host(x[s])) + np.abs(host(y[s]))
        assert_within(host(r[s]), o["r"], 64 * U * size, "bf16", "r")
        assert_within(host(h[s]), o["h"],
                      128 * U * norm_size(o["r"], size, o["pre_stats"], 1.0, 0.0), "bf16", "h")
        b = ob.block_norm_backward(host(r[s]), host(y[s]), None, None, None, None, None, host(st[:, s]),
                                   host(x[s]), host(y[s]))
        rstd = host(st[1, s])[:, None]
        n = np.abs((host(r[s]) - host(st[0, s])[:, None]) * rstd)
        d = np.abs(host(y[s]))
        bound = 64 * U * (np.abs(host(x[s])) + rstd * (d + mean(d) + n * mean(d * n)))
        assert_within(host(dx[s]), b["residual"], bound, "bf16", "dx")
        assert_within(host(dy[s]), b["branch"], bound, "bf16", "dy")
