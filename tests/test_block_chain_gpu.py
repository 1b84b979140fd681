"""The block operators together, as a block uses them: core operator -> block norm
to e4m3 -> e4m3 linear layers, forward and backward, captured in a CUDA graph, on
several streams at once, and against the same chain in float64."""
import numpy as np
import pytest
import torch

import deformable_convolution_core_b200 as dcn
from oracle import block as ob
from tests.block_testutil import U, assert_within, dev, host

pytestmark = pytest.mark.gpu

N, H, W, G = 2, 12, 11, 10
C, M, WIDE = G * 16, N * H * W, 640
f32 = np.float32


class Weight:
    """A linear layer's weight laid out once for both products."""

    def __init__(self, rng, rows, cols):
        self.rows, self.cols = rows, cols
        self.w = dev((rng.standard_normal((rows, cols)) / np.sqrt(cols)).astype(f32))
        self.q = torch.empty(rows, ob.pitch(cols), dtype=torch.float8_e4m3fn, device="cuda")
        self.s = torch.empty(ob.blocks(cols), ob.blocks(rows), device="cuda")
        self.qt = torch.empty(cols, ob.pitch(rows), dtype=torch.float8_e4m3fn, device="cuda")
        self.st = torch.empty(ob.blocks(rows), ob.blocks(cols), device="cuda")
        dcn.dcn_core_quantize_fp8(self.w, rows, cols, "f32", 128, self.q, self.s, self.qt, self.st)
        self.bias = dev(0.1 * rng.standard_normal(rows).astype(f32))

    def values(self):
        return ob.values(host(self.q.view(torch.uint8)), host(self.s), self.cols, 128)


class Chain:
    """r = x + gate * LN(core(x)); h = LN(r) in e4m3; u = h W1^T + b1; v = Q(u) W2^T + b2;
    y = r + gate2 * v, and its gradients."""

    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        self.p = dcn.make_problem(N, H, W, G, 16, offset_scale=2.0, dtype="bf16")
        bf = lambda *s: dev(rng.standard_normal(s).astype(f32), "bf16")  # noqa: E731
        self.x, self.off, self.mask = bf(N, H, W, C), bf(N, H, W, G * 18), bf(N, H, W, G * 9)
        self.dy = dev(1e-2 * rng.standard_normal((M, C)).astype(f32), "bf16")
        par = lambda m: dev((m + 0.2 * rng.standard_normal(C)).astype(f32))  # noqa: E731
        self.gp, self.bp, self.gq, self.bq, self.gate, self.gate2 = (par(m) for m in (1, 0, 1, 0, 0.5, 0.5))
        self.w1, self.w2 = Weight(rng, WIDE, C), Weight(rng, C, WIDE)
        e = lambda *s, d=torch.bfloat16: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
        q8, f = torch.float8_e4m3fn, torch.float32
        self.core, self.r, self.y = e(N, H, W, C), e(M, C), e(M, C)
        self.h, self.hs = e(M, ob.pitch(C), d=q8), e(ob.blocks(C), M, d=f)
        self.post, self.pre = e(2, M, d=f), e(2, M, d=f)
        self.u, self.v = e(M, WIDE), e(M, C)
        self.uq, self.us = e(M, ob.pitch(WIDE), d=q8), e(ob.blocks(WIDE), M, d=f)
        self.ut, self.uts = e(WIDE, ob.pitch(M), d=q8), e(ob.blocks(M), WIDE, d=f)
        self.hb = e(M, C)  # the normed rows once more in bf16, for their transpose
        self.ht, self.hts = e(C, ob.pitch(M), d=q8), e(ob.blocks(M), C, d=f)
        self.dv, self.du, self.dh, self.dr, self.dcore = e(M, C), e(M, WIDE), e(M, C), e(M, C), e(M, C)
        self.dw1, self.db1, self.dw2, self.db2 = e(WIDE, C, d=f), e(WIDE, d=f), e(C, WIDE, d=f), e(C, d=f)
        self.grads = [e(C, d=f) for _ in range(6)]
        self.n1 = dcn.make_block_norm(M, C, "bf16", post_norm="layer", pre_norm="layer")
        self.n2 = dcn.make_block_norm(M, C, "bf16", post_norm="none", pre_norm="none")
        need = [dcn.dcn_core_linear_fp8_workspace(M, C, WIDE), dcn.dcn_core_linear_fp8_workspace(M, WIDE, C),
                dcn.dcn_core_linear_fp8_backward_workspace(M, C, WIDE),
                dcn.dcn_core_linear_fp8_backward_workspace(M, WIDE, C),
                dcn.dcn_core_block_norm_backward_workspace(self.n1),
                dcn.dcn_core_block_norm_backward_workspace(self.n2)]
        self.ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")

    def run(self):
        ws, n = self.ws, self.ws.numel()
        dcn.dcn_core_forward(self.p, self.x, self.off, self.mask, self.core)
        x, core = self.x.view(M, C), self.core.view(M, C)
        dcn.dcn_core_block_norm(self.n1, x, core, self.gate, self.gp, self.bp, self.gq, self.bq, self.r,
                                self.h, self.hs, self.post, self.pre)
        dcn.dcn_core_block_norm(self.n1, x, core, self.gate, self.gp, self.bp, self.gq, self.bq, None, self.hb)
        dcn.dcn_core_quantize_fp8(self.hb, M, C, "bf16", 1, None, None, self.ht, self.hts)
        dcn.dcn_core_linear_fp8(self.h, self.hs, M, C, self.w1.q, self.w1.s, WIDE, self.w1.bias, self.u,
                                "bf16", ws, n)
        dcn.dcn_core_quantize_fp8(self.u, M, WIDE, "bf16", 1, self.uq, self.us, self.ut, self.uts)
        dcn.dcn_core_linear_fp8(self.uq, self.us, M, WIDE, self.w2.q, self.w2.s, C, self.w2.bias, self.v,
                                "bf16", ws, n)
        dcn.dcn_core_block_norm(self.n2, self.r, self.v, self.gate2, None, None, None, None, self.y, None)
        # backward
        dcn.dcn_core_block_norm_backward(self.n2, None, self.v, self.gate2, None, None, None, None, None, self.dy,
                                         None, None, self.dv, grad_gate=self.grads[0], workspace=ws,
                                         workspace_bytes=n)
        dcn.dcn_core_linear_fp8_backward(self.dv, "bf16", M, WIDE, C, self.w2.qt, self.w2.st, self.ut, self.uts,
                                         self.du, self.dw2, self.db2, ws, n)
        dcn.dcn_core_linear_fp8_backward(self.du, "bf16", M, C, WIDE, self.w1.qt, self.w1.st, self.ht, self.hts,
                                         self.dh, self.dw1, self.db1, ws, n)
        dcn.dcn_core_block_norm_backward(self.n1, self.r, core, self.gate, self.gp, self.bp, self.gq, self.post,
                                         self.pre, self.dy, self.dh, self.dr, self.dcore, *self.grads[1:], ws, n)

    def outputs(self):
        return [self.r, self.h.view(torch.uint8), self.hs, self.u, self.v, self.y, self.dv, self.du, self.dh, self.dr,
                self.dcore, self.dw1, self.db1, self.dw2, self.db2, *self.grads]


@pytest.fixture(scope="module")
def chain():
    c = Chain(1)
    c.run()
    dcn.dcn_core_sync_status()
    return c


def test_each_step_against_the_oracle_on_its_inputs(chain):
    c = chain
    x, core = host(c.x).reshape(M, C), host(c.core).reshape(M, C)
    o = ob.block_norm(x, core, host(c.gate), host(c.gp), host(c.bp), host(c.gq), host(c.bq), post="layer",
                      pre="layer")
    # ordinary rows: every intermediate is within 20 of its row's scale, 128 u of which is 2e-4
    assert_within(host(c.r), o["r"], 2e-4, "bf16", "r")
    h = ob.values(host(c.h.view(torch.uint8)), host(c.hs), C)
    assert (np.abs(h - o["h"]) <= 2.0 ** -4 * np.abs(o["h"]) + 2.0 ** -10 * np.repeat(host(c.hs).T, 128, 1)[:, :C] + 2e-4).all()
    for a, s, k, w, out in ((c.h, c.hs, C, c.w1, c.u), (c.uq, c.us, WIDE, c.w2, c.v)):
        ref, mag = ob.linear_fp8(host(a.view(torch.uint8)), host(s), host(w.q.view(torch.uint8)), host(w.s), k,
                                 host(w.bias))
        assert_within(host(out), ref, (4 * k + 8) * U * mag, "bf16", "linear")
    y = host(c.r) + host(c.gate2) * host(c.v)
    assert_within(host(c.y), y, 4 * U * (np.abs(host(c.r)) + np.abs(host(c.gate2) * host(c.v))), "bf16", "y")


def test_gradients_follow_a_small_step_of_the_whole_block(chain):
    """The chain's gradient of its branch input against differences of the chain in
    float64 without the quantisations.  They agree up to what e4m3 loses: each of the
    quantised operands of a product (input, weight, gradient) is off by at most 2^-4
    relative a value, independently, so a directional derivative over M * C = 42240
    values stays within 5% of the gradient's size (a wrong factor, sign or transpose is
    off by its whole size)."""
    c = chain
    x, core, r = host(c.x).reshape(M, C), host(c.core).reshape(M, C), None
    w1, w2 = host(c.w1.w), host(c.w2.w)

    def forward(z):
        o = ob.block_norm(x, z, host(c.gate), host(c.gp), host(c.bp), host(c.gq), host(c.bq), post="layer", pre="layer")
        u = o["h"] @ w1.T + host(c.w1.bias)
        return o["r"] + host(c.gate2) * (u @ w2.T + host(c.w2.bias))

    rng = np.random.default_rng(3)
    g = host(c.dcore)
    for d in (rng.standard_normal((M, C)), g / np.abs(g).max()):
        e = 1e-4
        slope = ((forward(core + e * d) - forward(core - e * d)) / (2 * e) * host(c.dy)).sum()
        size = np.linalg.norm(g) * np.linalg.norm(d)
        assert abs(slope - (g * d).sum()) <= 0.05 * size


def test_captured_and_replayed(chain):
    c = chain
    first = [t.clone() for t in c.outputs()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(2):
        for t in c.outputs():
            t.zero_()
        c.ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        dcn.dcn_core_sync_status()
        assert all(torch.equal(a, b) for a, b in zip(first, c.outputs()))


def test_two_chains_at_once_on_two_streams(chain):
    """Workspaces of their own, launches interleaved: the results of each alone."""
    other = Chain(2)
    other.run()
    torch.cuda.synchronize()
    want = [[t.clone() for t in c.outputs()] for c in (chain, other)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for c, s in zip((chain, other), streams):
            with torch.cuda.stream(s):
                c.run()
    torch.cuda.synchronize()
    dcn.dcn_core_sync_status()
    for c, w in zip((chain, other), want):
        assert all(torch.equal(a, b) for a, b in zip(w, c.outputs()))
