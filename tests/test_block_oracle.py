"""The float64 oracle of the block operators against independent forms: torch's
own e4m3 type, layer_norm and autograd, closed forms and finite differences (CPU)."""
import numpy as np
import pytest
import torch

from oracle import block as ob

RNG = np.random.default_rng(5)


def test_code_values_are_torchs():
    ours = ob.e4m3_values()
    theirs = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ours, theirs, equal_nan=True)


def test_rounding_is_torchs():
    v = np.concatenate([RNG.uniform(-448, 448, 20000), RNG.uniform(-0.05, 0.05, 20000),
                        ob.e4m3_values()[:127], (ob.e4m3_values()[:126] + ob.e4m3_values()[1:127]) / 2,
                        [0.0, -0.0, 2.0 ** -10, 2.0 ** -11]]).astype(np.float32)
    ours = ob.e4m3_codes(v)
    theirs = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ours, theirs)
    assert ob.e4m3_codes([1e30, -460.0, np.nan]).tolist() == [126, 254, 127]


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 130), (129, 256), (200, 77)])
def test_quantize_stays_within_half_a_step(rows, cols, block_rows):
    x = (RNG.standard_normal((rows, cols)) * np.exp(RNG.uniform(-30, 30, (rows, 1)))).astype(np.float32)
    q, s = ob.quantize(x, block_rows)
    assert q.shape == (rows, ob.pitch(cols)) and s.shape == (ob.blocks(cols), -(-rows // block_rows))
    assert not q[:, cols:].any()
    v = ob.values(q, s, cols, block_rows)
    step = np.repeat(np.repeat(s.astype(np.float64), block_rows, 1)[:, :rows].T, 128, 1)[:, :cols]
    # half a step of the value (2^-4 relative) or of the subnormals (2^-10 of the
    # scale); fl32 of scale, inv and product move the value by at most 2^-22
    assert (np.abs(v - x) <= (2.0 ** -4 + 2.0 ** -21) * np.abs(x) + 2.0 ** -10 * step).all()
    # each block's largest magnitude has the largest code
    assert (q[:, :cols] & 127).max() == 126


def test_quantize_of_zeros_and_non_finite_blocks():
    x = np.zeros((4, 256), dtype=np.float32)
    x[1, 3], x[2, 200], x[3, 0] = np.inf, np.nan, 2.0 ** -130
    q, s = ob.quantize(x)
    assert (s[:, 0] == 2.0 ** -64).all() and not q[0].any()
    assert np.isnan(s[0, 1]) and (q[1, :128] == 127).all() and not q[1, 128:].any()
    assert np.isnan(s[1, 2]) and not q[2, :128].any() and (q[2, 128:] == 127).all()
    assert s[0, 3] == 2.0 ** -64 and not q[3].any()  # far below the floor: zero codes


def test_linear_is_the_product_of_the_values():
    M, K, N = 5, 300, 140
    a, sa = ob.quantize(RNG.standard_normal((M, K)))
    w, sw = ob.quantize(RNG.standard_normal((N, K)), 128)
    b = RNG.standard_normal(N)
    out, mag = ob.linear_fp8(a, sa, w, sw, K, b)
    ref = np.zeros((M, N))
    table = ob.e4m3_values()
    for m in range(M):
        for n in range(N):
            t = table[a[m, :K]] * table[w[n, :K]]
            ref[m, n] = b[n] + sum(float(sa[k, m]) * float(sw[k, n // 128]) * t[k * 128:k * 128 + 128].sum()
                                   for k in range(3))
    assert np.allclose(out, ref, rtol=1e-12, atol=1e-12) and (mag >= np.abs(out) - 1e-12).all()


def torch_forward(x, y, gate, gp, bp, gq, bq, post, pre, per_gate, alpha, eps=1e-6):
    C = x.shape[1]

    def norm(v, kind, g, b):
        if kind == "layer":
            return torch.nn.functional.layer_norm(v, (C,), g, b, eps)
        out = torch.nn.functional.rms_norm(v, (C,), g, eps)
        return out if b is None else out + b

    r = alpha * x
    if y is not None:
        p = y if post == "none" else norm(y, post, gp, bp)
        if gate is not None:
            p = p * (gate.repeat_interleave(per_gate, 0)[:x.shape[0]] if per_gate else gate)
        r = r + p
    return r, None if pre == "none" else norm(r, pre, gq, bq)


@pytest.mark.parametrize("post", ["none", "layer", "rms"])
@pytest.mark.parametrize("pre", ["none", "layer", "rms"])
@pytest.mark.parametrize("per_gate", [None, 0, 1, 3])
def test_block_norm_is_torchs_and_its_gradient_autograds(post, pre, per_gate):
    M, C, alpha = 7, 20, 0.75
    t = lambda *s: torch.tensor(RNG.standard_normal(s), dtype=torch.float64, requires_grad=True)  # noqa: E731
    x, y = t(M, C), t(M, C)
    gate = None if per_gate is None else t(-(-M // per_gate) if per_gate else 1, C)
    gp, bp = (t(C), t(C)) if post != "none" else (None, None)
    gq, bq = (t(C), t(C)) if pre != "none" else (None, None)
    r, h = torch_forward(x, y, gate, gp, bp, gq, bq, post, pre, per_gate, alpha)
    n = lambda v: None if v is None else v.detach().numpy()  # noqa: E731
    kw = dict(post=post, pre=pre, rows_per_gate=per_gate or 0, alpha=alpha)
    o = ob.block_norm(n(x), n(y), n(gate), n(gp), n(bp), n(gq), n(bq), **kw)
    assert np.allclose(o["r"], n(r), rtol=1e-12, atol=1e-12)
    dr = torch.tensor(RNG.standard_normal((M, C)))
    loss = (r * dr).sum()
    dh = None
    if pre != "none":
        assert np.allclose(o["h"], n(h), rtol=1e-11, atol=1e-11)
        dh = torch.tensor(RNG.standard_normal((M, C)))
        loss = loss + (h * dh).sum()
    leaves = dict(residual=x, branch=y, gate=gate, post_gamma=gp, post_beta=bp, pre_gamma=gq, pre_beta=bq)
    leaves = {k: v for k, v in leaves.items() if v is not None}
    grads = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    got = ob.block_norm_backward(o["r"], n(y), n(gate), n(gp), n(bp), n(gq), o.get("post_stats"),
                                 o.get("pre_stats"), n(dr), n(dh), **kw)
    assert set(got) == set(grads)
    for k, g in grads.items():
        assert np.allclose(got[k].reshape(g.shape), g.numpy(), rtol=1e-9, atol=1e-9), k


def test_block_norm_without_a_branch_and_constant_rows():
    x = np.full((2, 6), 3.0)
    o = ob.block_norm(x, None, pre_beta=np.arange(6.0), alpha=2.0)
    assert (o["r"] == 6.0).all() and np.array_equal(o["h"], np.tile(np.arange(6.0), (2, 1)))
    o = ob.block_norm(x, None, pre="rms", pre_eps=0.0)
    assert np.allclose(o["h"], 1.0)


def test_block_norm_gradient_is_the_difference_quotient():
    M, C = 3, 9
    x, y, g = RNG.standard_normal((M, C)), RNG.standard_normal((M, C)), RNG.standard_normal((1, C))
    gp, bp, gq = (RNG.standard_normal(C) for _ in range(3))
    dr, dh = RNG.standard_normal((M, C)), RNG.standard_normal((M, C))

    def loss(y):
        o = ob.block_norm(x, y, g, gp, bp, gq, None, post="layer", pre="rms")
        return (o["r"] * dr).sum() + (o["h"] * dh).sum()

    o = ob.block_norm(x, y, g, gp, bp, gq, None, post="layer", pre="rms")
    got = ob.block_norm_backward(o["r"], y, g, gp, bp, gq, o["post_stats"], o["pre_stats"], dr, dh,
                                 post="layer", pre="rms")["branch"]
    e = 1e-6
    for i in range(M):
        for c in range(C):
            d = np.zeros((M, C))
            d[i, c] = e
            assert abs((loss(y + d) - loss(y - d)) / (2 * e) - got[i, c]) <= 1e-6 * (1 + abs(got[i, c]))
