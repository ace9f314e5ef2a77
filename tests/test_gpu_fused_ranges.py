"""GPU tests of the fused products with packed layers at the ends of their
range: values near the largest of their type, slopes of far arguments, operands
of very different sizes, rows wider than the LDS, and calls around their edges.

Tolerances as in test_gpu_fused.py unless a test states its own.
"""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_fused import (DEV, DT, F64, Layer, P, check, mm, product_error, ref_backward, ref_gated,  # noqa: E402
                            ref_linear, say, slope64, values)


def scaled(layer, f):
    """The layer with its scales times f, a power of two."""
    for t in (layer.q.scales, layer.w, layer.mag):
        t *= f
    return layer


def large_rows(rng, m, n, dt, lo, hi):
    """Rows of normal values times channel factors, each row times 10^lo .. 10^hi."""
    size = torch.from_numpy(10.0 ** rng.uniform(lo, hi, size=(m, 1))).to(DEV)
    x = (values(rng, (m, n), "f32").to(F64) * size).to(DT[dt])
    assert torch.isfinite(x).all()
    return x


# ---------------------------------------------------------------------------
# large finite values: results that fp32 holds are finite, and as exact as any
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_rows_dense(dt):
    rng = np.random.default_rng(1)
    m, d_out, d_in = 200, 400, 1024
    gate = Layer(rng, d_out, d_in, 4, 32, False, True)
    up = Layer(rng, d_out, d_in, 4, 32, False, True, gate.perm)
    A = large_rows(rng, m, d_in, dt, 29, 34)
    (y, ey), _ = ref_linear(A, gate, None, "none", None, dt)
    check(P.dequant_linear(A, gate.q), y, ey, "Y")
    for layer in (gate, up):   # (so that H stays finite)
        scaled(layer, 2.0 ** -60)
    (h, eh), (g, eg), (u, eu) = ref_gated(A, gate, up, None, None, "silu", dt)
    H, G, U = P.dequant_gated(A, gate.q, up.q, save_preact=True)
    check(G, g, eg, "G")
    check(U, u, eu, "U")
    check(H, h, eh, "H")
    dY = large_rows(rng, m, d_out, dt, 29, 33)
    Z = values(rng, (m, d_out), dt)
    (da, ea), _ = ref_backward(dY, [gate], [Z], "gelu", dt, dt)
    check(P.dequant_linear_backward(dY, gate.q, "gelu", Z)[0], da, ea, "dA")
    (da, ea), _ = ref_backward(dY, [gate, up], [Z, Z], "silu", dt, dt)
    check(P.dequant_gated_backward(dY, gate.q, up.q, Z, Z)[0], da, ea, "dA gated")


FACTORS = [(2.0 ** 110, 2.0 ** -115), (2.0 ** -110, 2.0 ** 115), (2.0 ** -70, 2.0 ** -56)]   # of weights, of rows


def test_factors_out_of_fp32_dense():
    """Rows and weights whose scale factors multiply to less or more than fp32
    holds, with results that it does hold."""
    rng = np.random.default_rng(2)
    for weight, size in FACTORS:
        l = scaled(Layer(rng, 96, 256, 4, 64, False, False), weight)
        A, dY = (values(rng, (150, n), "f32") * size for n in (256, 96))
        for got, ref, x in ((P.dequant_linear(A, l.q), mm(A, l.w.t()), A),
                            (P.dequant_linear_backward(dY, l.q)[0], mm(dY, l.w), dY)):
            bound = product_error([x], [l], x is dY, "f32") + 2.0 ** -24 * ref.abs() + 2.0 ** -149
            check(got, ref, bound, f"{weight} {size}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 16])
def test_large_rows_packed_backward(m, dt):
    rng = np.random.default_rng(m)
    d_out, d_in = 1400, 512
    gate = Layer(rng, d_out, d_in, 4, 32, False, True)
    up = Layer(rng, d_out, d_in, 4, 32, False, True, gate.perm)
    dY, Z = large_rows(rng, m, d_out, dt, 29, 33), values(rng, (m, d_out), dt)
    (da, ea), _ = ref_backward(dY, [gate], [None], "none", dt, dt)
    check(P.dequant_linear_backward(dY, gate.q)[0], da, ea, "dA")
    (da, ea), _ = ref_backward(dY, [gate, up], [Z, Z], "silu", dt, dt)
    check(P.dequant_gated_backward(dY, gate.q, up.q, Z, Z)[0], da, ea, "dA gated")


def test_factors_out_of_fp32_packed_backward():
    rng = np.random.default_rng(2)
    for weight, size in FACTORS:
        l = scaled(Layer(rng, 300, 256, 4, 64, False, False), weight)
        dY = values(rng, (9, 300), "f32") * size
        ref = mm(dY, l.w)
        bound = product_error([dY], [l], True, "f32") + 2.0 ** -24 * ref.abs() + 2.0 ** -149
        check(P.dequant_linear_backward(dY, l.q)[0], ref, bound, f"{weight} {size}")


# chunks of four units, of one, of halves; one group over all columns
@pytest.mark.parametrize("bits,g,d_in", [(4, 128, 1024), (3, 32, 992), (2, 48, 960), (8, -1, 1024), (8, 16, 512)])
@pytest.mark.parametrize("m,dt", [(3, "bf16"), (3, "f32"), (100, "bf16")])
def test_large_rows_packed_forward(m, dt, bits, g, d_in):
    """A group's sum of a (q - z), before its scale, can pass fp32's largest
    value where the scaled sum does not."""
    rng = np.random.default_rng(m)
    d_out = 8200 if bits == 4 else 300   # (two outputs per lane or one)
    gate = Layer(rng, d_out, d_in, bits, g, False, True)
    up = Layer(rng, d_out, d_in, bits, g, False, True, gate.perm)
    A = large_rows(rng, m, d_in, dt, 33, 35.5)
    (y, ey), _ = ref_linear(A, gate, None, "none", None, dt)
    check(P.dequant_linear(A, gate.q), y, ey, "Y")
    for layer in (gate, up):   # (so that H stays finite)
        scaled(layer, 2.0 ** -60)
    (h, eh), (gr, eg), (u, eu) = ref_gated(A, gate, up, None, None, "silu", dt)
    H, G, U = P.dequant_gated(A, gate.q, up.q, save_preact=True)
    check(G, gr, eg, "G")
    check(U, u, eu, "U")
    check(H, h, eh, "H")


@pytest.mark.parametrize("g", [48, 32, 128])
def test_fp32_values_above_bf16(g):
    """Finite fp32 activations beyond the largest bf16 value, few rows."""
    rng = np.random.default_rng(g)
    l = scaled(Layer(rng, 200, 384, 4, g, False, False), 2.0 ** -40)
    A = values(rng, (5, 384), "f32")
    top = torch.finfo(torch.float32).max
    A[0, 7], A[1, 11], A[1, 350], A[2, 0] = top, -top, top * (1 - 2.0 ** -10), 3.3961775e38
    (y, ey), _ = ref_linear(A, l, None, "none", None, "f32")
    check(P.dequant_linear(A, l.q), y, ey, "Y")
    # NaN whose payload lies in the bits that bf16 does not hold
    A.view(torch.int32)[3, 9] = 0x7f800001
    got = P.dequant_linear(A, l.q)
    assert torch.isnan(got[3]).all()
    check(got[:3], y[:3], ey[:3], "the other rows")


# ---------------------------------------------------------------------------
# slopes
# ---------------------------------------------------------------------------
def slope_bound(act, z):
    """Error of a slope, sigmoid(x) + z x' sigmoid(x) sigmoid(-x) or Phi(z) +
    z phi(z), in fp32: the argument of the exponential (of erfc) is off by a few
    times 2^-24 of itself, functions and products by a few steps of the two
    terms, and a factor below the smallest normal number may be taken for 0."""
    if act in ("none", "relu"):
        return torch.zeros_like(z)
    if act == "gelu":
        p, dp, grow = 0.5 * torch.erfc(-z / 2 ** 0.5), torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5, 1.0
        moved = 4 * z.abs() * dp * (1 + z * z)
    else:
        c = 2 * (2 / np.pi) ** 0.5
        x, grow = (z, 1.0) if act == "silu" else (c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z))
        p = torch.sigmoid(x)
        dp = p * torch.sigmoid(-x) * grow
        moved = 4 * x.abs() * (p * torch.sigmoid(-x) + z.abs() * dp)
    return 2.0 ** -23 * (moved + 16 * (p + z.abs() * dp)) + 2.0 ** -126 * (1 + z.abs() * grow)


@pytest.mark.parametrize("m", [1, 20])
@pytest.mark.parametrize("act", list(P.ACTIVATIONS))
def test_slopes(act, m):
    """The slope itself, as the bias gradient of one row of ones."""
    z = torch.cat([torch.arange(-1120, 1121, device=DEV) / 8, torch.tensor([1e4, -1e4, 1e30, -1e30], device=DEV)])
    rng = np.random.default_rng(3)
    l = Layer(rng, len(z), 64, 4, 32, True, False)
    dY, Z = torch.zeros(m, len(z), device=DEV), z.repeat(m, 1)
    dY[m // 2] = 1
    _, db = P.dequant_linear_backward(dY, l.q, act, Z, True)
    near = z.to(F64).clamp(-200, 200)   # (beyond, every slope is 0 or 1 to the last bit)
    err, bound = (db.to(F64) - slope64(act, near)).abs(), slope_bound(act, near)
    worst = (err - bound).argmax()
    say(f"  {act}: worst at z = {float(z[worst])}: {float(db[worst])}, bound {float(bound[worst]):.3g}")
    assert (err <= bound).all()
    ones = torch.ones_like(Z)
    _, dbg, _ = P.dequant_gated_backward(dY, l.q, l.q, Z, ones, act, True)
    assert ((dbg.to(F64) - slope64(act, near)).abs() <= bound).all()


@pytest.mark.parametrize("m", [2, 40])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gate_gradient_of_large_factors(m, dt):
    """dG = dH U act'(G) where dH U passes fp32's largest value and act'(G)
    brings it back, or is 0."""
    rng = np.random.default_rng(m)
    l = Layer(rng, 64, 64, 4, 32, True, False)
    dH, U = torch.full((m, 64), 2.0 ** 70, device=DEV).to(DT[dt]), torch.full((m, 64), 2.0 ** 66, device=DEV).to(DT[dt])
    G = torch.full((m, 64), -40.0, device=DEV).to(DT[dt])
    dA, dbg, dbu = P.dequant_gated_backward(dH, l.q, l.q, G, U, "relu", True)
    assert not dbg.any() and not dbu.any() and not dA.any()
    dA, dbg, dbu = P.dequant_gated_backward(dH, l.q, l.q, G, U, "silu", True)
    p = 1 / (1 + np.exp(40.0))
    dg, du = 2.0 ** 136 * (p - 40 * p * (1 - p)) * m, 2.0 ** 70 * -40 * p * m
    # (the sigmoid's exponent is off by 40 times a few 2^-24; m terms of a sum)
    for got, want in ((dbg, dg), (dbu, du)):
        assert ((got.to(F64) - want).abs() <= abs(want) * (100 + m) * 2.0 ** -23).all()
    assert torch.isfinite(dA).all()


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def test_pair_with_equal_orders_in_two_tensors():
    """Layers read back from storage hold equal orders in tensors of their own."""
    rng = np.random.default_rng(7)
    gate = Layer(rng, 64, 128, 4, 32, True, True)
    up = Layer(rng, 64, 128, 4, 32, True, True, gate.perm)
    again = P.QuantizedLayer(up.q.qpacked, up.q.scales, up.q.zeros, up.q.perm.clone(), 4, 32, 128, True)
    side = torch.cuda.Stream()
    for m in (3, 150):
        A, dH, G, U = (values(rng, (m, n), "bf16", True) for n in (128, 64, 64, 64))
        side.wait_stream(torch.cuda.current_stream())
        for stream in (None, side):
            got = P.dequant_gated(A, gate.q, again, stream=stream)
            grad = P.dequant_gated_backward(dH, gate.q, again, G, U, stream=stream)[0]
            side.synchronize()
            assert torch.equal(got, P.dequant_gated(A, gate.q, up.q))
            assert torch.equal(grad, P.dequant_gated_backward(dH, gate.q, up.q, G, U)[0])
    again.perm[:2] = again.perm[:2].flip(0)
    with pytest.raises(ValueError, match="share one perm"):
        P.dequant_gated(A, gate.q, again)
    again.perm = gate.perm[:-1].contiguous()
    with pytest.raises(ValueError, match="perm"):
        P.dequant_gated(A, gate.q, again)
    again.perm = gate.perm.clone()
    P.dequant_gated(A, gate.q, up.q)   # (warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="share one perm"):   # (the values cannot be looked at here)
            P.dequant_gated(A, gate.q, again)
        held = P.dequant_gated(A, gate.q, up.q)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, P.dequant_gated(A, gate.q, up.q))


def test_forward_mode_tangents_are_refused():
    import torch.autograd.forward_ad as fwAD

    rng = np.random.default_rng(8)
    gate = Layer(rng, 64, 128, 4, 32, True, True)
    up = Layer(rng, 64, 128, 4, 32, True, True, gate.perm)
    A, dY, Z = (values(rng, (4, n), "f32") for n in (128, 64, 64))
    b = values(rng, (64,), "f32")
    with fwAD.dual_level():
        dual = lambda t: fwAD.make_dual(t, torch.ones_like(t))   # noqa: E731
        calls = [lambda: P.dequant_linear(dual(A), gate.q), lambda: P.dequant_linear(A, gate.q, bias=dual(b)),
                 lambda: P.dequant_linear(A, gate.q, residual=dual(Z)),
                 lambda: P.dequant_linear_backward(dual(dY), gate.q),
                 lambda: P.dequant_linear_backward(dY, gate.q, "silu", dual(Z)),
                 lambda: P.dequant_gated(dual(A), gate.q, up.q),
                 lambda: P.dequant_gated(A, gate.q, up.q, bias_up=dual(b)),
                 lambda: P.dequant_gated(A, gate.q, P.QuantizedLayer(up.q.qpacked, dual(up.q.scales), up.q.zeros,
                                                                     up.q.perm, 4, 32, 128, True)),
                 lambda: P.dequant_gated_backward(dY, gate.q, up.q, Z, dual(Z))]
        for i, call in enumerate(calls):
            with pytest.raises(ValueError, match="tangent"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="tangent"):   # (which does not stop tangents)
                call()
        plain = P.dequant_linear(A, gate.q)   # operands without tangents pass
        assert torch.equal(P.dequant_linear(fwAD.unpack_dual(dual(A)).primal, gate.q), plain)
    assert torch.equal(P.dequant_linear(A, gate.q), plain)


# ---------------------------------------------------------------------------
# operands of very different sizes, to what the calls promise
# ---------------------------------------------------------------------------
def held(x, top, out):
    """Largest error of operands x that share the largest value top."""
    step, reach = (2.0 ** -22, 2.0 ** -17) if out == "f32" else (2.0 ** -11, 2.0 ** -28)
    return torch.where(x >= reach * top, step * x, 2.0 ** -39 * top)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m", [3, 16, 200])
def test_outliers_beside_small_values(m, out):
    """One activation (one dZ) 2^8 to 2^26 times the others of its row meets a
    column (row) of zero weights in most outputs: what is left has the
    operands' errors relative to the outlier.  Weights differ by up to 2^16."""
    rng = np.random.default_rng(m)
    d_out, d_in, g = 256, 320, 64
    l = Layer(rng, d_out, d_in, 4, g, False, False, spread=2.0 ** 8)
    l.q.zeros.fill_(0)   # (w = s q)
    codes = rng.integers(0, 16, size=(d_out, d_in))
    codes[:200, 7] = 0
    codes[9, :300] = 0
    l.q.qpacked = torch.from_numpy(O.pack(codes, 4).view(np.int32)).to(DEV)
    s = l.q.scales.to(F64).t()[:, torch.arange(d_in, device=DEV) // g]
    l.w = s * torch.from_numpy(codes).to(DEV)
    l.mag = l.w
    for transposed in (False, True):
        n, at = (d_out, 9) if transposed else (d_in, 7)
        x = values(rng, (m, n), "f32")
        x[:, at] = x.abs().amax(1) * torch.from_numpy(2.0 ** rng.integers(8, 27, size=m)).to(DEV).float()
        x64, w = x.to(F64).abs(), l.w if transposed else l.w.t().contiguous()
        # the weights' shared largest, scales times 15: of a layer's row forward, a group of columns backward
        top = (15 * (s.amax(0) if transposed else s.amax(1)))[None].expand(w.shape)
        ex, ew = held(x64, x64.amax(1, keepdim=True), out), held(w, top, out)
        ref = mm(x, w)
        bound = mm(ex, w) + mm(x64, ew) + mm(ex, ew) + 2.0 ** -22 * mm(x64, w)
        bound = bound + 2.0 ** -24 * (max(g, 16) + x.shape[1] / 16 + 100) * mm(x64, w)
        bound = bound + (2.0 ** -8 if out == "bf16" else 2.0 ** -24) * ref.abs() + 1e-37
        call = P.dequant_linear_backward if transposed else P.dequant_linear
        got = call(x, l.q, out_dtype=DT[out])
        check(got[0] if transposed else got, ref, bound, f"{'dA' if transposed else 'Y'} {out}")


# ---------------------------------------------------------------------------
# activation order over wide layers
# ---------------------------------------------------------------------------
# two rows just above 64 KB of LDS, the 70B down projection, the most that is
# staged, and the first width that is gathered one element at a time
@pytest.mark.parametrize("d_in", [16392, 28672, 32768, 32776])
@pytest.mark.parametrize("m", [129, 150])
def test_wide_layers_in_activation_order(m, d_in):
    """Bit for bit (a row's largest sum: 30 * 2^4 units of its finest scale per
    column, below 2^24 over 32776 columns); captured and replayed as well."""
    say(f"wide {m} x {d_in}")
    rng = np.random.default_rng(d_in)
    l = Layer(rng, 40, d_in, 4, 128, True, True)
    A, dY = values(rng, (m, d_in), "bf16", True), values(rng, (m, 40), "bf16", True)
    for out in ("bf16", "f32"):
        assert torch.equal(P.dequant_linear(A, l.q, out_dtype=DT[out]), mm(A, l.w.t()).to(DT[out]))
        assert torch.equal(P.dequant_linear_backward(dY, l.q, out_dtype=DT[out])[0], mm(dY, l.w).to(DT[out]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = P.dequant_linear(A, l.q)
    for _ in range(3):
        A.copy_(values(rng, (m, d_in), "bf16", True))
        eager = P.dequant_linear(A, l.q)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, eager) and torch.equal(Y, mm(A, l.w.t()).to(torch.bfloat16))
