"""GPU tests of the fused products with packed layers (gptq_dequant_linear,
gptq_dequant_gated and their backward calls) against the definitions in
float64.

Tolerances, from the arithmetic (a rounding is off by at most half a step:
2^-8 relative for bf16, 2^-11 for an 11-bit significand, 2^-24 for fp32):
  * exactly representable inputs (activations in {-2..2}, power-of-two scales,
    integer zero points, partial sums below 2^24 units of the finest scale):
    every product and sum is exact, also with operands of 11 bits, so the
    results equal the reference bit for bit;
  * otherwise, with T the sum of the magnitudes that a sum carries,
    T = sum |a| s (q + z) (codes and zero points may be summed apart):
      fp32 sums of K terms in pieces of 16: 2^-24 (max(g, 16) + K/16 + 100) T;
      a BF16 result: both operands rounded to 11 bits, 2 * 2^-11 T' with
      T' = sum |a| |w|, and half a bf16 step of the result;
      an F32 result: operands held in two 11-bit parts each, 4 * 2^-22 T';
      operands of the 11-bit form share a power-of-two range, at the bottom
      of which the step is 2^-25 of a quarter of the largest: K 2^-38 max|a|
      max|w|.
  * an activation passes errors on with its largest slope (below 1.13) and
    adds rounding of a few fp32 steps of its argument, 2^-20 (|z| + 1).
"""
import ctypes
import sys

import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import post_weight_quantization_04_amd as P  # noqa: E402

DEV = "cuda:0"
F64 = torch.float64
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


# ---------------------------------------------------------------------------
# inputs and the reference
# ---------------------------------------------------------------------------
class Layer:
    """A packed layer with its dense float64 weights (original column order)."""

    def __init__(self, rng, d_out, d_in, bits, g, exact=False, order=False, perm=None, spread=1.0):
        maxq = (1 << bits) - 1
        ge = d_in if g == -1 or g >= d_in else g
        groups = -(-d_in // ge)
        codes = rng.integers(0, maxq + 1, size=(d_out, d_in))
        zeros = rng.integers(0, maxq + 1, size=(groups, d_out)).astype(np.float32)
        if exact:
            scales = (2.0 ** -rng.integers(2, 7, size=(groups, d_out))).astype(np.float32)
        else:
            scales = (rng.uniform(0.5, 2.0, size=(groups, d_out)) * 0.02 / maxq).astype(np.float32)
            scales *= np.exp(np.log(spread) * rng.uniform(-1, 1, size=(groups, d_out))).astype(np.float32)
        if perm is None:
            perm = rng.permutation(d_in) if order else np.arange(d_in)
            perm = torch.from_numpy(perm.astype(np.int32)).to(DEV)
        self.q = P.QuantizedLayer(torch.from_numpy(O.pack(codes, bits).view(np.int32)).to(DEV),
                                  torch.from_numpy(scales).to(DEV), torch.from_numpy(zeros).to(DEV), perm, bits, ge,
                                  d_in, order)
        gi = np.arange(d_in) // ge
        s, z = scales[gi].T.astype(np.float64), zeros[gi].T.astype(np.float64)
        self.w = torch.empty(d_out, d_in, dtype=F64, device=DEV)
        self.w[:, perm.long()] = torch.from_numpy(s * (codes - z)).to(DEV)
        self.mag = torch.empty(d_out, d_in, dtype=F64, device=DEV)   # s (q + z)
        self.mag[:, perm.long()] = torch.from_numpy(s * (codes + z)).to(DEV)
        self.g, self.perm = ge, perm


def values(rng, shape, dt, exact=False, size=1.0):
    if exact:
        v = rng.integers(-2, 3, size=shape).astype(np.float32)
    else:
        v = (rng.standard_normal(shape) * size).astype(np.float32)
        if len(shape) == 2:
            v *= np.exp(rng.standard_normal(shape[1])).astype(np.float32)
    return torch.from_numpy(v).to(DEV).to(DT[dt])


def act64(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / 2 ** 0.5)
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(name, z):
    if name == "relu":
        return (z > 0).to(F64)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / 2 ** 0.5) + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5
    if name == "gelu_tanh":
        c = 2 * (2 / np.pi) ** 0.5
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    return torch.ones_like(z)


def mm(a, b):
    return torch.mm(a.to(F64), b.to(F64).contiguous())


def product_error(a, layers, transposed, out):
    """Bound on the error of sum_l a_l W_l^T (a_l W_l if transposed) before its rounding."""
    e = 0
    for x, l in zip(a, layers):
        x = x.abs().to(F64)
        mag, w = (l.mag, l.w.abs()) if transposed else (l.mag.t(), l.w.abs().t())
        k = x.shape[1]
        sums = 2.0 ** -24 * (max(l.g, 16) + k / 16 + 100) * len(layers)
        terms = 2 * 2.0 ** -11 if out == "bf16" else 4 * 2.0 ** -22
        e = e + sums * mm(x, mag) + terms * mm(x, w)
        e = e + k * 2.0 ** -38 * x.amax(1, keepdim=True) * w.max()
    return e


def rounding(ref, out):
    return HALF_STEP[out] * ref.abs() + 1e-37


def check(got, ref, bound, what):
    got = got.to(F64)
    worst = float(((got - ref).abs() / bound).max()) if ref.numel() else 0.0
    say(f"  {what}: max error / bound {worst:.3g}")
    assert torch.isfinite(got).all() and worst <= 1.0, what


def ref_linear(A, layer, bias, act, residual, out):
    z = mm(A, layer.w.t())
    ez = product_error([A], [layer], False, out)
    if bias is not None:
        z = z + bias.to(F64)
    y = act64(act, z)
    ey = 1.13 * ez + 2.0 ** -20 * (z.abs() + 1) * (act != "none") + 2.0 ** -23 * z.abs()
    if residual is not None:
        y = y + residual.to(F64)
    return (y, ey + rounding(y, out) + 2.0 ** -23 * y.abs()), (z, ez + 2.0 ** -23 * z.abs() + rounding(z, out))


def ref_gated(A, gate, up, bg, bu, act, out):
    (y, ey), (g, eg) = ref_linear(A, gate, bg, act, None, "f32" if out == "f32" else "bf16")
    u = mm(A, up.w.t())
    eu = product_error([A], [up], False, out)
    if bu is not None:
        u = u + bu.to(F64)
    eu = eu + 2.0 ** -23 * u.abs()
    # (ey holds a rounding of y to the output's type, which the kernel does not make: a looser bound)
    h = y * u
    return (h, ey * (u.abs() + eu) + y.abs() * eu + rounding(h, out)), (g, eg), (u, eu + rounding(u, out))


def ref_backward(dY, layers, pre, act, out, dt):
    d = dY.to(F64)
    if len(layers) == 1:
        dz = [d * slope64(act, pre[0].to(F64))] if act != "none" else [d]
        ez = [2.0 ** -19 * d.abs() * (act != "none")]   # slope: a few fp32 steps, |z| < 16 in its exponent
    else:
        g, u = pre[0].to(F64), pre[1].to(F64)
        dz = [d * u * slope64(act, g), d * act64(act, g)]
        ez = [2.0 ** -19 * (d * u).abs() * (act != "none") + 2.0 ** -23 * (d * u).abs(),
              2.0 ** -19 * d.abs() * (g.abs() + 1) * (act != "none") + 2.0 ** -23 * (d * g).abs()]
    da = sum(mm(x, l.w) for x, l in zip(dz, layers))
    ea = product_error(dz, layers, True, out) + sum(mm(e, l.w.abs()) for e, l in zip(ez, layers))
    m = dY.shape[0]
    db = [(x.sum(0), e.sum(0) + 2.0 ** -24 * (m + 4) * x.abs().sum(0) + 1e-37) for x, e in zip(dz, ez)]
    return (da, ea + rounding(da, out)), db


# ---------------------------------------------------------------------------
# exactly representable inputs: bit for bit
# ---------------------------------------------------------------------------
# (d_out, d_in, bits, g, m, order)
EXACT = [
    (1, 1, 4, -1, 1, False), (5, 16, 2, 16, 3, True), (64, 128, 4, 128, 1, False), (300, 333, 3, 16, 2, True),
    (77, 33, 3, 16, 9, True), (256, 256, 8, 64, 16, False), (130, 136, 2, 16, 17, True), (96, 512, 4, 128, 40, True),
    (251, 509, 8, -1, 33, False), (640, 96, 8, 32, 63, True), (512, 1024, 4, 64, 64, False),
    (200, 480, 4, 48, 65, True), (300, 992, 3, 32, 129, True), (333, 1000, 2, 16, 300, True),
    (1024, 520, 4, 128, 257, False), (516, 260, 3, 80, 8, False), (1030, 2052, 4, 32, 5, True),
    (260, 300, 4, 16, 512, True), (2050, 130, 2, 32, 700, False),
    # pairs of outputs per lane, whole chunks of four units or not, one and two blocks of rows
    (8200, 512, 4, 128, 3, True), (8210, 256, 2, -1, 70, False), (8202, 192, 3, 64, 20, True),
    (8196, 128, 8, 128, 100, False), (8300, 160, 8, 32, 2, False),
    # wide rows of dZ: held in registers (up to 16384), read twice beyond
    (9000, 48, 4, 16, 20, True), (16400, 40, 3, 16, 33, False), (4104, 72, 2, 32, 130, True),
]


def exact_id(c):
    return f"{c[0]}x{c[1]}-b{c[2]}-g{c[3]}-m{c[4]}"


@pytest.mark.parametrize("in_dt,out_dt", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("case", EXACT, ids=exact_id)
def test_linear_exact(case, in_dt, out_dt):
    d_out, d_in, bits, g, m, order = case
    say(f"linear exact {case} {in_dt}->{out_dt}")
    rng = np.random.default_rng(sum(case[:5]))
    l = Layer(rng, d_out, d_in, bits, g, True, order)
    A = values(rng, (m, d_in), in_dt, True)
    bias, res = values(rng, (d_out,), "bf16", True), values(rng, (m, d_out), out_dt, True)
    Y, Z = P.dequant_linear(A, l.q, bias, "relu", res, out_dtype=DT[out_dt], save_preact=True)
    z = mm(A, l.w.t()) + bias.to(F64)
    assert torch.equal(Z, z.to(DT[out_dt]))
    assert torch.equal(Y, (z.clamp(min=0) + res.to(F64)).to(DT[out_dt]))
    Y = P.dequant_linear(A, l.q, out_dtype=DT[out_dt])
    assert torch.equal(Y, mm(A, l.w.t()).to(DT[out_dt]))


@pytest.mark.parametrize("in_dt,out_dt", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("case", EXACT, ids=exact_id)
def test_gated_exact(case, in_dt, out_dt):
    d_out, d_in, bits, g, m, order = case
    say(f"gated exact {case} {in_dt}->{out_dt}")
    rng = np.random.default_rng(sum(case[:5]) + 1)
    gate = Layer(rng, d_out, d_in, bits, g, True, order)
    up = Layer(rng, d_out, d_in, bits, g, True, order, gate.perm)
    A = values(rng, (m, d_in), in_dt, True)
    bg, bu = values(rng, (d_out,), "f32", True), values(rng, (d_out,), "f32", True)
    H, G, U = P.dequant_gated(A, gate.q, up.q, "relu", bg, bu, out_dtype=DT[out_dt], save_preact=True)
    gr, ur = mm(A, gate.w.t()) + bg.to(F64), mm(A, up.w.t()) + bu.to(F64)
    assert torch.equal(G, gr.to(DT[out_dt])) and torch.equal(U, ur.to(DT[out_dt]))
    # the fp32 product of two exact factors, then the output's rounding
    assert torch.equal(H, (gr.clamp(min=0) * ur).float().to(DT[out_dt]))
    assert torch.equal(P.dequant_gated(A, gate.q, up.q, "none", out_dtype=DT[out_dt]),
                       (mm(A, gate.w.t()) * mm(A, up.w.t())).float().to(DT[out_dt]))


@pytest.mark.parametrize("in_dt,out_dt", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("case", EXACT, ids=exact_id)
def test_backward_exact(case, in_dt, out_dt):
    d_out, d_in, bits, g, m, order = case
    say(f"backward exact {case} {in_dt}->{out_dt}")
    rng = np.random.default_rng(sum(case[:5]) + 2)
    gate = Layer(rng, d_out, d_in, bits, g, True, order)
    up = Layer(rng, d_out, d_in, bits, g, True, order, gate.perm)
    dY, Z, U = (values(rng, (m, d_out), in_dt, True) for _ in range(3))
    d, z, u = dY.to(F64), Z.to(F64), U.to(F64)
    on = (z > 0).to(F64)
    dA, db = P.dequant_linear_backward(dY, gate.q, "relu", Z, True, DT[out_dt])
    assert torch.equal(dA, mm(d * on, gate.w).to(DT[out_dt]))
    assert torch.equal(db, (d * on).sum(0).float())
    dA, db = P.dequant_linear_backward(dY, gate.q, out_dtype=DT[out_dt])
    assert db is None and torch.equal(dA, mm(d, gate.w).to(DT[out_dt]))
    dA, dbg, dbu = P.dequant_gated_backward(dY, gate.q, up.q, Z, U, "relu", True, DT[out_dt])
    dg, du = d * u * on, d * z * on
    assert torch.equal(dA, (mm(dg, gate.w) + mm(du, up.w)).to(DT[out_dt]))
    assert torch.equal(dbg, dg.sum(0).float()) and torch.equal(dbu, du.sum(0).float())


def test_more_rows_than_one_pass():
    """More activation rows than the dense form takes at once (16384): later
    passes use the same weights, and bias gradients add up over them."""
    rng = np.random.default_rng(16)
    m, d_out, d_in = 16384 + 300, 72, 64
    gate = Layer(rng, d_out, d_in, 4, 32, True, True)
    up = Layer(rng, d_out, d_in, 4, 32, True, True, gate.perm)
    A, res = values(rng, (m, d_in), "bf16", True), values(rng, (m, d_out), "bf16", True)
    dY, Z, U = (values(rng, (m, d_out), "bf16", True) for _ in range(3))
    Y = P.dequant_linear(A, gate.q, residual=res)
    assert torch.equal(Y, (mm(A, gate.w.t()) + res.to(F64)).to(torch.bfloat16))
    H, G, _ = P.dequant_gated(A, gate.q, up.q, "relu", save_preact=True)
    assert torch.equal(G, mm(A, gate.w.t()).to(torch.bfloat16))
    assert torch.equal(H, (mm(A, gate.w.t()).clamp(min=0) * mm(A, up.w.t())).float().to(torch.bfloat16))
    d, z, u = dY.to(F64), Z.to(F64), U.to(F64)
    on = (z > 0).to(F64)
    for bias in (True, False):
        dA, dbg, dbu = P.dequant_gated_backward(dY, gate.q, up.q, Z, U, "relu", bias)
        assert torch.equal(dA, (mm(d * u * on, gate.w) + mm(d * z * on, up.w)).to(torch.bfloat16))
        if bias:
            assert torch.equal(dbg, (d * u * on).sum(0).float()) and torch.equal(dbu, (d * z * on).sum(0).float())


# ---------------------------------------------------------------------------
# ordinary values: within the bounds above
# ---------------------------------------------------------------------------
# (d_out, d_in, bits, g, m, order, in, out, act, bias)
ROUNDED = [
    (4096, 4096, 4, 128, 1, False, "bf16", "bf16", "none", False),
    (1407, 1000, 4, 32, 37, True, "bf16", "bf16", "gelu_tanh", True),
    (11008, 4096, 3, 32, 2, True, "bf16", "bf16", "silu", False),
    (251, 509, 8, -1, 509, False, "f32", "f32", "gelu", True),
    (333, 1000, 2, 16, 300, True, "f32", "f32", "relu", True),
    (1024, 2048, 4, 128, 8, True, "f32", "f32", "silu", True),
    (1024, 2048, 4, 128, 200, True, "bf16", "f32", "gelu", True),
    (4096, 11008, 4, 128, 515, True, "bf16", "bf16", "silu", True),
    (2048, 4096, 4, 64, 1024, False, "bf16", "bf16", "gelu", True),
    (700, 300, 4, 64, 64, False, "f32", "bf16", "gelu_tanh", False),
    (260, 8200, 2, -1, 16, True, "bf16", "f32", "none", True),
]


def rounded_id(c):
    return f"{c[0]}x{c[1]}-b{c[2]}-g{c[3]}-m{c[4]}-{c[6]}-{c[7]}-{c[8]}"


@pytest.mark.parametrize("case", ROUNDED, ids=rounded_id)
def test_linear_rounded(case):
    d_out, d_in, bits, g, m, order, in_dt, out_dt, act, has_bias = case
    say(f"linear {case}")
    rng = np.random.default_rng(m + d_out)
    l = Layer(rng, d_out, d_in, bits, g, False, order)
    A = values(rng, (m, d_in), in_dt)
    bias = values(rng, (d_out,), in_dt) if has_bias else None
    res = values(rng, (m, d_out), out_dt)
    (y, ey), (z, ez) = ref_linear(A, l, bias, act, res, out_dt)
    Y, Z = P.dequant_linear(A, l.q, bias, act, res, out_dtype=DT[out_dt], save_preact=True)
    check(Z, z, ez, "Z")
    check(Y, y, ey, "Y")


@pytest.mark.parametrize("case", ROUNDED, ids=rounded_id)
def test_gated_rounded(case):
    d_out, d_in, bits, g, m, order, in_dt, out_dt, act, has_bias = case
    say(f"gated {case}")
    rng = np.random.default_rng(m + d_out + 1)
    gate = Layer(rng, d_out, d_in, bits, g, False, order)
    up = Layer(rng, d_out, d_in, bits, g, False, order, gate.perm)
    A = values(rng, (m, d_in), in_dt)
    bg = values(rng, (d_out,), in_dt) if has_bias else None
    bu = values(rng, (d_out,), in_dt) if has_bias and d_out % 2 else None   # also one bias alone
    (h, eh), (gr, eg), (ur, eu) = ref_gated(A, gate, up, bg, bu, act, out_dt)
    H, G, U = P.dequant_gated(A, gate.q, up.q, act, bg, bu, out_dtype=DT[out_dt], save_preact=True)
    check(G, gr, eg, "G")
    check(U, ur, eu, "U")
    check(H, h, eh, "H")
    assert torch.equal(H, P.dequant_gated(A, gate.q, up.q, act, bg, bu, out_dtype=DT[out_dt]))


@pytest.mark.parametrize("case", ROUNDED, ids=rounded_id)
def test_backward_rounded(case):
    d_out, d_in, bits, g, m, order, in_dt, out_dt, act, has_bias = case
    say(f"backward {case}")
    rng = np.random.default_rng(m + d_out + 2)
    gate = Layer(rng, d_out, d_in, bits, g, False, order)
    up = Layer(rng, d_out, d_in, bits, g, False, order, gate.perm)
    dY = values(rng, (m, d_out), in_dt, size=1e-4)
    Z, U = values(rng, (m, d_out), in_dt), values(rng, (m, d_out), in_dt)
    (da, ea), db = ref_backward(dY, [gate], [Z], act, out_dt, in_dt)
    dA, dbias = P.dequant_linear_backward(dY, gate.q, act, Z, has_bias, DT[out_dt])
    check(dA, da, ea, "dA")
    if has_bias:
        check(dbias, *db[0], "dbias")
    (da, ea), db = ref_backward(dY, [gate, up], [Z, U], act, out_dt, in_dt)
    dA, dbg, dbu = P.dequant_gated_backward(dY, gate.q, up.q, Z, U, act, has_bias, DT[out_dt])
    check(dA, da, ea, "dA gated")
    if has_bias:
        check(dbg, *db[0], "dbias gate")
        check(dbu, *db[1], "dbias up")


@pytest.mark.parametrize("m", [3, 200])
@pytest.mark.parametrize("in_dt", ["bf16", "f32"])
def test_ranges_of_scales_and_rows(m, in_dt):
    """Rows and layers of very different sizes: each row of A (or dY) and each
    row (column) of the layer keeps its own accuracy."""
    rng = np.random.default_rng(m)
    l = Layer(rng, 200, 320, 4, 32, False, True, spread=2.0 ** 8)
    A, dY = values(rng, (m, 320), in_dt), values(rng, (m, 200), in_dt)
    size = torch.from_numpy(10.0 ** rng.uniform(-18, 14, size=(m, 1))).to(DEV).float()
    A, dY = (A * size).to(DT[in_dt]), (dY * size).to(DT[in_dt])
    (y, ey), _ = ref_linear(A, l, None, "none", None, in_dt)
    check(P.dequant_linear(A, l.q), y, ey, "Y")
    (da, ea), _ = ref_backward(dY, [l], [None], "none", in_dt, in_dt)
    check(P.dequant_linear_backward(dY, l.q)[0], da, ea, "dA")


# ---------------------------------------------------------------------------
# values that are not finite, zeros, empty batches
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("m", [4, 20, 140])
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_nonfinite_rows_stay_their_own(m, dt, out):
    rng = np.random.default_rng(m)
    l = Layer(rng, 150, 256, 4, 64, False, False)
    for n, call in ((256, lambda x: P.dequant_linear(x, l.q, out_dtype=DT[out])),
                    (150, lambda x: P.dequant_linear_backward(x, l.q, out_dtype=DT[out])[0])):
        x = values(rng, (m, n), dt)
        x[1, 3], x[2, 5] = float("nan"), float("inf")
        clean = x.clone()
        clean[1], clean[2] = 0, 0
        y, yc = call(x), call(clean)
        keep = [i for i in range(m) if i not in (1, 2)]
        assert torch.equal(y[keep], yc[keep])
        assert torch.isnan(y[1]).all()
        w = l.w[:, 5] if n == 256 else l.w[5]
        assert torch.equal(y[2].to(F64)[w > 0], torch.full_like(w[w > 0], float("inf")))
        assert torch.equal(y[2].to(F64)[w < 0], torch.full_like(w[w < 0], float("-inf")))
        assert torch.isnan(y[2][w == 0]).all()
        assert (yc[1] == 0).all() and (yc[2] == 0).all()


def test_empty_batches():
    rng = np.random.default_rng(1)
    gate = Layer(rng, 40, 64, 4, 32, True, True)
    up = Layer(rng, 40, 64, 4, 32, True, True, gate.perm)
    A, dY = torch.zeros(0, 64, device=DEV), torch.zeros(0, 40, device=DEV)
    assert P.dequant_linear(A, gate.q).shape == (0, 40)
    assert P.dequant_gated(A, gate.q, up.q).shape == (0, 40)
    dA, db = P.dequant_linear_backward(dY, gate.q, bias_grad=True)
    assert dA.shape == (0, 64) and torch.equal(db, torch.zeros(40, device=DEV))
    dA, dbg, dbu = P.dequant_gated_backward(dY, gate.q, up.q, dY, dY, bias_grad=True)
    assert dA.shape == (0, 64) and not dbg.any() and not dbu.any()


def test_activation_limits():
    """Slopes and values far out are 0, 1 or the argument itself, never NaN."""
    rng = np.random.default_rng(2)
    l = Layer(rng, 64, 64, 4, 32, True, False)
    z = torch.tensor([0.0, -0.0, 30.0, -30.0, 1e4, -1e4, 1e30, -1e30], device=DEV).repeat(8)[None].contiguous()
    dY = torch.ones(1, 64, device=DEV)
    for act in P.ACTIVATIONS:
        _, db = P.dequant_linear_backward(dY, l.q, act, z, True)
        ref = slope64(act, z[0].to(F64).clamp(-100, 100))
        assert torch.isfinite(db).all() and (db.to(F64) - ref).abs().max() < 2.0 ** -20, act
        _, dbg, dbu = P.dequant_gated_backward(dY, l.q, l.q, z, torch.ones_like(z), act, True)
        assert (dbg.to(F64) - ref).abs().max() < 2.0 ** -20, act
        va = torch.where(z[0].abs() > 100, z[0].clamp(min=0) if act != "none" else z[0], act64(act, z[0].to(F64)).float())
        assert ((dbu - va).abs() <= 2.0 ** -20 * (va.abs() + 1)).all(), act


# ---------------------------------------------------------------------------
# gradients against differences of the forward call
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("act", list(P.ACTIVATIONS))
@pytest.mark.parametrize("m", [3, 90])
def test_gradients_against_differences(m, act):
    """L = sum C Y in fp32; (L(A + hV) - L(A - hV)) / 2h against <dA, V>.  The
    central difference leaves h^2/6 times a third derivative of order |C| |V W|^3
    (zero for none; for relu, pre-activations within h |V W| of 0 may count
    half), and the fp32 forward errors divided by h."""
    rng = np.random.default_rng(m)
    gate = Layer(rng, 96, 160, 4, 32, False, True)
    up = Layer(rng, 96, 160, 4, 32, False, True, gate.perm)
    A, V = values(rng, (m, 160), "f32"), values(rng, (m, 160), "f32")
    C = values(rng, (m, 96), "f32")
    h = 2.0 ** -6
    ap, am = A + h * V, A - h * V
    step = (ap.to(F64) - am.to(F64)) / (2 * h)

    def forward(x, gated):
        if gated:
            return P.dequant_gated(x, gate.q, up.q, act, save_preact=True)
        return P.dequant_linear(x, gate.q, activation=act, save_preact=True)

    for gated in (False, True):
        lp, lm = (forward(x, gated)[0].to(F64) for x in (ap, am))
        diff = float((C.to(F64) * (lp - lm)).sum() / (2 * h))
        _, *pre = forward(A, gated)
        dA = P.dequant_gated_backward(C, gate.q, up.q, *pre, act)[0] if gated else \
            P.dequant_linear_backward(C, gate.q, act, pre[0])[0]
        got = float((dA.to(F64) * step).sum())
        vg, vu = mm(V, gate.w.t()).abs(), mm(V, up.w.t()).abs()
        z, u = pre[0].to(F64), pre[-1].to(F64)
        c = C.to(F64).abs()
        # |act'''| < 2, |act''| < 1.2, |act'| < 1.13
        if act == "none":
            third = torch.zeros_like(c)
        elif gated:
            third = c * (2 * vg ** 3 * u.abs() + 3 * 1.2 * vg ** 2 * vu)
        else:
            third = c * 2 * vg ** 3
        tol = float((h * h / 6 * 1.5 * third).sum())
        if act == "relu":
            near = (z.abs() <= 1.01 * h * vg) * c * vg * (u.abs() + h * vu if gated else 1)
            tol = float(near.sum())
        _, e = ref_linear(A, gate, None, act, None, "f32")[0]
        scale = (c * (e + 2.0 ** -22 * lp.abs())).sum() * (float(u.abs().max()) + 1 if gated else 1)
        tol += 2 * float(scale) / h + 2.0 ** -20 * float((dA.abs().to(F64) * step.abs()).sum())
        say(f"  {act} gated={gated}: difference {diff:.6g}, gradient {got:.6g}, tolerance {tol:.3g}")
        assert abs(diff - got) <= tol


# ---------------------------------------------------------------------------
# a feed-forward block, as used: forward and backward
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("m", [1, 6, 50, 384])
def test_feed_forward_block(m):
    """y = x + W_down (silu(W_gate x) * (W_up x)), and the gradient of x."""
    rng = np.random.default_rng(m)
    d, ff = 512, 1376
    gate = Layer(rng, ff, d, 4, 128, False, True)
    up = Layer(rng, ff, d, 4, 128, False, True, gate.perm)
    down = Layer(rng, d, ff, 4, 32, False, True)
    x = values(rng, (m, d), "bf16")
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    H, G, U = P.dequant_gated(x, gate.q, up.q, save_preact=True, workspace=ws)
    y = P.dequant_linear(H, down.q, residual=x, workspace=ws)
    (h, eh), (g, _), (u, _) = ref_gated(x, gate, up, None, None, "silu", "bf16")
    check(H, h, eh, "H")
    ref = x.to(F64) + mm(h, down.w.t())
    bound = mm(eh, down.w.abs().t()) + ref_linear(H, down, None, "none", x, "bf16")[0][1]
    check(y, ref, bound, "y")
    dy = values(rng, (m, d), "bf16", size=1e-3)
    dH, _ = P.dequant_linear_backward(dy, down.q, workspace=ws)
    dx, _, _ = P.dequant_gated_backward(dH, gate.q, up.q, G, U, workspace=ws)
    (rh, eh), _ = ref_backward(dy, [down], [None], "none", "bf16", "bf16")
    check(dH, rh, eh, "dH")
    (rx, ex), _ = ref_backward(dH, [gate, up], [G, U], "silu", "bf16", "bf16")
    check(dx, rx, ex, "dx")


# ---------------------------------------------------------------------------
# streams, graphs, alignment, bounds of the outputs, refusals
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("m", [1, 5, 40, 200])
def test_captured_and_replayed(m):
    """Every call captured into one graph and replayed with other inputs, with
    eager calls in between on the same workspace size; all replays equal the
    eager results."""
    rng = np.random.default_rng(m)
    gate = Layer(rng, 384, 512, 4, 128, False, True)
    up = Layer(rng, 384, 512, 4, 128, False, True, gate.perm)
    down = Layer(rng, 512, 384, 4, 128, False, False)
    x, dy = torch.zeros(m, 512, device=DEV, dtype=torch.bfloat16), torch.zeros(m, 512, device=DEV, dtype=torch.bfloat16)

    def run():
        H, G, U = P.dequant_gated(x, gate.q, up.q, save_preact=True)
        y = P.dequant_linear(H, down.q, residual=x)
        dH, db = P.dequant_linear_backward(dy, down.q, bias_grad=True)
        dx, dbg, dbu = P.dequant_gated_backward(dH, gate.q, up.q, G, U, bias_grad=True)
        return [H, y, dH, db, dx, dbg, dbu]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(4):
        x.copy_(values(rng, (m, 512), "bf16"))
        dy.copy_(values(rng, (m, 512), "bf16"))
        eager = [t.clone() for t in run()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), i


@pytest.mark.parametrize("m", [3, 150])
def test_other_stream_and_shared_workspace(m):
    rng = np.random.default_rng(m)
    layers = [Layer(rng, n, k, b, 32, True, False) for n, k, b in ((256, 512, 4), (900, 96, 3), (64, 1024, 8))]
    xs = [values(rng, (m, l.q.d_in), "bf16", True) for l in layers]
    dys = [values(rng, (m, l.w.shape[0]), "bf16", True) for l in layers]
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV)   # any contents will do
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        ys = [P.dequant_linear(x, l.q, workspace=ws, stream=side, out_dtype=torch.float32) for x, l in zip(xs, layers)]
        das = [P.dequant_linear_backward(d, l.q, workspace=ws, stream=side, out_dtype=torch.float32)[0]
               for d, l in zip(dys, layers)]
    side.synchronize()
    for x, d, y, da, l in zip(xs, dys, ys, das, layers):
        assert torch.equal(y, mm(x, l.w.t()).float()) and torch.equal(da, mm(d, l.w).float())


@pytest.mark.parametrize("m", [2, 30, 130])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_element_aligned_operands(m, dt):
    """Operands at addresses aligned to their elements only, outputs inside
    larger buffers whose other elements stay as they were (the C calls)."""
    rng = np.random.default_rng(m)
    d_out, d_in = 144, 192
    l = Layer(rng, d_out, d_in, 4, 32, True, True)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    q = P.QuantizedLayer(shifted(l.q.qpacked), shifted(l.q.scales), shifted(l.q.zeros), shifted(l.perm), 4, l.g, d_in,
                         True)
    A, dY = shifted(values(rng, (m, d_in), dt, True)), shifted(values(rng, (m, d_out), dt, True))
    bias, res = shifted(values(rng, (d_out,), dt, True)), shifted(values(rng, (m, d_out), dt, True))
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    code = P.F32 if dt == "f32" else P.BF16
    st = torch.cuda.current_stream().cuda_stream
    outs = [torch.full((m * n + 130,), 7.0, dtype=DT[dt], device=DEV) for n in (d_out, d_out, d_in)]
    at = [o[65:].data_ptr() for o in outs]
    s = P.lib.gptq_dequant_linear(A.data_ptr(), code, m, d_in, q.qpacked.data_ptr(), q.scales.data_ptr(),
                                  q.zeros.data_ptr(), q.perm.data_ptr(), d_out, 4, l.g, bias.data_ptr(), code, 1,
                                  res.data_ptr(), at[0], code, at[1], ws.data_ptr(), ws.numel(), st)
    assert s == 0, P.lib.gptq_last_error()
    s = P.lib.gptq_dequant_linear_backward(dY.data_ptr(), code, m, d_out, None, 0, q.qpacked.data_ptr(),
                                           q.scales.data_ptr(), q.zeros.data_ptr(), q.perm.data_ptr(), d_in, 4, l.g,
                                           at[2], code, None, ws.data_ptr(), ws.numel(), st)
    assert s == 0, P.lib.gptq_last_error()
    z = mm(A, l.w.t()) + bias.to(F64)
    for o, ref in zip(outs, (z.clamp(min=0) + res.to(F64), z, mm(dY, l.w))):
        assert (o[:65] == 7).all() and (o[65 + ref.numel():] == 7).all()
        assert torch.equal(o[65:65 + ref.numel()].view(ref.shape), ref.to(DT[dt]))


def test_residual_in_place():
    rng = np.random.default_rng(4)
    for m in (3, 200):
        l = Layer(rng, 160, 256, 4, 64, True, False)
        A, res = values(rng, (m, 256), "bf16", True), values(rng, (m, 160), "bf16", True)
        want = P.dequant_linear(A, l.q, residual=res)
        need = max(1, P.dequant_linear_workspace_size(m, 160, 256, 4, 64, P.BF16, P.BF16))
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        s = P.lib.gptq_dequant_linear(A.data_ptr(), P.BF16, m, 256, l.q.qpacked.data_ptr(), l.q.scales.data_ptr(),
                                      l.q.zeros.data_ptr(), None, 160, 4, 64, None, 0, 0, res.data_ptr(),
                                      res.data_ptr(), P.BF16, None, ws.data_ptr(), need,
                                      torch.cuda.current_stream().cuda_stream)
        assert s == 0 and torch.equal(res, want)


def test_refusals():
    rng = np.random.default_rng(5)
    gate = Layer(rng, 64, 128, 4, 32, True, True)
    up = Layer(rng, 64, 128, 4, 32, True, True, gate.perm)
    A, dY = values(rng, (4, 128), "bf16", True), values(rng, (4, 64), "bf16", True)
    with pytest.raises(ValueError, match="activation"):
        P.dequant_linear(A, gate.q, activation="swish")
    with pytest.raises(ValueError, match="columns"):
        P.dequant_linear(A[:, :64].contiguous(), gate.q)
    with pytest.raises(ValueError, match="contiguous"):
        P.dequant_linear(A.t(), gate.q)
    with pytest.raises(ValueError, match="device tensor"):
        P.dequant_linear(A.cpu(), gate.q)
    with pytest.raises(ValueError, match="device tensor"):
        P.dequant_linear(A, gate.q, bias=torch.zeros(64))
    with pytest.raises(TypeError, match="residual"):
        P.dequant_linear(A, gate.q, residual=torch.zeros(4, 64, device=DEV))
    with pytest.raises(ValueError, match="bias"):
        P.dequant_linear(A, gate.q, bias=torch.zeros(63, device=DEV))
    with pytest.raises(TypeError):
        P.dequant_linear(A.half(), gate.q)
    with pytest.raises(TypeError, match="out_dtype"):
        P.dequant_linear(A, gate.q, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="preact"):
        P.dequant_linear_backward(dY, gate.q, "silu")
    with pytest.raises(ValueError, match="gate_pre"):
        P.dequant_gated_backward(dY, gate.q, up.q, None, dY)
    with pytest.raises(TypeError, match="gate_pre"):
        P.dequant_gated_backward(dY, gate.q, up.q, dY.float(), dY)
    other = Layer(rng, 64, 128, 4, 32, True, True)
    with pytest.raises(ValueError, match="share one perm"):
        P.dequant_gated(A, gate.q, other.q)
    plain = Layer(rng, 64, 128, 4, 32, True, False)
    with pytest.raises(ValueError, match="share one perm"):
        P.dequant_gated(A, gate.q, plain.q)
    wide = Layer(rng, 65, 128, 4, 32, True, True, gate.perm)
    with pytest.raises(ValueError, match="same sizes"):
        P.dequant_gated(A, gate.q, wide.q)
    with pytest.raises(TypeError, match="same dtype"):
        P.dequant_gated(A, gate.q, up.q, bias_gate=torch.zeros(64, device=DEV),
                        bias_up=torch.zeros(64, device=DEV, dtype=torch.bfloat16))
    leaf = A.clone().requires_grad_()
    with pytest.raises(ValueError, match="autograd"):
        P.dequant_linear(leaf, gate.q)
    with torch.no_grad():
        P.dequant_linear(leaf, gate.q)
    short = P.QuantizedLayer(gate.q.qpacked[:-1].contiguous(), gate.q.scales, gate.q.zeros, gate.perm, 4, 32, 128, True)
    with pytest.raises(ValueError, match="qpacked"):
        P.dequant_linear(A, short)
