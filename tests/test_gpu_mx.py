"""GPU tests of the MX formats, the products with MX weights and the norm
against the definitions in float64.

Tolerances, from the arithmetic (a rounding is off by at most half a step:
2^-8 relative for bf16, 2^-24 for fp32, 2^-11 for an 11-bit significand):
  * quantization, dequantization to fp32, and a norm's MX output are rounded
    once from values that are exact or hold 53 bits: equal bit for bit;
  * products of exactly representable operands whose sums stay below 2^24 of
    the finest unit: exact, equal bit for bit;
  * other products, with T = sum |a| |w| over a sum's K terms: fp32 sums
    2^-24 (K + 100) T (each addition at most half a step of a partial sum below
    T); a BF16 result of the dense form: the activations (fp32) or dZ rounded to
    11 bits, 2^-11 T, and half a bf16 step of the result; an F32 result of it:
    operands held to 22 bits, 2^-22 T, one term of products dropped, 2^-22 T;
    at the bottom of a row's shared range K 2^-38 max|a| max|w|;
  * FP8 activations with a BF16 result: the matrix cores keep 14 bits below the
    largest product of a group, 2^-13 T;
  * an activation passes errors on with its largest slope (below 1.13) and adds
    a few fp32 steps of its argument, 2^-20 (|z| + 1);
  * a norm's plain output: half a step (all else in 64 bits); its gradients:
    fp32 with terms r (g w - s f), seven roundings of either and one of the
    sum, 2^-21 (|r g w| + |r s f| + |dS|); dw: 2^-22 sum |g s r| from three
    roundings a term, and additions of up to 64 rows in fp32, 2^-24 * 64 of it.
"""
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import post_weight_quantization_04_amd as P  # noqa: E402

DEV = "cuda:0"
F64 = torch.float64
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SLOPE = 1.13


def say(*a):
    print(*a, file=sys.stderr, flush=True)


# ---------------------------------------------------------------------------
# the formats from their tables
# ---------------------------------------------------------------------------
GRID = {"fp4": [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0],
        "fp8": [(i % 8) * 2.0 ** -9 if i < 8 else (8 + i % 8) * 2.0 ** (i // 8 - 10) for i in range(127)]}
EMAX = {"fp4": 2, "fp8": 8}


def ref_quantize(x, fmt):
    """(code indices with sign [rows][128 steps], scale bytes [rows][blocks]) of float64 x on the CPU."""
    rows, d = x.shape
    x = torch.cat([x.cpu(), torch.zeros(rows, -d % 128, dtype=F64)], 1).view(rows, -1, 32)
    bad = ~torch.isfinite(x).all(2)
    top = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs().amax(2)
    e = torch.frexp(top)[1] - 1 - EMAX[fmt]
    e = torch.where(top > 0, e.clamp(-127, 127), torch.full_like(e, -127))
    v = torch.ldexp(torch.where(bad[:, :, None], torch.zeros_like(x), x), -e[:, :, None].to(F64))
    grid = torch.tensor(GRID[fmt], dtype=F64)
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.bucketize(v.abs(), mid), torch.bucketize(v.abs(), mid, right=True)
    index = torch.where(lo % 2 == 0, lo, hi)
    sign = torch.signbit(v) & ~bad[:, :, None]
    scale = torch.where(bad, torch.full_like(e, 255), e + 127)
    return (index + (8 if fmt == "fp4" else 128) * sign).view(rows, -1), scale


def codes_of(t):
    """The same from an MxTensor."""
    c = t.codes.cpu().to(torch.int64)
    if t.format == "fp4":
        c = torch.stack([c & 15, c >> 4], 2).flatten(1)
    return c, t.scales.cpu().to(torch.int64).transpose(0, 1).flatten(1)


def values_of(t):
    """float64 values [rows][d] of an MxTensor, on its device."""
    c, s = codes_of(t)
    half = 8 if t.format == "fp4" else 128
    grid = torch.tensor(GRID[t.format] + ([float("nan")] if t.format == "fp8" else []), dtype=F64)
    v = grid[c % half] * torch.where(c >= half, -1.0, 1.0)
    unit = torch.where(s == 255, torch.full(s.shape, float("nan"), dtype=F64), torch.ldexp(torch.ones(s.shape, dtype=F64), (s - 127).to(F64)))
    return (v * unit.repeat_interleave(32, 1))[:, :t.d].to(t.codes.device)


def same(a, b):
    return torch.equal(torch.nan_to_num(a.double(), nan=-77.0), torch.nan_to_num(b.double(), nan=-77.0))


def seeded_gen(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return gen


def ints(seed, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=seeded_gen(seed), device=DEV).float()


def gauss(seed, *shape):
    return torch.randn(*shape, generator=seeded_gen(seed), device=DEV)


SHAPES = [(1, 1), (3, 31), (2, 32), (5, 33), (17, 127), (4, 128), (3, 129), (9, 1000), (1, 4096), (257, 520), (1000, 128), (999, 100), (70, 256), (131, 200),
          (2, 20001), (0, 64)]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_quantize(rows, d, dtype, fmt):
    say("quantize", rows, d, dtype, fmt)
    x = (gauss(rows * 7 + d, rows, d) * torch.exp2(ints(d, -20, 20, rows, 1))).to(DT[dtype])
    t = P.mx_quantize(x, fmt)
    assert t.shape == (rows, d)
    if rows == 0:
        assert P.mx_dequantize(t).shape == (0, d)
        return
    codes, scales = codes_of(t)
    want, byte = ref_quantize(x.double(), fmt)
    assert torch.equal(scales, byte.to(torch.int64))
    assert torch.equal(codes, want)
    y = P.mx_dequantize(t)
    assert y.dtype == torch.float32 and torch.equal(y.double(), values_of(t))
    assert torch.equal(P.mx_dequantize(t, torch.bfloat16).double(), values_of(t))


def special_rows():
    inf, nan = float("inf"), float("nan")
    rows = [[0.0] * 32, [-0.0] * 32, [nan] + [1.0] * 31, [1.0] * 31 + [inf], [-inf] * 32, [2.0 ** 127] * 32,
            [3.38e38, -3.38e38] + [1.0] * 30, [2.0 ** -126] * 32, [2.0 ** -133] * 32, [2.0 ** -120, 2.0 ** -126] * 16,
            [7.99] + [2.0 ** -i for i in range(31)], [-6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25] * 4,
            [448.0, 464.0, 479.0, 500.0, 511.0, 432.0, 440.0, 17.0] * 4, [1.0 + 2.0 ** -4, 1.0 + 3 * 2.0 ** -4] * 16,
            [256.0] + [2.0 ** -10, 3 * 2.0 ** -10, 5 * 2.0 ** -10, 2.0 ** -9] * 7 + [0.0] * 3,
            [4.0] + [0.25, -0.25, 0.2500001, 0.2499999, 0.75, -1.25] * 5 + [0.0]]
    return torch.tensor(rows, dtype=torch.float32)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_special_values(dtype, fmt):
    x = special_rows()
    x = torch.cat([x, x.flip(0)], 1).to(DT[dtype])        # other blocks of a row are not touched
    t = P.mx_quantize(x.to(DEV), fmt)
    codes, scales = codes_of(t)
    want, byte = ref_quantize(x.double(), fmt)
    assert torch.equal(scales, byte.to(torch.int64))
    assert torch.equal(codes, want)
    assert same(P.mx_dequantize(t), values_of(t))


def test_quantize_every_bf16_value():
    # every finite bf16 value against blocks whose largest magnitude is a power of two away
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = v[torch.isfinite(v.float())]
    v = v[:v.numel() // 32 * 32].view(-1, 32)
    for fmt in ("fp4", "fp8"):
        t = P.mx_quantize(v.to(DEV), fmt)
        want, byte = ref_quantize(v.double(), fmt)
        codes, scales = codes_of(t)
        assert torch.equal(scales, byte.to(torch.int64)) and torch.equal(codes, want)


def test_misaligned_views():
    base = gauss(3, 12 * 256 + 8)
    for dtype in DT.values():
        b = base.to(dtype)
        x = b[1:1 + 12 * 256].view(12, 256)               # aligned to its element only
        y = x.clone()
        for fmt in ("fp4", "fp8"):
            a, c = P.mx_quantize(x, fmt), P.mx_quantize(y, fmt)
            assert torch.equal(a.codes, c.codes) and torch.equal(a.scales, c.scales)
        w = P.mx_quantize(gauss(4, 40, 256), "fp4")
        for m in (12, 1):
            assert torch.equal(P.mx_linear(x[:m], w), P.mx_linear(y[:m], w))
        g = b[3:259]
        assert torch.equal(P.rms_norm(x, g)[0], P.rms_norm(y, g.clone())[0])
        for p, q in zip(P.rms_norm_backward(y, x, g), P.rms_norm_backward(y.clone(), y, g.clone())):
            assert torch.equal(p, q)
        v = b[5:5 + 12 * 40].view(12, 40)
        assert torch.equal(P.mx_linear(x, w, residual=v), P.mx_linear(y, w, residual=v.clone()))
        assert torch.equal(P.mx_linear_backward(v, w)[0], P.mx_linear_backward(v.clone(), w)[0])
    t = P.mx_quantize(gauss(5, 40, 256), "fp4")
    for bad in (P.MxTensor(t.codes[1:], t.scales, "fp4", 256), P.MxTensor(t.codes, t.scales[:1], "fp4", 256),
                P.MxTensor(t.codes, t.scales, "fp4", 500), P.MxTensor(t.codes.t(), t.scales, "fp4", 256)):
        with pytest.raises(ValueError):
            P.mx_dequantize(bad)
        with pytest.raises(ValueError):
            P.mx_linear(y, bad)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z * 0.5 ** 0.5)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    z = z.clone().requires_grad_()
    with torch.enable_grad():
        return torch.autograd.grad(act64(z, act).sum(), z)[0] if act != "none" else torch.ones_like(z)


def make_acts(kind, x):
    """(the operand of mx_linear, its float64 values)."""
    if kind in DT:
        a = x.to(DT[kind])
        return a, a.double()
    t = P.mx_quantize(x, kind)
    return t, values_of(t)


KINDS = ["bf16", "f32", "fp8", "fp4"]
# rows on both sides of every form's and tile's edge
PRODUCTS = [(1, 1, 1), (1, 16, 128), (2, 17, 33), (7, 100, 129), (16, 64, 4096), (17, 5, 1000), (33, 257, 256),
            (64, 31, 640), (65, 64, 128), (65, 3, 1), (100, 130, 500), (130, 257, 1000), (300, 333, 384),
            (513, 1030, 1100), (70, 4096, 2048)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_products_of_exact_operands(m, n, k, kind):
    say("exact", m, n, k, kind)
    x = ints(m * 31 + k, -2, 3, m, k)
    w = ints(n * 17 + k, -3, 4, n, k) * torch.exp2(ints(n, -2, 3, n, 1))
    x[:, 0] = 2.0
    wq = P.mx_quantize(w, "fp4")
    a, a64 = make_acts(kind, x)
    want = a64 @ values_of(wq).t()
    got = P.mx_linear(a, wq, out_dtype=torch.float32)
    assert torch.equal(got.double(), want)
    assert torch.equal(P.mx_linear(a, wq, out_dtype=torch.bfloat16), want.float().to(torch.bfloat16))


def bounds(kind, out, m, a64, w64, dense):
    T = a64.abs() @ w64.abs().t()
    K = a64.shape[1]
    e = 2.0 ** -24 * (K + 100) * T
    if kind == "fp8" and out == "bf16":
        e = e + 2.0 ** -13 * T
    if dense:
        if kind == "f32" or kind == "dz":
            e = e + (2.0 ** -11 if out == "bf16" else 2.0 ** -21) * T
        e = e + K * 2.0 ** -38 * a64.abs().amax(1, keepdim=True) * w64.abs().amax()
    return e


CASES = [(1, 48, 256, "silu", True, True, True), (5, 100, 1000, "gelu", True, False, True),
         (40, 333, 777, "gelu_tanh", False, True, False), (64, 64, 2048, "none", True, True, False),
         (77, 257, 513, "relu", True, True, True), (300, 1000, 900, "silu", True, True, True),
         (700, 520, 4096, "gelu_tanh", False, False, False), (129, 1407, 1000, "gelu", True, False, False)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k,act,bias,res,save", CASES)
def test_linear(m, n, k, act, bias, res, save, kind, out):
    say("linear", m, n, k, act, kind, out)
    x = gauss(m + n, m, k) * torch.exp(gauss(k, k))
    wq = P.mx_quantize(gauss(n * k, n, k) * 0.05, "fp4")
    a, a64 = make_acts(kind, x)
    w64 = values_of(wq)
    b = gauss(1, n).to(DT[out]) if bias else None
    r = gauss(2, m, n).to(DT[out]) if res else None
    got = P.mx_linear(a, wq, bias=b, activation=act, residual=r, out_dtype=DT[out], save_preact=save)
    y, z = got if save else (got, None)
    assert y.dtype == DT[out]
    z64 = a64 @ w64.t() + (b.double() if bias else 0)
    e = bounds(kind, out, m, a64, w64, m > 32 and (kind in DT or (kind, out) == ("fp8", "f32"))) + 2.0 ** -24 * z64.abs()
    if save:
        assert ((z.double() - z64).abs() <= e + HALF_STEP[out] * (z64.abs() + e)).all()
    y64 = act64(z64, act) + (r.double() if res else 0)
    e = SLOPE * e + (2.0 ** -20 * (z64.abs() + 1) if act != "none" else 0) + 2.0 ** -24 * y64.abs()
    assert ((y.double() - y64).abs() <= e + HALF_STEP[out] * (y64.abs() + e)).all()


@pytest.mark.parametrize("m", [20, 150])
def test_fp8_activations_of_wide_range_in_fp32(m):
    """Elements and blocks that span the format's range: an F32 result adds their products in fp32, not in the
    scaled matrix cores' 14 bits."""
    n, k = 60, 640
    x = gauss(1, m, k) * torch.exp2(ints(3, -17, 1, m, k)) * 448
    t, a64 = make_acts("fp8", x)
    wq = P.mx_quantize(gauss(2, n, k), "fp4")
    w64 = values_of(wq)
    got = P.mx_linear(t, wq, out_dtype=torch.float32)
    want = a64 @ w64.t()
    assert ((got.double() - want).abs() <= bounds("fp8", "f32", m, a64, w64, m > 32)).all()
    assert float((got.double() - want).norm() / want.norm()) < 1e-6


BACK = [(1, 48, 256, "none", False), (7, 333, 1000, "silu", True), (65, 100, 31, "gelu", True),
        (300, 333, 1000, "relu", True), (513, 1100, 520, "gelu_tanh", False), (130, 257, 129, "silu", True),
        (16, 40, 300, "gelu", True), (32, 257, 1000, "silu", True), (33, 333, 1000, "silu", True),
        (48, 1100, 257, "none", True), (64, 64, 2048, "gelu", True), (64, 2500, 4100, "silu", True),
        (50, 2500, 4100, "none", True)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k,act,bias", BACK)
def test_linear_backward(m, n, k, act, bias, dtype, out):
    say("backward", m, n, k, act, dtype, out)
    wq = P.mx_quantize(gauss(n * k, n, k) * 0.05, "fp4")
    w64 = values_of(wq)
    dy, z = gauss(5, m, n).to(DT[dtype]), (gauss(6, m, n) * 1.5).to(DT[dtype])
    da, db = P.mx_linear_backward(dy, wq, activation=act, preact=None if act == "none" else z, bias_grad=bias,
                                  out_dtype=DT[out])
    dz = dy.double() * slope64(z.double(), act)
    want = dz @ w64
    e = bounds("dz", out, m, dz, w64.t(), True) + (2.0 ** -20 * (dy.double().abs() @ w64.abs()) if act != "none" else 0)
    assert da.dtype == DT[out]
    assert ((da.double() - want).abs() <= e + HALF_STEP[out] * (want.abs() + e)).all()
    if bias:
        e = 2.0 ** -24 * (m + 4) * dz.abs().sum(0) + 2.0 ** -20 * dy.double().abs().sum(0)
        assert db.dtype == torch.float32 and ((db.double() - dz.sum(0)).abs() <= e).all()
    else:
        assert db is None


def test_linear_backward_against_differences():
    # the gradient of sum(dY * linear(A)) along directions of A, in exact arithmetic of small integers
    n, k, m = 37, 96, 5
    wq = P.mx_quantize(ints(1, -3, 4, n, k), "fp4")
    a, dy = ints(2, -4, 5, m, k), ints(3, -2, 3, m, n)
    da, _ = P.mx_linear_backward(dy, wq)
    for i in range(4):
        v = ints(10 + i, -2, 3, m, k)
        up, down = P.mx_linear(a + v, wq), P.mx_linear(a - v, wq)
        assert float(((up - down).double() / 2 * dy.double()).sum()) == float((da.double() * v.double()).sum())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m", [9, 150])
def test_values_that_are_not_finite(m, kind):
    n, k = 70, 260
    x = gauss(7, m, k)
    w = gauss(8, n, k)
    w[5, 200] = float("nan")
    wq = P.mx_quantize(w, "fp4")
    bad = [2, 4]
    x[2, 100], x[4, 3] = float("inf"), float("nan")
    a, _ = make_acts(kind, x)
    y = P.mx_linear(a, wq, out_dtype=torch.float32)
    fine = torch.ones(m, n, dtype=torch.bool, device=DEV)
    fine[:, 5] = False
    for i in bad:
        fine[i] = False
    assert torch.equal(torch.isfinite(y), fine)
    assert torch.isnan(y[:, 5]).all()
    if kind in DT:   # an infinity times a weight that is not zero is one, times zero NaN
        w64 = values_of(wq)
        col = w64[:, 100]
        got = y[2]
        assert torch.equal(torch.isnan(got), (col == 0) | torch.isnan(w64).any(1))
        assert torch.equal(torch.sign(got[col != 0])[~torch.isnan(got[col != 0])],
                           torch.sign(col[col != 0]).float()[~torch.isnan(got[col != 0])])
    dy = gauss(9, m, n)
    dy[3, 1] = float("nan")
    ok = P.mx_quantize(torch.nan_to_num(w), "fp4")
    da, db = P.mx_linear_backward(dy, ok, bias_grad=True)
    assert torch.isnan(da[3]).all() and torch.isfinite(da[:3]).all() and torch.isfinite(da[4:]).all()
    assert torch.equal(torch.isfinite(db), torch.arange(n, device=DEV) != 1)


@pytest.mark.parametrize("kind", KINDS)
def test_scales_of_any_size(kind):
    # rows of weights and activations at both ends of the exponents' range, products that fp32 holds
    m, n, k = 80, 40, 256
    x, w = ints(1, -2, 3, m, k), ints(2, -3, 4, n, k)
    x[:, 0], w[:, 0] = 2.0, 3.0
    se = ints(3, -60, 60, m, 1)
    we = ints(4, -50, 40, n, 1)
    wq = P.mx_quantize(w * torch.exp2(we), "fp4")
    for rows in (80, 12):
        a, a64 = make_acts(kind, (x * torch.exp2(se))[:rows].contiguous())
        want = a64 @ values_of(wq).t()
        got = P.mx_linear(a, wq, out_dtype=torch.float32)
        assert torch.equal(got.double(), want.float().double())


@pytest.mark.parametrize("kind", KINDS)
def test_many_rows(kind):
    """More rows than one pass of the dense form takes (16384)."""
    m, n, k = 16384 + 131, 72, 160
    wq = P.mx_quantize(ints(1, -3, 4, n, k), "fp4")
    x = ints(2, -2, 3, m, k)
    x[:, 0] = 2.0
    a, a64 = make_acts(kind, x)
    assert torch.equal(P.mx_linear(a, wq, out_dtype=torch.float32).double(), a64 @ values_of(wq).t())
    if kind in DT:
        dy = ints(3, -2, 3, m, n).to(DT[kind])
        da, db = P.mx_linear_backward(dy, wq, bias_grad=True, out_dtype=torch.float32)
        assert torch.equal(da.double(), dy.double() @ values_of(wq))
        assert torch.equal(db.double(), dy.double().sum(0))


def test_rows_of_an_mx_matrix():
    w = P.mx_quantize(gauss(1, 48, 200), "fp4")
    t = P.mx_quantize(gauss(2, 40, 200), "fp8")
    part = P.MxTensor(t.codes[3:20], t.scales[:, 3:20].contiguous(), "fp8", 200)
    assert torch.equal(P.mx_dequantize(part), P.mx_dequantize(t)[3:20])
    assert torch.equal(P.mx_linear(part, w), P.mx_linear(t, w)[3:20])
    assert torch.equal(P.mx_linear(t, P.MxTensor(w.codes[16:], w.scales[:, 16:].contiguous(), "fp4", 200)),
                       P.mx_linear(t, w)[:, 16:])


def test_outputs_over_inputs():
    """What the C interface allows: Y over the residual, S over X or the residual, dX over dS."""
    m, k, n = 90, 264, 72
    st = torch.cuda.current_stream().cuda_stream
    L = P.lib
    for rows in (90, 7):
        x, w = gauss(1, rows, k).bfloat16(), P.mx_quantize(gauss(2, n, k), "fp4")
        for a in (x, P.mx_quantize(x, "fp8")):
            r = gauss(3, rows, n).bfloat16()
            want = P.mx_linear(a, w, activation="silu", residual=r)
            kind = "fp8" if isinstance(a, P.MxTensor) else P.BF16
            need = P.mx_linear_workspace_size(rows, n, k, kind, P.BF16)
            ws = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
            rest = (rows, k, w.codes.data_ptr(), w.scales.data_ptr(), n, None, 0, 4, r.data_ptr(), r.data_ptr(), P.BF16,
                    None, ws.data_ptr(), ws.numel(), st)
            if kind == "fp8":
                assert L.gptq_mx_linear_mx(a.codes.data_ptr(), a.scales.data_ptr(), 0, *rest) == 0
            else:
                assert L.gptq_mx_linear(a.data_ptr(), kind, *rest) == 0
            assert torch.equal(r, want)
    for m, d in ((3, 100), (300, 4096), (2, 40000)):
        x, r, g = gauss(4, m, d).bfloat16(), gauss(5, m, d).bfloat16(), gauss(6, d).bfloat16()
        y, s = P.rms_norm(x, g, residual=r)
        for over in (0, 1):
            a, b, out = x.clone(), r.clone(), torch.empty_like(x)
            S = (a, b)[over]
            assert L.gptq_rms_norm(a.data_ptr(), b.data_ptr(), g.data_ptr(), P.BF16, m, d, 1e-6, S.data_ptr(),
                                   out.data_ptr(), st) == 0
            assert torch.equal(S, s) and torch.equal(out, y)
        dx, dw = P.rms_norm_backward(y, s, g, dS=r)
        b = r.clone()
        ws = torch.empty(P.rms_norm_backward_workspace_size(m, d) + 256, dtype=torch.uint8, device=DEV)
        dw2 = torch.empty_like(dw)
        assert L.gptq_rms_norm_backward(y.data_ptr(), s.data_ptr(), g.data_ptr(), b.data_ptr(), P.BF16, m, d, 1e-6,
                                        b.data_ptr(), dw2.data_ptr(), ws.data_ptr(), ws.numel(), st) == 0
        assert torch.equal(b, dx) and torch.equal(dw, dw2)


def test_no_rows_and_bias_gradients():
    wq = P.mx_quantize(gauss(1, 50, 64), "fp4")
    for kind in KINDS:
        a, _ = make_acts(kind, torch.zeros(0, 64, device=DEV))
        assert P.mx_linear(a, wq).shape == (0, 50)
    da, db = P.mx_linear_backward(torch.zeros(0, 50, device=DEV), wq, bias_grad=True)
    assert da.shape == (0, 64) and torch.equal(db, torch.zeros(50, device=DEV))
    y, s = P.rms_norm(torch.zeros(0, 64, device=DEV), torch.ones(64, device=DEV), format="fp8")
    assert y.shape == (0, 64) and s.shape == (0, 64)
    dx, dw = P.rms_norm_backward(s, s, torch.ones(64, device=DEV))
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros(64, device=DEV))


# ---------------------------------------------------------------------------
# the norm
# ---------------------------------------------------------------------------
NORMS = [(1, 1), (1, 4096), (3, 7), (5, 64), (300, 96), (257, 513), (256, 1024), (300, 2048), (2, 2056), (259, 4096),
         (260, 8192), (3, 8200), (2, 16384), (5, 33000), (2, 70000), (1000, 130), (1000, 128), (999, 100), (257, 1)]


@pytest.mark.parametrize("fmt", [None, "fp8", "fp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,d", NORMS)
def test_norm(m, d, dtype, fmt):
    say("norm", m, d, dtype, fmt)
    x = (gauss(d, m, d) * torch.exp(gauss(1, d))).to(DT[dtype])
    r = (gauss(d + 1, m, d) * 3).to(DT[dtype])
    w = (1 + 0.2 * gauss(2, d)).to(DT[dtype])
    for res in (None, r):
        y, s = P.rms_norm(x, w, residual=res, eps=1e-5, format=fmt)
        want_s = x if res is None else (x.double() + res.double()).to(DT[dtype])
        assert torch.equal(s, want_s)
        v = s.double()
        y64 = v * w.double() / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5)
        if fmt is None:
            e = HALF_STEP[dtype] * y64.abs() + 2.0 ** -48 * y64.abs()
            assert y.dtype == DT[dtype] and ((y.double() - y64).abs() <= e).all()
        else:
            codes, scales = codes_of(y)
            want, byte = ref_quantize(y64, fmt)
            assert torch.equal(scales, byte.to(torch.int64)) and torch.equal(codes, want)


def test_norm_of_very_many_rows():
    m, d = (1 << 20) + 3, 2056                            # more rows than one launch takes
    x = torch.empty(m, d, dtype=torch.bfloat16, device=DEV)
    for i in range(0, m, 1 << 18):
        x[i:i + (1 << 18)].normal_(generator=seeded_gen(i))
    w = (1 + 0.2 * gauss(2, d)).bfloat16()
    y, _ = P.rms_norm(x, w, format="fp8")
    rows = torch.tensor([0, 1, 1000, (1 << 20) - 1, 1 << 20, m - 1], device=DEV)
    v = x[rows].double()
    want, byte = ref_quantize(v * w.double() / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6), "fp8")
    part = P.MxTensor(y.codes[rows].contiguous(), y.scales[:, rows].contiguous(), "fp8", d)
    codes, scales = codes_of(part)
    assert torch.equal(scales, byte.to(torch.int64)) and torch.equal(codes, want)


def test_norm_of_unusual_rows():
    d = 200
    x = torch.zeros(8, d, device=DEV)
    x[1], x[2, 3], x[3, 4] = 3e38, float("inf"), float("nan")
    x[4] = 1e-30
    x[5, 7] = -2.0
    x[6] = 1e25
    w = 1 + 0.1 * gauss(1, d)
    for dtype in DT.values():
        y, s = P.rms_norm(x.to(dtype), w.to(dtype), eps=1e-6)
        v = s.double()
        y64 = v * w.to(dtype).double() / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
        fine = torch.isfinite(y64)
        assert torch.equal(torch.isfinite(y), fine)
        assert ((y.double() - y64)[fine].abs() <= 2.0 ** -7 * y64[fine].abs()).all()
        q, _ = P.rms_norm(x.to(dtype), w.to(dtype), eps=1e-6, format="fp8")
        bad = torch.isnan(P.mx_dequantize(q))
        assert torch.equal(bad.any(1), ~fine.all(1)) and int(bad.sum()) == 32 + d   # one block; a whole row
        dx, dw = P.rms_norm_backward(torch.ones_like(s), s, w.to(dtype), eps=1e-6)
        assert torch.isfinite(dx[[0, 1, 4, 5, 6, 7]]).all()
    y, _ = P.rms_norm(torch.zeros(2, 64, device=DEV), torch.ones(64, device=DEV), eps=0.0)
    assert torch.isnan(y).all()                           # 0 / 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,d", NORMS + [(3000, 64), (1500, 4096), (37, 1407), (16, 4096), (17, 4096), (16, 4104), (9, 1000), (9, 1001)])
def test_norm_backward(m, d, dtype):
    say("norm backward", m, d, dtype)
    s = (gauss(d, m, d) * torch.exp(gauss(1, d))).to(DT[dtype])
    w = (1 + 0.2 * gauss(2, d)).to(DT[dtype])
    dy, ds = gauss(3, m, d).to(DT[dtype]), gauss(4, m, d).to(DT[dtype])
    v, g = s.double(), dy.double()
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
    f = r * r * (g * w.double() * v).mean(1, keepdim=True)
    for extra in (None, ds):
        dx, dw = P.rms_norm_backward(dy, s, w, dS=extra)
        t = 0 if extra is None else extra.double()
        want = r * (g * w.double() - v * f) + t
        e = 2.0 ** -21 * ((r * g * w.double()).abs() + (r * v * f).abs() + (0 if extra is None else t.abs()))
        assert dx.dtype == DT[dtype]
        assert ((dx.double() - want).abs() <= e + HALF_STEP[dtype] * (want.abs() + e)).all()
        terms = (g * v * r)
        assert dw.dtype == torch.float32
        assert ((dw.double() - terms.sum(0)).abs() <= (2.0 ** -22 + 2.0 ** -18) * terms.abs().sum(0)).all()
    dx2, none = P.rms_norm_backward(dy, s, w, dS=ds, weight_grad=False)
    assert none is None and torch.equal(dx2, dx)


def test_norm_backward_against_differences():
    m, d = 3, 40
    s, w, dy = gauss(1, m, d), 1 + 0.2 * gauss(2, d), gauss(3, m, d)
    dx, dw = P.rms_norm_backward(dy, s, w, eps=1e-5)

    def f(s, w):
        v = s.double()
        return (v * w.double() / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5) * dy.double()).sum()

    for i in range(4):
        ds, dv, h = gauss(10 + i, m, d).double(), gauss(20 + i, d).double(), 1e-4
        along = (f(s.double() + h * ds, w) - f(s.double() - h * ds, w)) / (2 * h)
        assert abs(float(along - (dx.double() * ds).sum())) <= 1e-4 * float((dx.double() * ds).abs().sum())
        along = (f(s, w.double() + h * dv) - f(s, w.double() - h * dv)) / (2 * h)
        assert abs(float(along - (dw.double() * dv).sum())) <= 1e-4 * float((dw.double() * dv).abs().sum())


# ---------------------------------------------------------------------------
# together, and how calls run
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("m", [1, 200])
def test_a_block_forward_and_backward(m, fmt):
    """norm -> up projection -> down projection back onto the stream, and the gradients, as a model runs them."""
    d, ff = 512, 1100
    x, r = gauss(1, m, d).bfloat16(), gauss(2, m, d).bfloat16()
    w = (1 + 0.1 * gauss(3, d)).bfloat16()
    up, down = P.mx_quantize(gauss(4, ff, d) * 0.05, "fp4"), P.mx_quantize(gauss(5, d, ff) * 0.05, "fp4")
    h, s = P.rms_norm(x, w, residual=r, format=fmt)
    a, z = P.mx_linear(h, up, activation="silu", save_preact=True)
    y = P.mx_linear(a, down, residual=s)
    h64, s64, up64, down64 = values_of(h), s.double(), values_of(up), values_of(down)
    z64 = h64 @ up64.t()
    y64 = act64(z64, "silu").to(torch.bfloat16).double() @ down64.t() + s64
    # the stored activations carry half a bf16 step, which the second product passes on
    e = 2.0 ** -7 * ((act64(z64, "silu").abs() + 2.0 ** -8) @ down64.abs().t()) + 2.0 ** -7 * y64.abs()
    assert ((y.double() - y64).abs() <= e).all()
    dy = gauss(6, m, d).bfloat16()
    da, _ = P.mx_linear_backward(dy, down)
    dh, _ = P.mx_linear_backward(da, up, activation="silu", preact=z)
    dx, dw = P.rms_norm_backward(dh, s, w, dS=dy)
    v = s64.clone().requires_grad_()
    w64 = w.double().requires_grad_()
    n = v * w64 / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
    loss = ((act64(n @ up64.t(), "silu") @ down64.t() + v) * dy.double()).sum()
    gx, gw = torch.autograd.grad(loss, (v, w64))
    # h and the saved z are quantized and rounded where the reference is not: compared in norm, by the
    # steps' relative sizes (2^-4 of e4m3, 2^-2 of e2m1, in the argument of the slope)
    tol = {"fp8": 2.0 ** -4, "fp4": 2.0 ** -2}[fmt]
    assert float((dx.double() - gx).norm() / gx.norm()) < tol
    assert float((dw.double() - gw).norm() / gw.norm()) < tol


def all_calls(x, r, w, wq, dy, ws=None):
    """Every operator once, with outputs that only depend on the inputs' present values."""
    m = x.shape[0]
    out = []
    for fmt in ("fp8", "fp4"):
        h, s = P.rms_norm(x, w, residual=r, format=fmt)
        out += [h.codes, h.scales, s, P.mx_linear(h, wq, activation="gelu", workspace=ws)]
        q = P.mx_quantize(x, fmt)
        out += [P.mx_dequantize(q, torch.bfloat16)]
    out += [P.mx_linear(x, wq, activation="silu", workspace=ws), P.mx_linear(x.float(), wq, workspace=ws)]
    out += list(P.mx_linear_backward(dy, wq, bias_grad=True, workspace=ws))
    out += list(P.rms_norm_backward(x, r, w, dS=x, workspace=ws))
    out.append(P.rms_norm(x, w)[0])
    return out


@pytest.mark.parametrize("m", [3, 200])
def test_capture_and_replay(m):
    d, n = 384, 520
    x, r, w = gauss(1, m, d).bfloat16(), gauss(2, m, d).bfloat16(), gauss(3, d).bfloat16()
    dy, wq = gauss(4, m, n).bfloat16(), P.mx_quantize(gauss(5, n, d), "fp4")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    all_calls(x, r, w, wq, dy, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = all_calls(x, r, w, wq, dy, ws)
    for step in range(4):
        x.copy_(gauss(10 + step, m, d))
        dy.copy_(gauss(20 + step, m, n))
        ws.fill_(255)                                     # whatever other calls left
        graph.replay()
        torch.cuda.synchronize()
        again = all_calls(x, r, w, wq, dy)
        assert all(torch.equal(a, b) for a, b in zip(kept, again)), step


@pytest.mark.parametrize("m", [5, 180])
def test_streams_and_repeats(m):
    d, n = 1000, 300
    args = []
    for i in range(2):
        args.append((gauss(1 + i, m, d).bfloat16(), gauss(2 + i, m, d).bfloat16(), gauss(3 + i, d).bfloat16(),
                     P.mx_quantize(gauss(5 + i, n, d), "fp4"), gauss(4 + i, m, n).bfloat16()))
    want = [all_calls(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = all_calls(*args[i])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    st = streams[0]
    st.wait_stream(torch.cuda.current_stream())
    y = P.mx_linear(args[0][0], args[0][3], stream=st)
    q = P.mx_quantize(args[0][0], "fp8", stream=st)
    st.synchronize()
    assert torch.equal(y, P.mx_linear(args[0][0], args[0][3]))
    assert torch.equal(q.codes, P.mx_quantize(args[0][0], "fp8").codes)


def test_refusals():
    x, w = gauss(1, 4, 256), P.mx_quantize(gauss(2, 32, 256), "fp4")
    with pytest.raises(ValueError):
        P.mx_linear(x[:, :200].contiguous(), w)
    with pytest.raises(ValueError):
        P.mx_linear(x.t(), w)
    with pytest.raises(TypeError):
        P.mx_linear(x.half(), w)
    with pytest.raises(ValueError):
        P.mx_linear(x, w, activation="tanh")
    with pytest.raises(TypeError):
        P.mx_linear(x, w, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        P.mx_linear(x, w, residual=torch.zeros(4, 32, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        P.mx_linear(x, w, bias=torch.zeros(31, device=DEV))
    with pytest.raises(ValueError):
        P.mx_linear_backward(x, w)
    with pytest.raises(ValueError, match="preact"):
        P.mx_linear_backward(torch.zeros(4, 32, device=DEV), w, activation="silu")
    with pytest.raises(ValueError):
        P.rms_norm(x, torch.ones(255, device=DEV))
    with pytest.raises(TypeError):
        P.rms_norm(x, torch.ones(256, device=DEV).bfloat16())
    with pytest.raises(P.GptqError):
        P.rms_norm(x, torch.ones(256, device=DEV), eps=-1.0)
    with pytest.raises(ValueError):
        P.rms_norm(x, torch.ones(256, device=DEV), format="fp6")
    with pytest.raises(ValueError, match="no_grad"):
        P.mx_linear(x.clone().requires_grad_(), w)
    with pytest.raises(ValueError, match="no_grad"):
        P.rms_norm(x, torch.ones(256, device=DEV, requires_grad=True))
    with torch.no_grad():
        P.mx_linear(x.clone().requires_grad_(), w)
