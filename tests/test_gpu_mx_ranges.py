"""GPU tests of the MX operators and the norm at the ends of their range, and
of the product forms that only large or particular shapes select.

Tolerances as in test_gpu_mx.py unless a test states its own.
"""
from fractions import Fraction

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_mx import (DEV, DT, F64, HALF_STEP, P, SLOPE, act64, bounds, codes_of, gauss, ints,  # noqa: E402
                         make_acts, ref_quantize, say, slope64, values_of)


# ---------------------------------------------------------------------------
# the norm's backward pass
# ---------------------------------------------------------------------------
# sizes of a row's S and dY, such that r dY w stays inside fp32 (and bf16)
SIZES = [(1e38, 1e10), (1e30, 1e-5), (1.0, 1.0), (1e-25, 1e-10), (1e-36, 1e-12), (3e37, 1e25), (1e-40, 1e-20)]


@pytest.mark.parametrize("wsize", [1.0, 1e-20, 1e20])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,d", [(9, 1000), (14, 96), (300, 520), (260, 8192), (37, 1407), (20, 9000), (7, 33000)])
def test_norm_backward_at_the_ends_of_the_range(m, d, dtype, wsize):
    """Rows whose factor r, r^2, or whose products dY w leave fp32 although the results do not; eps = 0.

    In 64 bits, with a relative error far below 2^-40 of the terms; dX is rounded to fp32, and from
    there to bf16, dw's groups to fp32 and their sum again."""
    say("norm backward range", m, d, dtype, wsize)
    size = torch.tensor(SIZES, dtype=F64, device=DEV)[torch.arange(m, device=DEV) % len(SIZES)]
    # (clamped: no value beyond the type's largest, and of subnormal rows some that are not zero)
    s = (gauss(d, m, d).double().clamp(-3, 3) * size[:, :1]).to(DT[dtype])
    w = ((1 + 0.2 * gauss(2, d)).double() * wsize).to(DT[dtype])
    dy = (gauss(3, m, d).double() * size[:, 1:] * (1e-8 if wsize > 1 else 1)).to(DT[dtype])
    v, g = s.double(), dy.double()
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True))
    n, gw = v * r, g * w.double()
    want = r * (gw - n * (gw * n).mean(1, keepdim=True))
    assert torch.isfinite(want).all() and float(want.abs().max()) < 1e38
    size = r * (gw.abs() + n.abs() * (gw * n).abs().mean(1, keepdim=True))
    step = {"bf16": 2.0 ** -8 + 2.0 ** -23, "f32": 2.0 ** -24}[dtype]
    least = {"bf16": 2.0 ** -134 + 2.0 ** -150, "f32": 2.0 ** -150}[dtype]
    dx, dw = P.rms_norm_backward(dy, s, w, eps=0.0)
    e = 2.0 ** -40 * size
    assert ((dx.double() - want).abs() <= e + step * (want.abs() + e) + least).all()
    terms = g * n
    assert ((dw.double() - terms.sum(0)).abs() <= 2.0 ** -22 * terms.abs().sum(0)).all()


@pytest.mark.parametrize("m,d", [(51456, 8192), (10251, 40000)])
def test_norm_weight_gradients_of_many_rows(m, d):
    """dw where a column's later terms are 2^-25 of the first ones: a chain of fp32 additions would lose each.

    Terms are exact; the groups' sums and the result are rounded to fp32: 2^-23 of the sum, as all are positive."""
    first, small = 256, 2.0 ** -25
    s = torch.ones(m, d, dtype=torch.bfloat16, device=DEV)
    dy = torch.ones(m, d, dtype=torch.bfloat16, device=DEV)
    column = (1 + (torch.arange(d, device=DEV) % 8) / 8).bfloat16()
    dy[first:] = column * small
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    _, dw = P.rms_norm_backward(dy, s, w, eps=0.0)
    want = first + (m - first) * small * column.double()
    assert ((dw.double() - want).abs() <= 2.0 ** -23 * want).all()


# ---------------------------------------------------------------------------
# the norm's outputs
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", [None, "fp8", "fp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1, 32, 98, 100, 1407, 4096, 9000])
def test_norm_of_rows_with_exact_results(d, dtype, fmt):
    """Constant rows with eps = 0: the results are the weights themselves, on the borders of the grids."""
    m = 256
    x = (torch.arange(m, device=DEV) + 1.0).view(m, 1).expand(m, d)
    sign = 1 - 2 * (torch.arange(d, device=DEV) % 3 == 1).float()
    w = torch.tensor([1.0, 2.0, 0.5, 448.0, 6.0, 0.875], device=DEV)[torch.arange(d, device=DEV) % 6]
    y, _ = P.rms_norm((x * sign).to(DT[dtype]).contiguous(), w.to(DT[dtype]), eps=0.0, format=fmt)
    want = (w * sign).double().expand(m, d)
    if fmt is None:
        assert torch.equal(y.double(), want)
    else:
        codes, byte = ref_quantize(want, fmt)
        got, scales = codes_of(y)
        assert torch.equal(scales, byte.to(torch.int64)) and torch.equal(got, codes)


def test_norm_with_eps_of_exact_results():
    """mean + eps a square: 3^2 + 7 = 4^2, 12^2 + 25 = 13^2, 49^2 + 200 = 51^2, 0 + 9."""
    for value, eps, root in ((3, 7, 4), (12, 25, 13), (49, 200, 51), (0, 9, 3)):
        x = torch.full((300, 200), float(value), device=DEV)
        for weight in (1.0, 7.0, float(root)):
            want = Fraction(value) * Fraction(weight) / root
            y, _ = P.rms_norm(x, torch.full((200,), weight, device=DEV), eps=float(eps))
            assert torch.equal(y, torch.full_like(y, float(want))), (value, weight)
            q, _ = P.rms_norm(x, torch.full((200,), weight, device=DEV), eps=float(eps), format="fp8")
            codes, byte = ref_quantize(torch.full((300, 200), float(want), dtype=F64), "fp8")
            got, scales = codes_of(q)
            assert torch.equal(scales, byte.to(torch.int64)) and torch.equal(got, codes), (value, weight)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,d", [(5, 200), (300, 70), (300, 130), (3, 20010)])
def test_padding_behind_rows_that_are_not_finite(m, d, dtype, fmt):
    """Columns and blocks behind d have codes and scale bytes 0, whatever the row."""
    x = gauss(1, m, d)
    x[0] = 0                                              # with eps = 0: 0 / 0
    x[1, 3], x[2, d - 1] = float("inf"), float("nan")
    y, _ = P.rms_norm(x.to(DT[dtype]), (1 + 0.1 * gauss(2, d)).to(DT[dtype]), eps=0.0, format=fmt)
    for t in (y, P.mx_quantize(x.to(DT[dtype]), fmt)):
        codes, scales = codes_of(t)
        assert (codes[:, d:] == 0).all() and (scales[:, -(-d // 32):] == 0).all()
    codes, scales = codes_of(y)
    assert (scales[0, :-(-d // 32)] == 255).all() and (scales[2, :-(-d // 32)] == 255).all()
    assert (scales[3:] != 255).all()


# ---------------------------------------------------------------------------
# product forms that particular shapes select
# ---------------------------------------------------------------------------
# (m, n, k, kind, out): MX activations through tiles of 256 x 256 (at least 128 of them, 32 stages), ragged at
# both ends, outputs 8, 4 and 1 at a time; the dense form's tiles of that size with MX weights, and with fp8
# activations; rows up to 64 through the few-row form
FORMS = [(2051, 3864, 4129, "fp8", "bf16"), (2051, 3860, 4129, "fp4", "f32"), (2051, 3857, 4129, "fp8", "bf16"),
         (2051, 3857, 4129, "fp4", "bf16"), (2051, 3857, 1033, "f32", "f32"), (2051, 3860, 1033, "fp8", "f32"),
         (2051, 3864, 1033, "bf16", "bf16"), (2051, 3857, 1033, "f32", "bf16"),
         *((m, n, k, kind, out) for m, n, k in ((33, 2049, 1000), (64, 2500, 4100))
           for kind in ("bf16", "f32", "fp8", "fp4") for out in ("bf16", "f32"))]


@pytest.mark.parametrize("m,n,k,kind,out", FORMS)
def test_forms_with_exact_operands(m, n, k, kind, out):
    say("form, exact", m, n, k, kind, out)
    x = ints(m * 31 + k, -2, 3, m, k)
    w = ints(n * 17 + k, -3, 4, n, k) * torch.exp2(ints(n, -2, 3, n, 1))
    x[:, 0] = 2.0
    wq = P.mx_quantize(w, "fp4")
    a, a64 = make_acts(kind, x)
    want = a64 @ values_of(wq).t()
    b, r = ints(1, -9, 10, n).to(DT[out]), ints(2, -9, 10, m, n).to(DT[out])
    y = P.mx_linear(a, wq, out_dtype=DT[out])
    assert torch.equal(y, want.float().to(DT[out]))
    y, z = P.mx_linear(a, wq, bias=b, activation="relu", residual=r, out_dtype=DT[out], save_preact=True)
    want = want + b.double()
    assert torch.equal(z, want.float().to(DT[out]))
    assert torch.equal(y, (want.clamp(min=0) + r.double()).float().to(DT[out]))


@pytest.mark.parametrize("m,n,k,kind,out", FORMS)
def test_forms(m, n, k, kind, out):
    say("form", m, n, k, kind, out)
    x = gauss(m + n, m, k) * torch.exp(gauss(k, k))
    wq = P.mx_quantize(gauss(n * k, n, k) * 0.05, "fp4")
    a, a64 = make_acts(kind, x)
    w64 = values_of(wq)
    b, r = gauss(1, n).to(DT[out]), gauss(2, m, n).to(DT[out])
    y, z = P.mx_linear(a, wq, bias=b, activation="silu", residual=r, out_dtype=DT[out], save_preact=True)
    z64 = a64 @ w64.t() + b.double()
    e = bounds(kind, out, m, a64, w64, m > 32 and (kind in DT or (kind, out) == ("fp8", "f32"))) + 2.0 ** -24 * z64.abs()
    assert ((z.double() - z64).abs() <= e + HALF_STEP[out] * (z64.abs() + e)).all()
    y64 = act64(z64, "silu") + r.double()
    e = SLOPE * e + 2.0 ** -20 * (z64.abs() + 1) + 2.0 ** -24 * y64.abs()
    assert ((y.double() - y64).abs() <= e + HALF_STEP[out] * (y64.abs() + e)).all()


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("m,n,k", [(2051, 1033, 3857), (2051, 1033, 3860), (2051, 1033, 3864)])
def test_backward_through_large_tiles(m, n, k, dtype, out):
    say("backward, large tiles", m, n, k, dtype, out)
    wq = P.mx_quantize(gauss(n * k, n, k) * 0.05, "fp4")
    w64 = values_of(wq)
    dy, z = gauss(5, m, n).to(DT[dtype]), (gauss(6, m, n) * 1.5).to(DT[dtype])
    da, db = P.mx_linear_backward(dy, wq, activation="gelu", preact=z, bias_grad=True, out_dtype=DT[out])
    dz = dy.double() * slope64(z.double(), "gelu")
    want = dz @ w64
    e = bounds("dz", out, m, dz, w64.t(), True) + 2.0 ** -20 * (dy.double().abs() @ w64.abs())
    assert ((da.double() - want).abs() <= e + HALF_STEP[out] * (want.abs() + e)).all()
    e = 2.0 ** -24 * (m + 4) * dz.abs().sum(0) + 2.0 ** -20 * dy.double().abs().sum(0)
    assert ((db.double() - dz.sum(0)).abs() <= e).all()


@pytest.mark.parametrize("m", [8, 20, 60])
@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8"])
def test_subnormal_activations_in_few_rows(m, kind):
    """The few-row form holds an activation to within 2^-133 (bf16's smallest step) at worst."""
    n, k = 2100, 256
    a, a64 = make_acts(kind, gauss(1, m, k) * 2.0 ** -126)
    wq = P.mx_quantize(gauss(2, n, k) * 2.0 ** 20, "fp4")
    w64 = values_of(wq)
    want = a64 @ w64.t()
    got = P.mx_linear(a, wq, out_dtype=torch.float32)
    e = bounds(kind, "f32", m, a64, w64, m > 32) + 2.0 ** -133 * w64.abs().sum(1)
    assert ((got.double() - want).abs() <= e + 2.0 ** -24 * (want.abs() + e)).all()
    if kind in DT:
        dy = (gauss(3, m, n) * 2.0 ** -126).to(DT[kind])
        da, _ = P.mx_linear_backward(dy, wq, out_dtype=torch.float32)
        want = dy.double() @ w64
        e = bounds("dz", "f32", m, dy.double(), w64.t(), True) + 2.0 ** -133 * w64.abs().sum(0)
        assert ((da.double() - want).abs() <= e + 2.0 ** -24 * (want.abs() + e)).all()
