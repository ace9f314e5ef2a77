"""GPU tests of the MX operators on matrices whose offsets pass 32 bits, and at
the largest number of columns.

Operands are small integers whose sums fp32 holds, so that every form gives the
same bits, and parts of a large call can be compared with calls on its parts.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_mx import DEV, DT, P, gauss, ints, make_acts, say, values_of  # noqa: E402

KINDS = ["bf16", "f32", "fp8", "fp4"]


def part_of(t, rows):
    return P.MxTensor(t.codes[rows].contiguous(), t.scales[:, rows].contiguous(), t.format, t.d)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_quantize_beyond_32_bit_offsets(fmt):
    rows, d = 70001, 65536                                # 4.6 G elements
    x = torch.empty(rows, d, dtype=torch.bfloat16, device=DEV)
    for i in range(0, rows, 8192):
        x[i:i + 8192] = gauss(i, min(8192, rows - i), d).bfloat16()
    t = P.mx_quantize(x, fmt)
    y = P.mx_dequantize(t, torch.bfloat16)
    for first in (0, 32766, 65535, rows - 40):            # (2^31 and 2^32 elements are row 32768 and 65536)
        some = slice(first, first + 40)
        q = P.mx_quantize(x[some].contiguous(), fmt)
        assert torch.equal(t.codes[some], q.codes) and torch.equal(t.scales[:, some], q.scales), first
        assert torch.equal(y[some], P.mx_dequantize(q, torch.bfloat16)), first


@pytest.mark.parametrize("kind", KINDS)
def test_activations_beyond_32_bit_offsets(kind):
    m, n, k = 140001, 40, 65536                           # 9.2 G elements, fp4 4.6 GB
    say("large activations", kind)
    x = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
    tail = ints(1, -2, 3, 300, k)
    tail[:, 0] = 2.0
    x[-300:] = tail.bfloat16()
    x[32767] = tail[0].bfloat16()
    a = x if kind == "bf16" else (x[-66000:].float() if kind == "f32" else P.mx_quantize(x, kind))
    wq = P.mx_quantize(ints(2, -3, 4, n, k), "fp4")
    want = tail.double() @ values_of(wq).t()
    y = P.mx_linear(a, wq, out_dtype=torch.float32)
    assert torch.equal(y[-300:].double(), want)
    if kind != "f32":
        assert torch.equal(y[32767].double(), want[0])
        y[32767] = 0
    assert not y[:-300].any()


@pytest.mark.parametrize("kind", KINDS)
def test_weights_beyond_32_bit_offsets(kind):
    n, k = 140001, 65536                                  # 4.6 GB of codes
    w = torch.zeros(n, k, dtype=torch.bfloat16, device=DEV)
    tail = ints(1, -3, 4, 70, k)
    w[-70:] = tail.bfloat16()
    wq = P.mx_quantize(w, "fp4")
    del w
    part = values_of(part_of(wq, slice(n - 70, n)))
    for m in (3, 40, 100):
        say("large weights", kind, m)
        x = ints(2, -2, 3, m, k)
        x[:, 0] = 2.0
        a, a64 = make_acts(kind, x)
        y = P.mx_linear(a, wq, out_dtype=torch.float32)
        assert torch.equal(y[:, -70:].double(), a64 @ part.t())
        assert not y[:, :-70].any()
        if kind in DT:
            dy = ints(3, -2, 3, m, n).to(DT[kind])
            da, db = P.mx_linear_backward(dy, wq, bias_grad=True, out_dtype=torch.float32)
            assert torch.equal(da.double(), dy[:, -70:].double() @ part)
            assert torch.equal(db.double(), dy.double().sum(0))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m", [2, 50, 130])
def test_products_of_the_most_columns(m, kind):
    n, k = 33, 1 << 19
    say("most columns", m, kind)
    x = ints(1, -2, 3, m, k)
    x[:, 0] = 2.0
    wq = P.mx_quantize(ints(2, -3, 4, n, k), "fp4")
    a, a64 = make_acts(kind, x)
    assert torch.equal(P.mx_linear(a, wq, out_dtype=torch.float32).double(), a64 @ values_of(wq).t())
    if kind in DT:
        dy = ints(3, -2, 3, m, n).to(DT[kind])
        da, _ = P.mx_linear_backward(dy, wq, out_dtype=torch.float32)
        assert torch.equal(da.double(), dy.double() @ values_of(wq))


@pytest.mark.parametrize("m", [1, 300])
def test_norm_of_the_most_columns(m):
    d = 1 << 19
    x, w = gauss(1, m, d).bfloat16(), (1 + 0.1 * gauss(2, d)).bfloat16()
    y, s = P.rms_norm(x, w, residual=x)
    v = s.double()
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
    want = v * r * w.double()
    assert ((y.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -40) * want.abs()).all()
    q, _ = P.rms_norm(x, w, residual=x, format="fp8")
    back = P.mx_dequantize(q).double()
    # (half a step 2^-4, of subnormal elements 2^-10 2^E with a block's largest above 2^(E + 8); saturated
    # from below 512 to 448: 2^-3)
    top = want.abs().view(m, -1, 32).amax(2).repeat_interleave(32, 1)
    assert ((back - want).abs() <= 2.0 ** -3 * want.abs() + 2.0 ** -18 * top).all()
    del back, top
    dx, dw = P.rms_norm_backward(x, s, w)
    gw = x.double() * w.double()
    want = r * (gw - v * r * (gw * v * r).mean(1, keepdim=True))
    e = 2.0 ** -21 * (r * gw.abs() + r * (v * r).abs())
    assert ((dx.double() - want).abs() <= e + 2.0 ** -8 * (want.abs() + e)).all()
    terms = x.double() * v * r
    assert ((dw.double() - terms.sum(0)).abs() <= 2.0 ** -22 * terms.abs().sum(0)).all()
