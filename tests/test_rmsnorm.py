"""RMS norm into 8-bit operands and its backward pass on the GPU, against the
formulas in 64 bits.

Tolerances.  The fp32 sum of squares goes through at most 64 additions in a
thread and 10 across threads, each within 2^-24 of a positive sum, so rstd
and y are within 2^-18 of the formula, relative; an output type adds half a
step (bf16 2^-8, E4M3 2^-4 of the value or half its smallest step, 2^-10).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32_REL = 2.0 ** -18
BF16 = torch.bfloat16


def _data(rows, cols, seed, ld=None, residual=False):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn((rows, ld or cols), generator=g) * torch.exp(torch.randn((rows, 1), generator=g))
    x = wide.to(BF16).cuda()[:, :cols]
    w = (1 + 0.2 * torch.randn((cols,), generator=g)).to(BF16).cuda()
    r = (2 * torch.randn((rows, cols), generator=g)).to(BF16).cuda() if residual else None
    return x, w, r


def _ref(x, w, r, eps):
    s = x.double() + (r.double() if r is not None else 0)
    rstd = 1 / (s.square().mean(1) + eps).sqrt()
    return s, rstd, s * rstd[:, None] * w.double()


def _near(got, want, rel, floor=0.0):
    """|got - want| <= rel |want| + floor, and the same values that are not finite."""
    got, want = got.double(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    over = (got - want).abs() - (rel * want.abs() + floor)
    over = over[fine]
    assert over.numel() == 0 or over.max().item() <= 0, f"over by {over.max().item():.3g}"


def _check_codes(fpq, fmt, q, scales, y):
    """Codes and scales of the fp32 y: the scale from the block's largest
    magnitude, each code the nearest E4M3 value of y / scale."""
    rows, cols = y.shape
    width = 128 if fmt == fpq.FP8_1x128 else 32
    t = y.view(rows, cols // width, width)
    top = t.abs().amax(-1)
    if fmt == fpq.FP8_1x128:
        s = scales.double()
        _near(s, torch.where(top > 0, top / 448, torch.ones_like(top)), F32_REL + 2.0 ** -24)
    else:
        s = torch.exp2(scales.double() - 127)
        exact = torch.exp2(torch.ceil(torch.log2((top / 448).clamp_min(2.0 ** -127))))
        near = torch.exp2(torch.ceil(torch.log2((top * (1 - F32_REL) / 448).clamp_min(2.0 ** -127)))), \
            torch.exp2(torch.ceil(torch.log2((top * (1 + F32_REL) / 448).clamp_min(2.0 ** -127))))
        assert torch.all((s == exact) | (s == near[0]) | (s == near[1]))
    want = t / s[..., None]
    got = q.view(torch.float8_e4m3fn).double().view_as(want)
    # a quotient up to 2^-17 above 448 saturates to it
    _near(got, want, 2.0 ** -4 + 2.0 ** -17, 2.0 ** -10 * (1 + 2.0 ** -17))


SHAPES = [(1, 128), (3, 256), (9, 384), (17, 1024), (5, 1152), (2, 7168), (301, 2048), (700, 7168), (1, 16384),
          (305, 8320), (3, 32768)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("name", ["FP8_1x128", "MXFP8", None])
def test_forward(fpq, rows, cols, residual, name):
    fmt = None if name is None else getattr(fpq, name)
    x, w, r = _data(rows, cols, rows + cols, residual=residual)
    out = fpq.rmsnorm_quantize(x, w, fmt, eps=1e-5, residual=r, want_y=True, want_rstd=True)
    s, rstd, y = _ref(x, w, r, 1e-5)
    _near(out.rstd, rstd, F32_REL)
    _near(out.y, y, 2.0 ** -8 + F32_REL)
    if residual:
        _near(out.h, s, 2.0 ** -8 + 2.0 ** -23)
    else:
        assert out.h is None
    if fmt is not None:
        _check_codes(fpq, fmt, out.q, out.scales, y)
    assert fpq.fpq_get_device_error() == 0


@pytest.mark.parametrize("cols", [8, 24, 40, 1000, 1032, 2056, 7176, 16392])
@pytest.mark.parametrize("rows", [1, 7, 320])
def test_odd_widths(fpq, rows, cols):
    x, w, r = _data(rows, cols, cols, residual=True)
    out = fpq.rmsnorm_quantize(x, w, residual=r, want_rstd=True)
    s, rstd, y = _ref(x, w, r, 1e-6)
    _near(out.y, y, 2.0 ** -8 + F32_REL)
    _near(out.rstd, rstd, F32_REL)
    assert out.q is None and out.scales is None


@pytest.mark.parametrize("cols", [32, 96, 1056, 4128])
def test_mxfp8_odd_widths(fpq, cols):
    x, w, _ = _data(13, cols, cols)
    out = fpq.rmsnorm_quantize(x, w, fpq.MXFP8)
    assert out.y is None and out.h is None and out.rstd is None
    _check_codes(fpq, fpq.MXFP8, out.q, out.scales, _ref(x, w, None, 1e-6)[2])


@pytest.mark.parametrize("rows,cols,ld", [(67, 512, 576), (300, 1536, 1544), (2, 128, 4096), (1, 256, 264)])
def test_strided_rows(fpq, rows, cols, ld):
    x, w, _ = _data(rows, cols, ld, ld=ld)
    a = fpq.rmsnorm_quantize(x, w, fpq.FP8_1x128, want_y=True, want_rstd=True)
    b = fpq.rmsnorm_quantize(x.contiguous(), w, fpq.FP8_1x128, want_y=True, want_rstd=True)
    for u, v in zip(a, b):
        assert u is v is None or torch.equal(u, v)
    dy = torch.randn((rows, cols), device="cuda").to(BF16)
    for u, v in zip(fpq.rmsnorm_backward(dy, x, w, a.rstd), fpq.rmsnorm_backward(dy, x.contiguous(), w, a.rstd)):
        assert torch.equal(u, v)


def test_in_place_residual_and_rows_behind(fpq):
    """h over the residual's buffer; the rows behind the given ones stay."""
    rows, cols = 5, 1152
    x, w, r = _data(rows + 2, cols, 7, residual=True)
    want = fpq.rmsnorm_quantize(x[:rows], w, residual=r[:rows])
    h, y = r.clone(), torch.full_like(r, 3.0)
    fpq.fpq_rmsnorm_quantize(0, x, cols, h, w, rows, cols, 1e-6, h=h, y=y)
    assert torch.equal(h[:rows], want.h) and torch.equal(y[:rows], want.y)
    assert torch.equal(h[rows:], r[rows:]) and torch.all(y[rows:] == 3.0)


@pytest.mark.parametrize("name", ["FP8_1x128", "MXFP8"])
def test_rows_that_are_not_ordinary(fpq, name):
    """Zero rows, rows with a NaN or an infinity, tiny and huge values: the
    formula's values, and no effect on the rows beside them."""
    fmt = getattr(fpq, name)
    x, w, _ = _data(8, 256, 11)
    x = x.clone()
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 2.0 ** -60
    x[5] = (x[5].float() * 2.0 ** 50).to(BF16)
    out = fpq.rmsnorm_quantize(x, w, fmt, want_y=True, want_rstd=True)
    clean = fpq.rmsnorm_quantize(x[[0, 6, 7]], w, fmt, want_y=True, want_rstd=True)
    for u, v in zip(out, clean):
        assert u is v is None or torch.equal(u[[0, 6, 7]], v)
    assert torch.all(out.q[1] == 0) and torch.all(out.y[1] == 0)
    assert torch.all(out.scales[1] == (1.0 if fmt == fpq.FP8_1x128 else 0))
    assert torch.isnan(out.rstd[2]) and torch.all(torch.isnan(out.y[2]))
    assert torch.all((out.q[2] & 0x7F) == 0x7F)
    # an infinity: rstd is 0, the finite entries 0, the infinite one NaN
    assert out.rstd[3] == 0 and torch.isnan(out.y[3, 7]) and torch.all(out.y[3, :7] == 0)
    y = _ref(x[4:6], w, None, 1e-6)[2]
    _near(out.y[4:6], y, 2.0 ** -8 + F32_REL)
    _check_codes(fpq, fmt, out.q[4:6], out.scales[4:6], y)
    assert fpq.fpq_get_device_error() == 0


def _ref_backward(dy, x, w, rstd, dres):
    d, v, r = dy.double(), x.double(), rstd.double()[:, None]
    g = d * w.double()
    dx = r * g - v * r ** 3 * (g * v).mean(1, keepdim=True)
    size = r * g.abs() + v.abs() * r ** 3 * (g * v).abs().mean(1, keepdim=True)
    if dres is not None:
        dx, size = dx + dres.double(), size + dres.double().abs()
    return dx, size, (d * v * r).sum(0), (d * v * r).abs().sum(0)


@pytest.mark.parametrize("rows,cols", SHAPES + [(1, 8), (4, 40), (2050, 64), (1500, 1032), (40, 16392),
                                                (1500, 2048), (900, 4096), (310, 16384), (310, 16392)])
@pytest.mark.parametrize("residual", [False, True])
def test_backward(fpq, rows, cols, residual):
    """Errors count against the sums of magnitudes: 2^-17 of them covers the
    dot product's additions (at most 74) and, for dweight, those over rows (a
    CTA's rows, then its share of the partial rows: under 100; each at most
    2^-24 of the sum)."""
    x, w, _ = _data(rows, cols, rows + cols + 1)
    g = torch.Generator().manual_seed(3)
    dy = torch.randn((rows, cols), generator=g).to(BF16).cuda()
    dres = torch.randn((rows, cols), generator=g).to(BF16).cuda() if residual else None
    rstd = _ref(x, w, None, 1e-6)[1].float()
    dx, dw = fpq.rmsnorm_backward(dy, x, w, rstd, dres=dres)
    want, size, want_w, size_w = _ref_backward(dy, x, w, rstd, dres)
    _near(dx, want, 2.0 ** -8, 2.0 ** -17 * size)
    _near(dw, want_w, 0.0, 2.0 ** -17 * size_w)
    again = fpq.rmsnorm_backward(dy, x, w, rstd, dres=dres)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_backward_against_differences(fpq):
    """The gradient's direction against the change of sum(dy y) in 64 bits."""
    x, w, _ = _data(4, 256, 21)
    dy = torch.randn((4, 256), device="cuda").to(BF16)
    rstd = fpq.rmsnorm_quantize(x, w, want_rstd=True).rstd
    dx, dw = fpq.rmsnorm_backward(dy, x, w, rstd)
    f = lambda a, b: (_ref(a, b, None, 1e-6)[2] * dy.double()).sum()       # noqa: E731
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        u = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
        v = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        slope = (f(x.double() + h * u, w.double() + h * v) - f(x.double() - h * u, w.double() - h * v)) / (2 * h)
        got = (dx.double() * u).sum() + (dw.double() * v).sum()
        # dx is bf16: half a step of each term, and the difference's own h^2
        tol = 2.0 ** -8 * (dx.double() * u).abs().sum() + 1e-4
        assert abs(got - slope) <= tol


def test_no_rows(fpq):
    x = torch.empty((0, 256), dtype=BF16, device="cuda")
    w = torch.ones((256,), dtype=BF16, device="cuda")
    out = fpq.rmsnorm_quantize(x, w, fpq.MXFP8, want_y=True, want_rstd=True)
    assert out.q.shape == (0, 256) and out.scales.shape == (0, 8) and out.rstd.shape == (0,)
    dx, dw = fpq.rmsnorm_backward(x, x, w, out.rstd)
    assert dx.shape == (0, 256) and torch.all(dw == 0)


def test_same_as_quantizing_the_rows_of_a_product(fpq):
    """With a weight of ones and rows whose norm is exactly representable, the
    codes are those that quantize() gives for the normed rows."""
    x = torch.zeros((6, 256), dtype=BF16, device="cuda")
    x[:, ::2] = 1                                                                  # mean square 1/2
    w = torch.ones((256,), dtype=BF16, device="cuda")
    out = fpq.rmsnorm_quantize(x * 2, w, fpq.MXFP8, eps=2.0)                       # rstd = 1 / 2
    q, s = fpq.quantize(x, fpq.MXFP8)
    assert torch.equal(out.q, q) and torch.equal(out.scales, s)


@pytest.mark.parametrize("rows,cols", [(700, 40), (2000, 1024), (900, 2048), (500, 7168), (310, 16384), (310, 16392)])
@pytest.mark.parametrize("over", ["dy", "dres"])
def test_backward_in_place(fpq, rows, cols, over):
    x, w, _ = _data(rows, cols, 31)
    dy, dres = (torch.randn((rows, cols), device="cuda").to(BF16) for _ in range(2))
    rstd = _ref(x, w, None, 1e-6)[1].float()
    want = fpq.rmsnorm_backward(dy, x, w, rstd, dres=dres)
    buf = {"dy": dy, "dres": dres}
    dw = torch.empty((cols,), device="cuda")
    ws = torch.empty((fpq.fpq_rmsnorm_backward_workspace_bytes(rows, cols),), dtype=torch.uint8, device="cuda")
    fpq.fpq_rmsnorm_backward(dy, x, cols, w, rstd, dres, rows, cols, buf[over], dw, ws)
    assert torch.equal(buf[over], want[0]) and torch.equal(dw, want[1])


def test_without_a_weight_gradient(fpq):
    x, w, _ = _data(33, 512, 32)
    dy = torch.randn((33, 512), device="cuda").to(BF16)
    rstd = _ref(x, w, None, 1e-6)[1].float()
    dx = torch.empty_like(dy)
    fpq.fpq_rmsnorm_backward(dy, x, 512, w, rstd, None, 33, 512, dx)
    assert torch.equal(dx, fpq.rmsnorm_backward(dy, x, w, rstd)[0])


def test_far_rows(fpq):
    """Rows past 2^32 bytes and 2^31 elements from the first, dense and strided."""
    rows, cols = 330000, 8192
    x = torch.zeros((rows, cols), dtype=BF16, device="cuda")
    part, w, _ = _data(64, cols, 33)
    x[-64:] = part
    out = fpq.rmsnorm_quantize(x, w, fpq.MXFP8, want_y=True, want_rstd=True)
    _, rstd, y = _ref(part, w, None, 1e-6)
    _near(out.rstd[-64:], rstd, F32_REL)
    _near(out.y[-64:], y, 2.0 ** -8 + F32_REL)
    _check_codes(fpq, fpq.MXFP8, out.q[-64:], out.scales[-64:], y)
    half = fpq.rmsnorm_quantize(x[:, :4096], w[:4096].contiguous(), want_rstd=True)
    _near(half.y[-64:], _ref(part[:, :4096], w[:4096], None, 1e-6)[2], 2.0 ** -8 + F32_REL)
    dx, dw = fpq.rmsnorm_backward(out.y, x, w, out.rstd)
    dy, rstd = out.y[-64:].clone(), out.rstd[-64:].clone()
    dx_near, dw_near = fpq.rmsnorm_backward(dy, part.contiguous(), w, rstd)
    assert torch.equal(dx[-64:], dx_near)
    # the other rows add zeros; the same 64 products are added in two orders,
    # each within 64 steps of 2^-24 of the magnitudes' sum
    size = (dy.double() * part.double() * rstd.double()[:, None]).abs().sum(0)
    assert torch.all((dw.double() - dw_near.double()).abs() <= 2.0 ** -17 * size)


@pytest.mark.parametrize("rows,cols,residual", [(4099, 512, False), (700, 1024, True), (3, 7168, False), (700, 7168, True),
                                                (310, 16384, False), (310, 32768, True)])
def test_fp8_codes_are_those_of_the_fp32_quotient(fpq, rows, cols, residual):
    """Bit for bit the rule of quantize(): scale = fp32(amax / 448), code = the
    rounding of fp32(y / scale), for the fp32 y that the kernel forms.  bf16
    products meet the midpoints between codes often, so the quotient's last
    place counts."""
    x, w, r = _data(rows, cols, 61, residual=residual)
    x[0, :256] = -0.0                                                # zeros of both signs
    w[5], w[6] = 0.0, -0.0
    if residual:
        r[0, :256] = -0.0
    out = fpq.rmsnorm_quantize(x, w, fpq.FP8_1x128, residual=r, want_rstd=True)
    s = x.float() + r.float() if residual else x.float()
    t = (s * out.rstd[:, None] * w.float()).view(rows, cols // 128, 128)
    top = t.abs().amax(-1)
    # a tensor of divisors: by a Python number torch multiplies with its reciprocal
    scale = torch.where(top == 0, torch.ones_like(top), top / torch.full_like(top, 448.0))
    assert torch.equal(out.scales, scale)
    want = (t / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, cols)
    assert torch.equal(out.q, want), f"{(out.q != want).sum().item()} codes of {want.numel()}"


def test_fp8_tile_whose_scale_rounds_to_zero(fpq):
    """amax / 448 of a magnitude below 224 steps of fp32 rounds to 0: the
    tile's scale is 1 then and its codes 0, as for a tile of zeros."""
    x = torch.zeros((2, 384), dtype=BF16, device="cuda")
    x[0, 130], x[0, 131], x[0, 300] = 2.0 ** -60, -2.0 ** -60, 1.0
    x[1, 0], x[1, 200] = 2.0 ** -60, float("nan")
    w = torch.ones((384,), dtype=BF16, device="cuda")
    for residual in (None, torch.zeros_like(x)):
        # sum of squares 1: rstd is about 19.6, y 627 steps of 2^-149, its scale one step
        w[128:256] = 2.0 ** -84
        out = fpq.rmsnorm_quantize(x, w, fpq.FP8_1x128, residual=residual)
        q, s = out.q.cpu(), out.scales.cpu()
        assert s[0].tolist()[:2] == [1.0, 2.0 ** -149] and q[0, 130:132].tolist() == [0x7E, 0xFE]
        q[0, 130:132] = 0
        assert torch.all(q[0, :256] == 0) and q[0, 300] == 0x7E
        w[128:256] = 2.0 ** -89                                      # y 20 steps
        out = fpq.rmsnorm_quantize(x, w, fpq.FP8_1x128, residual=residual)
        q, s = out.q.cpu(), out.scales.cpu()
        assert s[0].tolist()[:2] == [1.0, 1.0] and torch.all(q[0, :256] & 0x7F == 0) and q[0, 300] == 0x7E
        assert torch.all(torch.isnan(s[1])) and torch.all(q[1] & 0x7F == 0x7F)
