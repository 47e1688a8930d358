"""Few bf16 rows times NVFP4 weights on the GPU, dense and by expert, against
the product of the decoded values in 64 bits.

Tolerance.  Weights are decoded exactly; the sums are fp32.  A tensor core
may truncate where it adds: k / 16 products of 16 in a row, each within 2^-22
of the sum of magnitudes, and under 64 further additions.  The output type
adds half a step (bf16 2^-8, fp32 2^-24).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _decode(wq, ws, wg):
    table = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device=wq.device)
    codes = torch.stack([wq & 15, wq >> 4], -1).flatten(-2).long()
    s = ws.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    return table[codes] * s * wg.double().view(-1, *([1] * (wq.dim() - 1)))


def _inside(y, x, w, out_dtype):
    """x [..., k], w [..., n, k] in 64 bits; y [..., n]."""
    want = torch.einsum("...k,...nk->...n", x, w)
    size = torch.einsum("...k,...nk->...n", x.abs(), w.abs())
    tol = STEP[out_dtype] * want.abs() + (x.shape[-1] / 16 + 64) * 2.0 ** -22 * size
    over = (y.double() - want).abs() - tol
    assert over.max().item() <= 0, over.max().item()


def _weights(fpq, shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return fpq.quantize((torch.randn(shape, generator=g, device="cuda") * 0.02).to(torch.bfloat16), fpq.NVFP4)


def _x(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("n,k", [(1, 32), (7, 64), (16, 96), (33, 544), (128, 512), (100, 2048), (2048, 7168),
                                 (5001, 1056), (40, 16384), (300, 14336), (20011, 544)])
@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 16])
def test_dense(fpq, n, k, m):
    wq, ws, wg = _weights(fpq, (n, k), n + k)
    x = _x((m, k), m)
    w = _decode(wq, ws, wg)
    for dtype in (torch.float32, torch.bfloat16):
        y = fpq.gemv_nvfp4(x, wq, ws, wg, out_dtype=dtype)
        assert y.shape == (m, n) and y.dtype == dtype
        _inside(y, x.double(), w[None], dtype)
    assert torch.equal(y, fpq.gemv_nvfp4(x, wq, ws, wg))
    assert fpq.fpq_get_device_error() == 0


@pytest.mark.parametrize("m", [1, 5, 16])
def test_every_code_and_scale(fpq, m):
    """All 16 codes with all 256 scale bytes (the NaN ones apart): exact
    products against one-hot rows."""
    n, k = 256, 256
    codes = torch.arange(16, dtype=torch.uint8, device="cuda").repeat(n, k // 16)
    wq = codes[:, 0::2] | (codes[:, 1::2] << 4)
    ws = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].expand(n, k // 16).to(torch.uint8).contiguous()
    ws[(ws & 0x7F) == 0x7F] = 0
    wg = torch.tensor([0.37], device="cuda")
    w = (_decode(wq, ws, torch.ones(1, device="cuda")).float() * wg).double()
    for first in range(0, k, m):
        x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
        for i in range(min(m, k - first)):
            x[i, first + i] = 1
        y = fpq.gemv_nvfp4(x, wq, ws, wg, out_dtype=torch.float32)
        for i in range(min(m, k - first)):
            assert torch.equal(y[i].double(), w[:, first + i])


def test_nan_scale_and_infinities_stay_in_their_rows(fpq):
    wq, ws, wg = _weights(fpq, (40, 256), 1)
    x = _x((3, 256), 2)
    clean = fpq.gemv_nvfp4(x, wq, ws, wg)
    ws2, x2 = ws.clone(), x.clone()
    ws2[17, 3] = 0x7F
    x2[1, 100] = float("inf")
    y = fpq.gemv_nvfp4(x2, wq, ws2, wg)
    assert torch.all(torch.isnan(y[:, 17]))
    keep = torch.arange(40, device="cuda") != 17
    assert torch.equal(y[0][keep], clean[0][keep]) and torch.equal(y[2][keep], clean[2][keep])
    assert not torch.isfinite(y[1]).any()
    # huge and tiny activations: a power of two passes through the product
    big = fpq.gemv_nvfp4((x.float() * 2.0 ** 100).to(torch.bfloat16), wq, ws, wg, out_dtype=torch.float32)
    small = fpq.gemv_nvfp4((x.float() * 2.0 ** -90).to(torch.bfloat16), wq, ws, wg, out_dtype=torch.float32)
    plain = fpq.gemv_nvfp4(x, wq, ws, wg, out_dtype=torch.float32)
    assert torch.equal(big, plain * 2.0 ** 100) and torch.equal(small, plain * 2.0 ** -90)


def test_a_row_does_not_depend_on_the_others(fpq):
    wq, ws, wg = _weights(fpq, (77, 1056), 4)
    x = _x((16, 1056), 5)
    all_ = fpq.gemv_nvfp4(x, wq, ws, wg, out_dtype=torch.float32)
    for m in (1, 3, 8, 11):
        assert torch.equal(fpq.gemv_nvfp4(x[:m], wq, ws, wg, out_dtype=torch.float32), all_[:m])
    assert torch.equal(fpq.gemv_nvfp4(x[5:6], wq, ws, wg, out_dtype=torch.float32), all_[5:6])


@pytest.mark.parametrize("tokens,topk,experts,n,k", [(1, 1, 1, 16, 32), (1, 8, 64, 256, 512), (8, 8, 64, 100, 1056),
                                                     (3, 2, 4, 33, 96), (30, 8, 16, 64, 256), (32, 32, 128, 24, 64),
                                                     (1, 4, 8, 2048, 7168), (1024, 1, 3, 17, 128)])
def test_experts(fpq, tokens, topk, experts, n, k):
    wq, ws, wg = _weights(fpq, (experts, n, k), tokens + n)
    g = torch.Generator().manual_seed(tokens)
    ids = torch.stack([torch.randperm(experts, generator=g).repeat(32)[:topk] for _ in range(tokens)]).int().cuda()
    w = _decode(wq, ws, wg)
    for x in (_x((tokens, k), 1), _x((tokens, topk, k), 2)):
        for dtype in (torch.bfloat16, torch.float32):
            y = fpq.gemv_nvfp4(x, wq, ws, wg, ids=ids, out_dtype=dtype)
            assert y.shape == (tokens, topk, n) and y.dtype == dtype
            xs = x.double() if x.dim() == 3 else x.double()[:, None].expand(-1, topk, -1)
            for t0 in range(0, tokens, 64):
                _inside(y[t0:t0 + 64], xs[t0:t0 + 64], w[ids[t0:t0 + 64].long()], dtype)
    assert torch.equal(y, fpq.gemv_nvfp4(x, wq, ws, wg, ids=ids, out_dtype=dtype))
    assert fpq.fpq_get_device_error() == 0


def test_expert_rows_are_those_of_the_dense_form(fpq):
    wq, ws, wg = _weights(fpq, (5, 64, 544), 6)
    x = _x((12, 544), 7)
    ids = torch.randint(0, 5, (12, 3), generator=torch.Generator().manual_seed(1)).int().cuda()
    y = fpq.gemv_nvfp4(x, wq, ws, wg, ids=ids, out_dtype=torch.float32)
    for e in range(5):
        dense = fpq.gemv_nvfp4(x, wq[e], ws[e], wg[e:e + 1].clone(), out_dtype=torch.float32)
        t, j = (ids == e).nonzero(as_tuple=True)
        assert torch.equal(y[t, j], dense[t])


def test_expert_ids_out_of_range(fpq):
    wq, ws, wg = _weights(fpq, (4, 48, 128), 8)
    x = _x((3, 128), 9)
    good = torch.tensor([[0, 1], [2, 3], [1, 1]], dtype=torch.int32, device="cuda")
    want = fpq.gemv_nvfp4(x, wq, ws, wg, ids=good)
    for value in (4, -1, 2 ** 31 - 1, -2 ** 31):
        ids = good.clone()
        ids[1, 0] = value
        y = fpq.gemv_nvfp4(x, wq, ws, wg, ids=ids)
        assert fpq.fpq_get_device_error() == 6
        assert torch.all(y[1, 0] == 0)
        y[1, 0] = want[1, 0]
        assert torch.equal(y, want)


def test_results_stay_inside_their_buffer(fpq):
    wq, ws, wg = _weights(fpq, (4, 37, 96), 10)
    x = _x((4, 96), 11)
    y = torch.full((4 * 2 * 37 + 64,), 5.0, device="cuda")
    ids = torch.tensor([[0, 3]] * 4, dtype=torch.int32, device="cuda")
    fpq.fpq_moe_gemv_nvfp4(x, 0, ids, 4, 2, 4, wq, ws, wg, 37, 96, y, fpq.OUT_F32)
    assert torch.equal(y[:-64].view(4, 2, 37), fpq.gemv_nvfp4(x, wq, ws, wg, ids=ids, out_dtype=torch.float32))
    assert torch.all(y[-64:] == 5.0)
    y.fill_(5.0)
    fpq.fpq_gemv_nvfp4(x, 4, wq[0], ws[0], wg, 37, 96, y, fpq.OUT_F32)
    assert torch.all(y[4 * 37:] == 5.0)


def test_no_rows(fpq):
    wq, ws, wg = _weights(fpq, (2, 16, 32), 12)
    x = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    assert fpq.gemv_nvfp4(x, wq[0], ws[0], wg[:1]).shape == (0, 16)
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    assert fpq.gemv_nvfp4(x, wq, ws, wg, ids=ids).shape == (0, 2, 16)


def test_far_experts(fpq):
    """Codes and scales past 2^32 bytes from the first."""
    experts, n, k = 640, 2048, 7168
    wq = torch.empty((experts, n, k // 2), dtype=torch.uint8, device="cuda")
    ws = torch.empty((experts, n, k // 16), dtype=torch.uint8, device="cuda")
    wg = torch.ones((experts,), device="cuda")
    assert wq.numel() > 2 ** 32
    used = [0, 584, 585, 586, experts - 1]                   # 2^32 bytes of codes end inside expert 585
    for e in used:
        q, s, g = _weights(fpq, (n, k), e)
        wq[e], ws[e], wg[e] = q, s, g[0]
    x = _x((1, k), 3)
    ids = torch.tensor([used], dtype=torch.int32, device="cuda")
    y = fpq.gemv_nvfp4(x, wq, ws, wg, ids=ids, out_dtype=torch.float32)
    for j, e in enumerate(used):
        _inside(y[:, j], x.double(), _decode(wq[e], ws[e], wg[e:e + 1])[None], torch.float32)


@pytest.mark.parametrize("tokens,topk,experts", [(1, 8, 4), (1, 32, 2), (2, 5, 3), (3, 32, 1), (33, 31, 2), (5, 8, 40)])
def test_experts_named_several_times(fpq, tokens, topk, experts):
    """A token that names an expert more than once, and every pair naming one."""
    wq, ws, wg = _weights(fpq, (experts, 40, 160), 14)
    x = _x((tokens, topk, 160), 15)
    w = _decode(wq, ws, wg)
    g = torch.Generator().manual_seed(16)
    for ids in (torch.zeros((tokens, topk)), torch.full((tokens, topk), experts - 1),
                torch.randint(0, min(experts, 3), (tokens, topk), generator=g)):
        ids = ids.int().cuda()
        y = fpq.gemv_nvfp4(x, wq, ws, wg, ids=ids, out_dtype=torch.float32)
        _inside(y, x.double(), w[ids.long()], torch.float32)


@pytest.mark.parametrize("m", [1, 9])
def test_small_elements_beside_a_large_one(fpq, m):
    """x is exact down to 2^-31 of the largest of its 128 columns, and within
    2^-39 of that below: a 1 under zero weights, and small elements with all
    their eight bits under the others."""
    n, k = 32, 256
    wq = torch.full((n, k // 2), 0x22, dtype=torch.uint8, device="cuda")               # ones
    wq[:, 0] = 0x20                                                                    # 0 at column 0
    ws = torch.full((n, k // 16), 0x38, dtype=torch.uint8, device="cuda")              # 1
    wg = torch.ones((1,), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(m)
    for top in (1.0, 1.9921875):
        for power in range(24, 48):
            x = torch.zeros((m, k), device="cuda")
            x[:, 0] = top
            at = 1 + torch.randint(0, 127, (m,), generator=g, device="cuda")
            small = (1 + torch.randint(0, 128, (m,), generator=g, device="cuda") / 128) * 2.0 ** -power
            x[torch.arange(m, device="cuda"), at] = small
            x = x.to(torch.bfloat16)
            y = fpq.gemv_nvfp4(x, wq, ws, wg, out_dtype=torch.float32)
            err = (y.double() - small.double()[:, None]).abs()
            assert torch.all(err <= (2.0 ** -39 * top if power > 31 else 0)), (top, power, err.max().item())
