"""The combination of the experts' rows, its backward pass and the row map on
the GPU.

Tolerances.  out is a chain of at most 33 fp32 fused multiply-adds, each
within 2^-24 of the sum of magnitudes; a dweight a chain of under 200; dy one
product.  An output type adds half a step (bf16 2^-8, fp32 2^-24).
"""
import numpy as np
import pytest
import torch

import workloads
from mxfp8_block_scaled_warp_b200 import moe

pytestmark = pytest.mark.gpu

STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _case(tokens, topk, hidden, seed, y_dtype, extra=0):
    g = torch.Generator().manual_seed(seed)
    y = torch.randn((tokens * topk + extra, hidden), generator=g).to(y_dtype).cuda()
    rows = torch.randperm(tokens * topk + extra, generator=g)[:tokens * topk].view(tokens, topk).int().cuda()
    w = torch.rand((tokens, topk), generator=g).cuda()
    add = torch.randn((tokens, hidden), generator=g).to(torch.bfloat16).cuda()
    return y, rows, w, add


def _inside(got, want, size, adds, dtype):
    over = (got.double() - want).abs() - STEP[dtype] * want.abs() * (1 + 2.0 ** -8) - adds * 2.0 ** -24 * size
    assert over.numel() == 0 or over.max().item() <= 0, over.max().item()


@pytest.mark.parametrize("tokens,topk,hidden", [(1, 1, 8), (1, 8, 7168), (5, 3, 40), (33, 8, 2048), (7, 9, 2056),
                                                (3, 32, 264), (200, 2, 136), (2, 4, 16392),
                                                (2400, 2, 72), (2401, 3, 552), (2500, 11, 136)])
@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_forward_and_backward(fpq, tokens, topk, hidden, y_dtype, out_dtype):
    y, rows, w, add = _case(tokens, topk, hidden, tokens + hidden, y_dtype, extra=3)
    picked = y.double()[rows.long()]
    for a in (None, add):
        out = moe.combine(y, w, rows=rows, add=a, out_dtype=out_dtype)
        want = (picked * w.double()[..., None]).sum(1) + (0 if a is None else a.double())
        size = (picked * w.double()[..., None]).abs().sum(1) + (0 if a is None else a.double().abs())
        _inside(out, want, size, topk + 1, out_dtype)
    dout = torch.randn((tokens, hidden), generator=torch.Generator().manual_seed(1)).to(out_dtype).cuda()
    dy0 = torch.full_like(y, 7.0)
    dy, dw = moe.combine_backward(dout, y, w, rows=rows, dy=dy0)
    assert dy is dy0
    d = dout.double()[:, None, :]
    _inside(dw, (picked * d).sum(-1), (picked * d).abs().sum(-1), 200, torch.float32)
    want = w.double()[..., None] * d
    _inside(dy[rows.long()], want, want.abs(), 1, y_dtype)
    left = torch.ones(y.shape[0], dtype=torch.bool, device="cuda")
    left[rows.flatten().long()] = False
    assert left.sum() == 3 and torch.all(dy[left] == 7.0)
    again = moe.combine_backward(dout, y, w, rows=rows)
    assert torch.equal(again[1], dw) and torch.equal(again[0][~left], dy[~left])
    assert fpq.fpq_get_device_error() == 0


def test_without_a_row_map(fpq):
    y, _, w, add = _case(6, 5, 72, 3, torch.bfloat16)
    rows = torch.arange(30, dtype=torch.int32, device="cuda").view(6, 5)
    dout = torch.randn((6, 72), device="cuda").to(torch.bfloat16)
    want = moe.combine(y, w, rows=rows, add=add)
    assert torch.equal(moe.combine(y, w, add=add), want)
    assert torch.equal(moe.combine(y.view(6, 5, 72), w, add=add), want)
    a, b = moe.combine_backward(dout, y, w, rows=rows), moe.combine_backward(dout, y.view(6, 5, 72), w)
    assert torch.equal(a[0], b[0].view(30, 72)) and torch.equal(a[1], b[1])


def test_dropped_and_bad_rows(fpq):
    """-1 drops a pair, all pairs of a token included; a row outside the buffer
    is dropped and reported; a NaN in a row that no pair names is not seen."""
    y, rows, w, add = _case(4, 3, 264, 5, torch.bfloat16, extra=2)
    dout = torch.randn((4, 264), device="cuda").to(torch.bfloat16)
    rows[1, 2] = -1
    rows[2] = -1
    named = torch.zeros(y.shape[0], dtype=torch.bool, device="cuda")
    named[rows[rows >= 0].long()] = True
    y[~named] = float("nan")
    out = moe.combine(y, w, rows=rows, add=add)
    dy, dw = moe.combine_backward(dout, y, w, rows=rows, dy=torch.zeros_like(y))
    assert fpq.fpq_get_device_error() == 0
    assert torch.equal(out[2], add[2]) and torch.all(torch.isfinite(out)) and torch.all(dw[2] == 0)
    assert dw[1, 2] == 0 and torch.all(dy[~named] == 0)
    bad = rows.clone()
    for value in (y.shape[0], -2, 2 ** 31 - 1, -2 ** 31):
        bad[1, 2] = value
        assert torch.equal(moe.combine(y, w, rows=bad, add=add), out)
        assert fpq.fpq_get_device_error() == 6
        _, dw_bad = moe.combine_backward(dout, y, w, rows=bad, dy=torch.zeros_like(y))
        assert torch.equal(dw_bad, dw)
        assert fpq.fpq_get_device_error() == 6


def test_backward_against_differences(fpq):
    y, rows, w, add = _case(3, 4, 64, 9, torch.float32)
    dout = torch.randn((3, 64), device="cuda")
    dy, dw = moe.combine_backward(dout, y, w, rows=rows)
    u, v = torch.randn_like(y), torch.randn_like(w)
    f = lambda a, b: ((a[rows.long()] * b[..., None]).sum(1) * dout.double()).sum()       # noqa: E731
    h = 1e-4
    slope = (f(y.double() + h * u, w.double() + h * v) - f(y.double() - h * u, w.double() - h * v)) / (2 * h)
    got = (dy.double() * u).sum() + (dw.double() * v).sum()
    # f is bilinear: the central difference is exact; fp32 gradients
    assert abs(got - slope) <= 200 * 2.0 ** -24 * ((dy.double() * u).abs().sum() + (dw.double() * v).abs().sum()) + 1e-7


@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (7, 8, 3), (5000, 16, 4), (9500, 64, 8), (300, 256, 6),
                                              (50, 64, 32), (200, 1024, 4)])
def test_pair_rows(fpq, orc, tokens, experts, k):
    """The map names the row that the dispatch wrote: expert offset plus the
    pair's slot."""
    ids = workloads.route_choices(tokens, experts, k, seed=tokens)
    x = workloads.normal_bf16((tokens, 32), 1.0, seed=1).cuda()
    rows = torch.empty((tokens, k), dtype=torch.int32, device="cuda")
    d = moe.dispatch(x, ids.cuda(), experts, rows=rows)
    counts, slot = orc.moe_route_plan(ids.numpy(), experts)
    first = np.concatenate([[0], np.cumsum(counts)])[:-1]
    assert np.array_equal(rows.cpu().numpy(), first[ids.numpy()] + slot)
    plain = moe.dispatch(x, ids.cuda(), experts)
    assert torch.equal(plain.codes, d.codes) and torch.equal(plain.scales, d.scales)


def test_pair_rows_of_bad_ids(fpq):
    ids = torch.tensor([[0, 4], [3, -1], [3, 0]], dtype=torch.int32, device="cuda")
    x = torch.ones((3, 32), dtype=torch.bfloat16, device="cuda")
    rows = torch.full((3, 2), 99, dtype=torch.int32, device="cuda")
    moe.dispatch(x, ids, 4, rows=rows)
    assert fpq.fpq_get_device_error() == 6
    assert rows.tolist() == [[0, -1], [2, -1], [3, 1]]


def test_no_tokens(fpq):
    y = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.empty((0, 4), device="cuda")
    assert moe.combine(y, w).shape == (0, 64)
    dy, dw = moe.combine_backward(y, y, w)
    assert dy.shape == (0, 64) and dw.shape == (0, 4)


def test_far_rows(fpq):
    """Rows past 2^31 elements from the first."""
    hidden, y_rows = 7168, 310000
    y = torch.zeros((y_rows, hidden), dtype=torch.bfloat16, device="cuda")
    y[-8:] = torch.randn((8, hidden), device="cuda").to(torch.bfloat16)
    rows = torch.arange(y_rows - 8, y_rows, dtype=torch.int32, device="cuda").view(2, 4)
    w = torch.rand((2, 4), device="cuda")
    near = y[-8:].clone()
    assert torch.equal(moe.combine(y, w, rows=rows), moe.combine(near, w))
    dout = torch.randn((2, hidden), device="cuda").to(torch.bfloat16)
    dy, dw = moe.combine_backward(dout, y, w, rows=rows)
    dy_near, dw_near = moe.combine_backward(dout, near, w)
    assert torch.equal(dy[-8:], dy_near) and torch.equal(dw, dw_near)


def test_many_tokens_without_a_row_map(fpq):
    y, _, w, add = _case(2600, 8, 64, 13, torch.bfloat16)
    rows = torch.arange(2600 * 8, dtype=torch.int32, device="cuda").view(2600, 8)
    rows[5, 3] = -1
    rows[2599] = -1
    dout = torch.randn((2600, 64), device="cuda").to(torch.bfloat16)
    dy, dw = moe.combine_backward(dout, y, w, rows=rows, dy=torch.zeros_like(y))
    full_dy, full_dw = moe.combine_backward(dout, y, w)
    keep = (rows >= 0)
    assert torch.equal(dw[keep], full_dw[keep]) and torch.all(dw[~keep] == 0)
    assert torch.equal(dy.view(2600, 8, 64)[keep], full_dy.view(2600, 8, 64)[keep])
    assert torch.all(dy.view(2600, 8, 64)[~keep] == 0)


@pytest.mark.parametrize("tokens,topk,hidden", [(4, 3, 264), (2600, 2, 72), (300, 8, 2048)])
@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
def test_rows_that_no_pair_names_have_no_gradient(fpq, tokens, topk, hidden, y_dtype):
    """A new buffer holds zeros there, whatever its memory held before."""
    y, rows, w, _ = _case(tokens, topk, hidden, 17, y_dtype, extra=70)
    rows[1, 0] = -1
    rows[tokens - 1] = -1
    named = torch.zeros(y.shape[0], dtype=torch.bool, device="cuda")
    named[rows[rows >= 0].long()] = True
    dout = torch.randn((tokens, hidden), device="cuda").to(torch.bfloat16)
    want, want_w = moe.combine_backward(dout, y, w, rows=rows, dy=torch.zeros_like(y))
    for _ in range(3):
        used = [torch.full_like(y, float("nan")) for _ in range(3)]
        used += [torch.zeros((y.shape[0],), dtype=torch.int32, device="cuda")]
        del used
        dy, dw = moe.combine_backward(dout, y, w, rows=rows)
        assert torch.equal(dy, want) and torch.equal(dw, want_w)
    assert torch.all(dy[~named] == 0)
    # without a map the first tokens * topk rows are named
    used = [torch.full_like(y, float("nan")) for _ in range(3)]
    del used
    dy, _ = moe.combine_backward(dout, y, w)
    assert torch.all(torch.isfinite(dy)) and torch.all(dy[tokens * topk:] == 0)
    assert torch.all(moe.combine_backward(dout, y, w, rows=torch.full_like(rows, -1))[0] == 0)
    assert fpq.fpq_get_device_error() == 0


def test_no_tokens_but_rows(fpq):
    y = torch.ones((40, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.empty((0, 4), device="cuda")
    used = [torch.full_like(y, float("nan")) for _ in range(3)]
    del used
    for rows in (None, torch.empty((0, 4), dtype=torch.int32, device="cuda")):
        dy, dw = moe.combine_backward(y[:0], y, w, rows=rows)
        assert torch.all(dy == 0) and dw.shape == (0, 4)


def test_every_row_written_from_any_workspace(fpq):
    """The C entry with a workspace that held the owners of another map, whose
    pairs name other rows now."""
    y, rows, w, _ = _case(50, 4, 64, 19, torch.bfloat16, extra=30)
    dout = torch.randn((50, 64), device="cuda").to(torch.bfloat16)
    ws = torch.empty((y.shape[0] + 4,), dtype=torch.int32, device="cuda")
    ws[-4:] = 9
    dw = torch.empty_like(w)
    for turn in range(3):
        rows = (rows + 17) % y.shape[0]                          # each row still named once
        named, rows = rows, rows.clone()
        rows[turn, 1] = -1
        dy = torch.full_like(y, float("nan"))
        fpq.fpq_moe_combine_backward_full(dout, 0, y, 0, y.shape[0], rows, w, 50, 4, 64, dy, dw, ws)
        want, want_w = moe.combine_backward(dout, y, w, rows=rows, dy=torch.zeros_like(y))
        assert torch.equal(dy, want) and torch.equal(dw, want_w) and torch.all(ws[-4:] == 9)
        rows = named


def test_backward_with_a_row_map_captured(fpq):
    """Replayed with other maps and dropped pairs; the gradient and its zeros follow."""
    y, rows, w, _ = _case(120, 4, 264, 23, torch.bfloat16, extra=60)
    dout = torch.randn((120, 264), device="cuda").to(torch.bfloat16)
    moe.combine_backward(dout, y, w, rows=rows)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dy, dw = moe.combine_backward(dout, y, w, rows=rows)
    for turn in range(4):
        other = torch.randperm(y.shape[0], generator=torch.Generator().manual_seed(turn))[:480].view(120, 4).int().cuda()
        other[turn::7, turn] = -1
        rows.copy_(other)
        dy.fill_(float("nan"))
        g.replay()
        want, want_w = moe.combine_backward(dout, y, w, rows=rows, dy=torch.zeros_like(y))
        assert torch.equal(dy, want) and torch.equal(dw, want_w)
