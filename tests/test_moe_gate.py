"""The expert gate and its backward pass on the GPU, against the definition in
64 bits: the choice greedily, one expert after the other, the lowest index
among equal keys; the weights and gradients by autograd in 64 bits.

Tolerances.  An fp32 score is within 2^-17 of its value, relative: exp and
the divisions within a few units of 2^-24, the difference from the row's
maximum within 2^-24 of at most 40 (smaller scores are below 2^-57 of the
sum), the sum's additions at most 37.  Gradients count against the sums of
magnitudes, with 2^-15 for products of up to four such factors; a bf16
output adds half a step, 2^-8.
"""
import math

import pytest
import torch

from mxfp8_block_scaled_warp_b200 import moe

pytestmark = pytest.mark.gpu


def _scores(lg, score):
    if score == moe.SIGMOID:
        return 1 / (1 + torch.exp(-lg))
    m = lg.max(1, keepdim=True).values
    e = torch.where(lg == -math.inf, torch.zeros_like(lg), torch.exp(lg - m))
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, torch.zeros_like(e))


def _definition(logits, topk, bias, score, n_group, topk_group, group_top, renormalize, scale):
    lg = logits.double()
    p = _scores(lg, score)
    key = lg if bias is None else p + bias.double()
    t, e = key.shape
    if n_group > 1:
        per = (p if bias is None else key).view(t, n_group, e // n_group)
        rank = per.topk(group_top, 2).values.sum(2)
        order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :topk_group]
        keep = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, order, True).repeat_interleave(e // n_group, 1)
    else:
        keep = torch.ones_like(key, dtype=torch.bool)
    # descending key, then index; experts outside the groups behind all others
    by_key = torch.sort(key, dim=1, descending=True, stable=True).indices
    kept_first = torch.sort(keep.gather(1, by_key).int(), dim=1, descending=True, stable=True).indices
    ids = by_key.gather(1, kept_first)[:, :topk]
    w = p.gather(1, ids)
    if renormalize:
        if score == moe.SOFTMAX:
            w = _scores(lg.gather(1, ids), score)
        else:
            total = w.sum(1, keepdim=True)
            w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return ids, w * scale


def _check(logits, topk, bias=None, score=moe.SOFTMAX, n_group=1, topk_group=1, group_top=1, renormalize=True,
           scale=1.0):
    ids, w = moe.gate(logits, topk, bias=bias, score=score, n_group=n_group, topk_group=topk_group,
                      group_top=group_top, renormalize=renormalize, scale=scale)
    want_ids, want = _definition(logits, topk, bias, score, n_group, topk_group, group_top, renormalize, scale)
    assert torch.equal(ids.long(), want_ids)
    over = (w.double() - want).abs() - 2.0 ** -17 * want.abs() - 1e-37
    assert over.max().item() <= 0
    return ids, w


def _logits(tokens, experts, seed, dtype=torch.float32, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((tokens, experts), generator=g) * std).to(dtype).cuda()


def _bias(experts, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(-50, 51, (experts,), generator=g).float() * 0.001).cuda()


@pytest.mark.parametrize("tokens,experts,topk", [(1, 1, 1), (1, 8, 2), (3, 8, 8), (33, 40, 6), (257, 64, 8),
                                                 (9, 100, 32), (1000, 256, 8), (130, 384, 6), (65, 1000, 10),
                                                 (17, 1024, 32)])
@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bias", [False, True])
def test_choice_and_weights(fpq, tokens, experts, topk, score, dtype, bias):
    lg = _logits(tokens, experts, tokens + experts, dtype)
    b = _bias(experts, experts) if bias else None
    for renormalize in (False, True):
        _check(lg, topk, b, score, renormalize=renormalize, scale=2.5)
    assert fpq.fpq_get_device_error() == 0


@pytest.mark.parametrize("experts,n_group,topk_group,topk", [(256, 8, 4, 8), (64, 8, 3, 6), (160, 8, 3, 6),
                                                             (64, 32, 5, 10), (1024, 4, 2, 32), (12, 3, 1, 4),
                                                             (24, 2, 2, 20)])
@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("bias", [False, True])
def test_groups(fpq, experts, n_group, topk_group, topk, score, group_top, bias):
    b = _bias(experts, experts) if bias else None
    for dtype in (torch.float32, torch.bfloat16):
        _check(_logits(333, experts, experts + topk, dtype), topk, b, score, n_group, topk_group, group_top)


@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("grouped", [False, True])
def test_ties_and_near_ties(fpq, score, grouped):
    """Logits of a few values only, a bias that makes different scores almost
    or exactly equal, saturated scores: the lowest index among equals, and
    the larger in exact arithmetic where fp32 cannot tell."""
    groups = dict(n_group=8, topk_group=3, group_top=2) if grouped else {}
    g = torch.Generator().manual_seed(5)
    few = torch.randint(-2, 3, (500, 64), generator=g).float().cuda()
    _check(few, 8, score=score, **groups)
    _check(few, 8, torch.zeros(64, device="cuda"), score, **groups)
    _check(few, 8, _bias(64, 1), score, **groups)
    _check(torch.zeros((5, 64), device="cuda"), 8, score=score, **groups)
    # scores that differ by less than an fp32 step at the sum with the bias
    base = torch.rand((400, 1), generator=g).cuda()
    close = base + torch.randint(0, 40, (400, 64), generator=g).cuda() * 2.0 ** -24
    _check(close, 8, torch.full((64,), 0.25, device="cuda"), score, **groups)
    _check(close, 8, _bias(64, 2) * 1e-5, score, **groups)
    _check(18 + close, 8, torch.zeros(64, device="cuda"), score, **groups)           # near 1 - 1e-8
    _check(torch.where(few > 0, 0.0, -0.0), 8, score=score, **groups)                # zeros of both signs


@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("bias", [False, True])
def test_masked_experts(fpq, score, bias):
    """-inf logits: never before another expert, weight 0, a whole row of them
    included; the type's lowest value is an ordinary logit."""
    b = _bias(64, 3).abs() if bias else None
    lg = _logits(200, 64, 9)
    g = torch.Generator().manual_seed(6)
    lg[torch.rand((200, 64), generator=g).cuda() < 0.6] = -math.inf
    lg[0] = -math.inf
    lg[1, 3:] = -math.inf
    lg[2] = torch.finfo(torch.float32).min
    for renormalize in (False, True):
        ids, w = moe.gate(lg, 8, bias=b, score=score, renormalize=renormalize)
        _, want = _definition(lg, 8, b, score, 1, 1, 1, renormalize, 1.0)
        assert torch.all((ids >= 0) & (ids < 64))
        assert torch.all(ids.sort(1).values.diff(dim=1) > 0)                         # distinct
        got = lg.gather(1, ids.long())
        assert torch.all(w[got == -math.inf] == 0) and torch.all(torch.isfinite(w))
        if b is None:
            assert torch.all((w.double() - want).abs() <= 2.0 ** -17 * want.abs())
            assert torch.equal(ids[0], torch.arange(8, device="cuda", dtype=torch.int32))
            assert torch.equal(ids[1, :3].sort().values, torch.arange(3, device="cuda", dtype=torch.int32))


@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("kw", [dict(), dict(n_group=4, topk_group=2, group_top=2)])
def test_not_a_number(fpq, score, kw):
    """NaN and +inf logits: valid, distinct ids, and the other rows untouched."""
    lg = _logits(6, 32, 4)
    clean = moe.gate(lg, 4, bias=_bias(32, 4), score=score, **kw)
    bad = lg.clone()
    bad[1, 3] = float("nan")
    bad[2] = float("nan")
    bad[3, 9] = float("inf")
    for b in (None, _bias(32, 4)):
        ids, w = moe.gate(bad, 4, bias=b, score=score, **kw)
        assert torch.all((ids >= 0) & (ids < 32)) and torch.all(ids.sort(1).values.diff(dim=1) > 0)
        if b is not None:
            for u, v in zip((ids, w), clean):
                assert torch.equal(u[[0, 4, 5]], v[[0, 4, 5]])
        elif not kw:
            assert not (ids[1] == 3).any() and ids[3, 0] == 9


@pytest.mark.parametrize("tokens,experts,topk", [(1, 1, 1), (1, 8, 8), (40, 40, 6), (333, 64, 8), (65, 100, 32),
                                                 (500, 256, 8), (33, 1023, 5), (17, 1024, 32)])
@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [False, True])
def test_backward(fpq, tokens, experts, topk, score, dtype, renormalize):
    lg = _logits(tokens, experts, tokens + 2 * experts, dtype)
    ids, _ = moe.gate(lg, topk, score=score, renormalize=renormalize)
    dw = torch.randn((tokens, topk), generator=torch.Generator().manual_seed(8)).cuda()
    d = moe.gate_backward(dw, lg, ids, score=score, renormalize=renormalize, scale=2.5)
    x = lg.double().requires_grad_(True)
    p = _scores(x, score).gather(1, ids.long())
    if renormalize and score == moe.SOFTMAX:
        # the same as p over its sum; written so that an expert that was not
        # chosen has a gradient of exactly 0 in 64 bits too
        w = 2.5 * _scores(x.gather(1, ids.long()), score)
    else:
        w = 2.5 * (p / p.sum(1, keepdim=True) if renormalize else p)
    (w * dw.double()).sum().backward()
    full = _scores(lg.double(), score)
    chosen = torch.zeros_like(full).scatter_(1, ids.long(), 1.0)
    # magnitudes of the terms that cancel: each chosen weight's own and the row's mean
    size = 2.5 * full * (dw.double().abs().max(1, keepdim=True).values) * 2
    if renormalize:
        size = size * chosen / p.sum(1, keepdim=True).detach()
    rel = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    over = (d.double() - x.grad).abs() - rel * x.grad.abs() - 2.0 ** -15 * size - 1e-37
    assert over.max().item() <= 0
    if renormalize or score == moe.SIGMOID:
        assert torch.all(d[chosen == 0] == 0)


def test_backward_against_differences(fpq):
    lg = _logits(6, 32, 31)
    dw = torch.randn((6, 4), device="cuda")
    for score in (moe.SOFTMAX, moe.SIGMOID):
        for renormalize in (False, True):
            ids, _ = moe.gate(lg, 4, score=score, renormalize=renormalize)
            d = moe.gate_backward(dw, lg, ids, score=score, renormalize=renormalize)

            def f(x):
                p = _scores(x, score).gather(1, ids.long())
                return ((p / p.sum(1, keepdim=True) if renormalize else p) * dw.double()).sum()

            u = torch.randn(lg.shape, device="cuda", dtype=torch.float64)
            h = 1e-5
            slope = (f(lg.double() + h * u) - f(lg.double() - h * u)) / (2 * h)
            # fp32 gradient: 2^-15 of the terms; the difference's h^2 times third derivatives of order one
            assert abs((d.double() * u).sum() - slope) <= 2.0 ** -13 * (d.double() * u).abs().sum() + 1e-6


def test_backward_edges(fpq):
    """A masked row has a zero gradient; an id out of range is dropped and
    reported; an id named twice gets the sum."""
    lg = _logits(4, 16, 2)
    lg[1] = -math.inf
    ids = torch.tensor([[1, 2], [0, 1], [5, 16], [7, 7]], dtype=torch.int32, device="cuda")
    dw = torch.ones((4, 2), device="cuda")
    d = moe.gate_backward(dw, lg, ids, score=moe.SIGMOID, renormalize=False)
    assert fpq.fpq_get_device_error() == 6
    p = _scores(lg.double(), moe.SIGMOID)
    want = torch.zeros((4, 16), dtype=torch.float64, device="cuda")
    for t, e in ((0, 1), (0, 2), (2, 5), (3, 7), (3, 7)):
        want[t, e] += p[t, e] * (1 - p[t, e])
    assert torch.all((d.double() - want).abs() <= 2.0 ** -17 * want)
    for score in (moe.SOFTMAX, moe.SIGMOID):
        for renormalize in (False, True):
            d = moe.gate_backward(dw, lg, ids.clamp(max=15), score=score, renormalize=renormalize)
            assert torch.all(d[1] == 0)
    assert fpq.fpq_get_device_error() == 0


def test_no_tokens(fpq):
    lg = torch.empty((0, 64), device="cuda")
    ids, w = moe.gate(lg, 8)
    assert ids.shape == w.shape == (0, 8)
    assert moe.gate_backward(w, lg, ids).shape == (0, 64)


@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("grouped", [False, True])
def test_masked_experts_do_not_gain_by_their_bias(fpq, score, grouped):
    """With a bias, too, a -inf logit is chosen after every other expert."""
    lg = _logits(120, 64, 21)
    g = torch.Generator().manual_seed(22)
    lg[torch.rand((120, 64), generator=g).cuda() < 0.5] = -math.inf
    lg[0, 3:] = -math.inf
    lg[1, 1:] = -math.inf
    lg[2] = -math.inf
    bias = torch.where(torch.arange(64, device="cuda") % 3 == 0, 2.0, -0.5)
    kw = dict(n_group=4, topk_group=2, group_top=2) if grouped else {}
    for topk in (1, 6, 32):
        ids, w = moe.gate(lg, topk, bias=bias, score=score, **kw)
        masked = lg.gather(1, ids.long()) == -math.inf
        assert torch.all(masked.int().diff(dim=1) >= 0)          # masked ones last
        assert torch.all(w[masked] == 0)
        for t in range(120):
            allowed = torch.isfinite(lg[t])
            if grouped:
                score_t = _scores(lg[t:t + 1].double(), score)[0] + bias.double()
                rank = score_t.view(4, 16).topk(2, 1).values.sum(1)
                best = torch.sort(rank, descending=True, stable=True).indices[:2]
                allowed &= torch.isin(torch.arange(64, device="cuda") // 16, best)
                assert torch.all(torch.isin(ids[t] // 16, best))
            assert (~masked[t]).sum().item() == min(topk, allowed.sum().item())
        assert torch.all(ids.sort(1).values.diff(dim=1) > 0)


def test_groups_pass_over_a_nan(fpq):
    """A NaN logit does not count toward its group's rank."""
    at = lambda p: math.log(p / (1 - p))
    lg = torch.full((2, 8), at(0.05), device="cuda")
    lg[:, 0], lg[:, 1], lg[:, 2] = at(0.9), at(0.1), math.nan        # 1.0
    lg[:, 4], lg[:, 5] = at(0.7), at(0.6)                            # 1.3
    lg[1, 2], lg[1, 0] = at(0.9), math.nan                           # before and behind the others
    ids, _ = moe.gate(lg, 2, score=moe.SIGMOID, n_group=2, topk_group=1, group_top=2)
    assert torch.equal(ids.cpu(), torch.tensor([[4, 5], [4, 5]], dtype=torch.int32))


@pytest.mark.parametrize("experts", [7, 64, 200, 1024])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward_of_the_full_softmax_with_an_id_named_twice(fpq, experts, dtype):
    lg = _logits(9, experts, experts, dtype)
    ids = torch.randint(0, experts, (9, 6), generator=torch.Generator().manual_seed(3)).int().cuda()
    ids[:, 3] = ids[:, 1]
    ids[4] = ids[4, 0]
    dw = torch.randn((9, 6), generator=torch.Generator().manual_seed(4)).cuda()
    d = moe.gate_backward(dw, lg, ids, renormalize=False, scale=0.5)
    p = _scores(lg.double(), moe.SOFTMAX)
    v = 0.5 * dw.double()
    dot = (v * p.gather(1, ids.long())).sum(1, keepdim=True)
    want = p * (torch.zeros_like(p).scatter_add_(1, ids.long(), v) - dot)
    size = p * (v.abs().sum(1, keepdim=True))
    rel = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    assert torch.all((d.double() - want).abs() <= rel * want.abs() + 2.0 ** -15 * size + 1e-37)


@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("size", [10.0, 100.0, 1000.0])
@pytest.mark.parametrize("n_group,topk_group,topk", [(8, 4, 8), (32, 8, 8)])
def test_groups_whose_best_keys_cancel(fpq, score, size, n_group, topk_group, topk):
    """One expert of a group with a large bias and the others with the
    opposite one: the keys' fp32 steps are those of the bias, their sum is of
    the order of a score."""
    bias = torch.full((256,), -size, device="cuda")
    bias[torch.arange(n_group, device="cuda") * (256 // n_group) + 3] = size
    _check(_logits(16384, 256, 41), topk, bias, score, n_group, topk_group, 2)
    # of one group only: the others' ranks are compared with it and with each other
    one = torch.zeros((256,), device="cuda")
    one[:256 // n_group] = -size
    one[3] = size
    _check(_logits(4096, 256, 42), topk, one, score, n_group, topk_group, 2)


def test_a_group_ahead_by_less_than_its_keys_steps(fpq):
    """Two groups whose fp32 ranks are in the wrong order by a step of the
    best key (2^-13 at 1024), while the exact ranks are 2^-20 apart."""
    t = 2.0 ** -20
    p = torch.full((3, 8), 0.25, dtype=torch.float64)
    p[:, 0], p[:, 1] = 0.5 + 2.0 ** -14 + t, 0.5                    # 1 + 2^-14 + t; in fp32 1 + 2^-13
    p[:, 4], p[:, 5] = 0.5 + 2.0 ** -14 - t, 0.5 + 3 * t            # 1 + 2^-14 + 2 t; in fp32 1
    p[1, 5] = 0.5                                                    # behind the first
    p[2] = p[2].roll(4)
    lg = torch.log(p / (1 - p)).float().cuda()
    bias = torch.tensor([1024.0, -1024, -1024, -1024] * 2, device="cuda")
    ids, _ = _check(lg, 2, bias, moe.SIGMOID, 2, 1, 2)
    assert torch.equal((ids[:, 0] // 4).cpu(), torch.tensor([1, 0, 0], dtype=torch.int32))
