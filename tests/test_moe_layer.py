"""The operators of a mixture-of-experts layer run together as they are used:
norm -> gate -> dispatch -> grouped product -> combination and back, and the
decoding form with NVFP4 weights; on a side stream, on two streams at once
and captured into graphs."""
import threading

import pytest
import torch

from mxfp8_block_scaled_warp_b200 import moe

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _normal(shape, std, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def _rel(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def test_prefill_layer(fpq):
    """300 tokens through a layer of 16 experts, against the same layer in 64
    bits on the decoded operands."""
    tokens, hidden, experts, topk, inter = 300, 512, 16, 4, 256
    x, res = _normal((tokens, hidden), 1, 1), _normal((tokens, hidden), 2, 2)
    w_norm, w_gate = _normal((hidden,), 0.1, 3) + 1, _normal((experts, hidden), 0.05, 4)
    w_up, w_down = _normal((experts, inter, hidden), 0.05, 5), _normal((experts, hidden, inter), 0.05, 6)
    uq, us = fpq.quantize(w_up, fpq.MXFP8)
    dq, ds = fpq.quantize(w_down, fpq.MXFP8)
    n = fpq.rmsnorm_quantize(x, w_norm, fpq.MXFP8, residual=res, want_y=True, want_rstd=True)
    logits = fpq.gemm_bf16(n.y, w_gate)
    ids, weights = moe.gate(logits, topk, bias=torch.zeros(experts, device="cuda"), score=moe.SIGMOID, n_group=4,
                            topk_group=2, scale=2.5)
    rows = torch.empty_like(ids)
    d = moe.dispatch(n.y, ids, experts, rows=rows)
    up = fpq.grouped_scaled_gemm(fpq.MXFP8, d.codes, d.scales, uq, us, d.group_offsets)
    act = torch.nn.functional.silu(up.float()).to(BF16)
    aq, a_s = fpq.quantize(act, fpq.MXFP8)
    down = fpq.grouped_scaled_gemm(fpq.MXFP8, aq, a_s, dq, ds, d.group_offsets)
    out = moe.combine(down, weights, rows=rows, add=n.h)

    s = x.double() + res.double()
    y = s / (s.square().mean(1, keepdim=True) + 1e-6).sqrt() * w_norm.double()
    assert _rel(n.y, y) < 2.0 ** -8
    row_of = torch.empty((tokens * topk,), dtype=torch.long, device="cuda")
    row_of[rows.flatten().long()] = torch.arange(tokens * topk, device="cuda")
    codes = fpq.dequantize(fpq.MXFP8, d.codes, d.scales).double()
    assert torch.equal(codes, fpq.dequantize(fpq.MXFP8, *fpq.quantize(n.y, fpq.MXFP8)).double()[row_of // topk])
    e_of = ids.flatten()[row_of].long()
    u = torch.einsum("rk,rnk->rn", codes, fpq.dequantize(fpq.MXFP8, uq, us).double()[e_of])
    assert _rel(up, u) < 2.0 ** -8
    v = torch.einsum("rk,rnk->rn", fpq.dequantize(fpq.MXFP8, aq, a_s).double(),
                     fpq.dequantize(fpq.MXFP8, dq, ds).double()[e_of])
    want = (v[rows.long()] * weights.double()[..., None]).sum(1) + s
    assert _rel(out, want) < 2.0 ** -8

    # backward of what surrounds the experts' products, for a gradient of the output
    dout = _normal((tokens, hidden), 1, 7)
    d_down, d_weights = moe.combine_backward(dout, down, weights, rows=rows)
    d_logits = moe.gate_backward(d_weights, logits, ids, score=moe.SIGMOID, scale=2.5)
    dy = fpq.gemm_bf16(d_logits, w_gate.T.contiguous())
    dx, dw = fpq.rmsnorm_backward(dy, n.h, w_norm, n.rstd, dres=dout)
    lg = logits.double().requires_grad_(True)
    hh, wn = n.h.double().requires_grad_(True), w_norm.double().requires_grad_(True)
    p = torch.sigmoid(lg).gather(1, ids.long())
    ((down.double()[rows.long()] * (2.5 * p / p.sum(1, keepdim=True))[..., None]).sum(1) * dout.double()).sum().backward()
    assert _rel(d_logits, lg.grad) < 2.0 ** -6        # bf16 logits; the sums in d_weights cancel
    (hh / (hh.square().mean(1, keepdim=True) + 1e-6).sqrt() * wn * dy.double()).sum().backward()
    assert _rel(dx, hh.grad + dout.double()) < 2.0 ** -7 and _rel(dw, wn.grad) < 2.0 ** -7
    assert d_down.shape == down.shape and fpq.fpq_get_device_error() == 0


def _decode_step(fpq, s):
    n = fpq.rmsnorm_quantize(s["x"], s["w_norm"], residual=s["res"])
    logits = (n.y.float() @ s["w_gate"].float().T)
    ids, weights = moe.gate(logits, 4, score=moe.SOFTMAX)
    up = fpq.gemv_nvfp4(n.y, *s["up"], ids=ids)
    act = torch.nn.functional.silu(up.float()).to(BF16)
    down = fpq.gemv_nvfp4(act, *s["down"], ids=ids)
    out = moe.combine(down, weights, add=n.h)
    return n, ids, weights, up, act, down, out


def _decode_state(fpq, tokens, seed):
    return {"x": _normal((tokens, 512), 1, seed), "res": _normal((tokens, 512), 2, seed + 1),
            "w_norm": _normal((512,), 0.1, 30) + 1, "w_gate": _normal((16, 512), 0.05, 31),
            "up": fpq.quantize(_normal((16, 256, 512), 0.05, 32), fpq.NVFP4),
            "down": fpq.quantize(_normal((16, 512, 256), 0.05, 33), fpq.NVFP4)}


@pytest.mark.parametrize("tokens", [1, 3, 32])
def test_decode_layer(fpq, tokens):
    s = _decode_state(fpq, tokens, 40)
    n, ids, weights, up, act, down, out = _decode_step(fpq, s)
    wu, wd = fpq.dequantize(fpq.NVFP4, *s["up"]).double(), fpq.dequantize(fpq.NVFP4, *s["down"]).double()
    u = torch.einsum("tk,tjnk->tjn", n.y.double(), wu[ids.long()])
    v = torch.einsum("tjk,tjnk->tjn", act.double(), wd[ids.long()])
    # dequantize() rounds the decoded weights to bf16
    assert _rel(up, u) < 2.0 ** -7 and _rel(down, v) < 2.0 ** -7
    want = (v * weights.double()[..., None]).sum(1) + s["x"].double() + s["res"].double()
    assert _rel(out, want) < 2.0 ** -7
    assert fpq.fpq_get_device_error() == 0


def test_decode_layer_captured(fpq):
    """The decoding step captured into two graphs that are replayed on new
    inputs, alternately, give the eager results."""
    states = [_decode_state(fpq, t, 50 + t) for t in (2, 5)]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for s in states:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _decode_step(fpq, s)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_decode_step(fpq, s))
        graphs.append(g)
    for turn in range(3):
        for s in states:
            s["x"].copy_(_normal(s["x"].shape, 1, 70 + turn))
        for g in graphs:
            g.replay()
        for s, o in zip(states, outs):
            for a, b in zip(o[1:], _decode_step(fpq, s)[1:]):
                assert torch.equal(a, b)
    assert fpq.fpq_get_device_error() == 0


def test_backward_captured(fpq):
    x, w = _normal((500, 1024), 1, 80), _normal((1024,), 0.1, 81) + 1
    dy, y = _normal((500, 1024), 1, 82), _normal((2000, 1024), 1, 83)
    lg = torch.randn((500, 64), device="cuda")

    def step():
        n = fpq.rmsnorm_quantize(x, w, fpq.FP8_1x128, want_rstd=True)
        ids, wt = moe.gate(lg, 4)
        dyy, dwt = moe.combine_backward(dy, y, wt)
        return (*fpq.rmsnorm_backward(dy, x, w, n.rstd), n.q, n.scales, ids, wt, dyy, dwt,
                moe.gate_backward(dwt, lg, ids))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (1, 2):
        x.copy_(_normal(x.shape, 1, seed))
        dy.copy_(_normal(x.shape, 1, seed + 10))
        lg.copy_(torch.randn_like(lg))
        g.replay()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


def test_side_stream_and_two_at_once(fpq):
    """Calls with a stream argument, and the same calls issued on two streams
    that overlap, give the results of one stream."""
    x, w = _normal((3000, 2048), 1, 90), _normal((2048,), 0.1, 91) + 1
    dy = _normal((3000, 2048), 1, 92)
    wq, ws, wg = fpq.quantize(_normal((16, 512, 2048), 0.02, 93), fpq.NVFP4)
    ids = torch.randint(0, 16, (16, 4), generator=torch.Generator().manual_seed(1)).int().cuda()
    wt = torch.rand((750, 4), device="cuda")

    def calls(stream):
        n = fpq.rmsnorm_quantize(x, w, fpq.MXFP8, want_rstd=True, stream=stream)
        dx, dw = fpq.rmsnorm_backward(dy, x, w, n.rstd, stream=stream)
        y = fpq.gemv_nvfp4(x[:16], wq, ws, wg, ids=ids, stream=stream)
        z = fpq.gemv_nvfp4(x[16:32], wq[3], ws[3], wg[3:4].clone(), stream=stream)
        return n.q, n.scales, n.rstd, dx, dw, y, z, moe.combine(x, wt, stream=stream)

    want = calls(None)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append(calls(a))
        got.append(calls(b.cuda_stream))
    torch.cuda.synchronize()
    for one in got:
        for u, v in zip(one, want):
            assert torch.equal(u, v)
    assert fpq.fpq_get_device_error() == 0


def test_two_host_threads(fpq):
    """The C entry points from two threads, with shapes of one kernel that need
    different amounts of shared memory: every call is accepted and right."""
    w = fpq.quantize(_normal((2048, 7168), 0.02, 100), fpq.NVFP4)
    x = _normal((16, 7168), 1, 101)
    lib = fpq.load()                                 # the library's functions themselves: the calls overlap often

    def product(m):
        y = torch.empty((m, 2048), dtype=BF16, device="cuda")
        args = [x.data_ptr(), m, *(p.data_ptr() for p in w), 2048, 7168, y.data_ptr(), fpq.OUT_BF16, None]
        return lambda: lib.fpq_gemv_nvfp4(*args), y

    def norm(rows, cols):
        a, wt, dy = _normal((rows, cols), 1, 102), _normal((cols,), 0.1, 103) + 1, _normal((rows, cols), 1, 104)
        rstd = torch.ones((rows,), device="cuda")
        dx, dw = torch.empty_like(a), torch.empty((cols,), device="cuda")
        ws = torch.empty((fpq.fpq_rmsnorm_backward_workspace_bytes(rows, cols),), dtype=torch.uint8, device="cuda")
        keep = (dy, a, wt, rstd, dx, dw, ws)
        args = [dy.data_ptr(), a.data_ptr(), cols, wt.data_ptr(), rstd.data_ptr(), None, rows, cols, dx.data_ptr(),
                dw.data_ptr(), ws.data_ptr(), ws.numel(), None]
        return lambda: (lib.fpq_rmsnorm_backward(*args), keep)[0], dx

    for pair in ((product(8), product(3)), (product(16), product(9)), (norm(20, 1024), norm(20, 528)),
                 (norm(20, 7168), norm(20, 1040))):
        want = []
        for call, out in pair:
            assert call() == 0
            want.append(out.clone())
            out.zero_()
        torch.cuda.synchronize()
        refused, start = [0, 0], threading.Barrier(2)

        def many(i):
            start.wait()
            for _ in range(10000):
                if pair[i][0]() != 0:
                    refused[i] += 1

        threads = [threading.Thread(target=many, args=(i,)) for i in range(2)]
        for th in threads:
            th.start()
        for th in threads:
            th.join()
        torch.cuda.synchronize()
        assert refused == [0, 0]
        for (_, out), u in zip(pair, want):
            assert torch.equal(out, u)


def test_large_and_small_shapes_in_one_graph(fpq):
    """A call that needs much shared memory captured before one of the same
    kernel that needs little."""
    w = fpq.quantize(_normal((2048, 7168), 0.02, 110), fpq.NVFP4)
    x, wn = _normal((20, 7168), 1, 111), _normal((7168,), 0.1, 112) + 1
    rstd = torch.ones((20,), device="cuda")

    def step():
        big = fpq.gemv_nvfp4(x[:8], *w), fpq.rmsnorm_backward(x, x, wn, rstd)[0]
        narrow, wn2 = x[:, :1040].contiguous(), wn[:1040].contiguous()
        return (*big, fpq.gemv_nvfp4(x[:3], *w), fpq.rmsnorm_backward(narrow, narrow, wn2, rstd)[0])

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for t in out:
        t.zero_()
    g.replay()
    for u, v in zip(out, want):
        assert torch.equal(u, v)
