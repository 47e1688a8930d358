"""Cases of the operators of a mixture-of-experts layer around the block-scaled
products: RMS norm into 8-bit operands, the expert gate, the weighted
combination of the experts' rows, and matrix-vector products with NVFP4
weights -- with their backward passes.

``run`` computes a case either in plain torch operations (``own`` false) or by
the library's own calls (``own`` true) on the same inputs; ``exact`` restates
each operator in 64 bits.  Formats are those of the library: E4M3 codes with
an fp32 scale per 1x128 tile or an E8M0 scale per 1x32 block, and packed E2M1
with an E4M3 scale per 16 and an fp32 scale per matrix.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoded token's residual stream on its way into an FP8 projection: latency only
        dict(name="norm_token", op="norm", rows=1, cols=7168, ld=7168, fmt="fp8", residual=True, y=False),
        # a prefill chunk: residual added, MXFP8 operand for the experts and bf16 rows for the gate, 1/rms kept for training
        dict(name="norm_prefill", op="norm", rows=8192, cols=7168, ld=7168, fmt="mxfp8", residual=True, y=True),
        # the norm of a narrow latent that is a column slice of a wider projection, ragged token count
        dict(name="norm_slice", op="norm", rows=4099, cols=512, ld=576, fmt="fp8", residual=False, y=False),
        # its backward in a training step, the residual stream's gradient joined in
        dict(name="norm_backward", op="norm_bwd", rows=8192, cols=7168, residual=True),
        # routing of a decode batch: 256 experts in 8 groups, a balance bias, sigmoid scores
        dict(name="gate_decode", op="gate", tokens=16, experts=256, topk=8, score="sigmoid", groups=8, topk_group=4,
             bias=True, renorm=True, dtype="f32"),
        # routing of a training batch over this repository's 64 experts from a bf16 product's logits
        dict(name="gate_train", op="gate", tokens=16384, experts=64, topk=8, score="softmax", groups=1, topk_group=1,
             bias=False, renorm=True, dtype="bf16"),
        # gradient of the gate's logits for 256 experts
        dict(name="gate_backward", op="gate_bwd", tokens=16384, experts=256, topk=8, score="sigmoid", renorm=True,
             dtype="f32"),
        # the experts' rows brought back to their tokens, a shared expert's output added
        dict(name="combine_train", op="combine", tokens=8192, hidden=7168, topk=8, experts=64, add=True, out="bf16"),
        # its backward: the rows' gradients and the routing weights'
        dict(name="combine_backward", op="combine_bwd", tokens=4097, hidden=7168, topk=8, experts=64),
        # one token through one projection with 4-bit weights
        dict(name="gemv_token", op="gemv", rows=1, n=2048, k=7168, out="bf16"),
        # sixteen sequences decoded together through a wide projection
        dict(name="gemv_batch", op="gemv", rows=16, n=32768, k=7168, out="f32"),
        # eight tokens, each through its eight of 64 experts
        dict(name="gemv_experts", op="gemv_moe", tokens=8, topk=8, experts=64, n=2048, k=7168, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "gate", "gate", "gate_bwd", "combine", "combine_bwd", "gemv", "gemv",
                     "gemv_moe"])
    if op in ("norm", "norm_bwd"):
        fmt = rng.choice(["fp8", "mxfp8", "none"]) if op == "norm" else "none"
        block = {"fp8": 128, "mxfp8": 32, "none": 8}[fmt]
        cols = max(1, _log(rng, 128, 16384) // block) * block
        rows = _log(rng, 1, min(20000, 8192 * 7168 // cols))
        if op == "norm_bwd":
            return dict(op=op, rows=rows, cols=cols, residual=rng.random() < 0.5)
        residual = rng.random() < 0.6
        ld = cols if residual or rng.random() < 0.5 else cols + 8 * rng.randrange(1, 40)
        return dict(op=op, rows=rows, cols=cols, ld=ld, fmt=fmt, residual=residual,
                    y=fmt == "none" or rng.random() < 0.4)
    if op in ("gate", "gate_bwd"):
        experts = rng.choice([8, 16, 40, 64, 96, 128, 160, 256, 384, 512])
        topk = rng.randrange(1, min(12, experts // 2) + 1)
        tokens = _log(rng, 1, 16384 * 256 // max(experts, 256))
        case = dict(op=op, tokens=tokens, experts=experts, topk=topk, score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.7, dtype=rng.choice(["f32", "bf16"]))
        if op == "gate":
            groups = rng.choice([1, 1, 4, 8])
            tg = max(1, groups // 2)
            if groups > 1 and (experts // groups < 2 or tg * (experts // groups) < topk):
                groups, tg = 1, 1
            case.update(groups=groups, topk_group=tg, bias=rng.random() < 0.5)
        return case
    if op in ("combine", "combine_bwd"):
        experts = rng.choice([8, 64, 128])
        topk = rng.randrange(1, 9)
        hidden = 8 * _log(rng, 16, 1024)
        most = 1_000_000_000 // (hidden * (2 * topk + 8 if op == "combine" else 4 * topk + 4))
        tokens = _log(rng, 1, min(16384, most))
        if op == "combine_bwd":
            return dict(op=op, tokens=tokens, hidden=hidden, topk=topk, experts=experts)
        return dict(op=op, tokens=tokens, hidden=hidden, topk=topk, experts=experts, add=rng.random() < 0.5,
                    out=rng.choice(["bf16", "f32"]))
    k = 32 * _log(rng, 8, 448)
    if op == "gemv":
        return dict(op=op, rows=rng.randrange(1, 17), n=_log(rng, 64, 32768 * 7168 // max(k, 7168)), k=k,
                    out=rng.choice(["bf16", "f32"]))
    experts = rng.choice([8, 32, 64])
    return dict(op=op, tokens=_log(rng, 1, 8), topk=rng.randrange(1, 9), experts=experts, n=_log(rng, 64, 2048),
                k=min(k, 7168), out=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nvfp4(w):
    """Packed codes, E4M3 scale bytes and the matrix's fp32 scale of w [n, k] (quantized as a checkpoint would be)."""
    n, k = w.shape
    w = w.float().view(n, k // 16, 16)
    g = w.abs().amax() / 2688.0
    s = (w.abs().amax(-1) / 6.0 / g).to(torch.float8_e4m3fn)
    big = (s.float() * g).unsqueeze(-1)
    mag = torch.where(big > 0, w.abs() / big, torch.zeros_like(w))
    mids = torch.tensor([(a + b) / 2 for a, b in zip(_LEVELS[:-1], _LEVELS[1:])], device=w.device)
    code = torch.bucketize(mag, mids, out_int32=True).to(torch.uint8) | ((w < 0).to(torch.uint8) << 3)
    code = code.view(n, k // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), s.view(torch.uint8), g.reshape(1)


def _choices(g, tokens, experts, topk):
    """Expert ids of each token: distinct, the popular ones more often (Gumbel-top-k on (e + 1)^-0.5)."""
    u = torch.rand((tokens, experts), generator=g, device="cuda").clamp_min(1e-20)
    pop = -0.5 * torch.log(torch.arange(1, experts + 1, device="cuda").float())
    return torch.topk(pop - torch.log(-torch.log(u)), topk, dim=1).indices.to(torch.int32).contiguous()


def _rows_of(ids):
    """Row of each (token, choice) pair in the buffer grouped by expert, then token."""
    flat = ids.flatten().long()
    order = torch.argsort(flat, stable=True)
    rows = torch.empty_like(order)
    rows[order] = torch.arange(flat.numel(), device=ids.device)
    return rows.view_as(ids).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    c, op, s = case, case["op"], {"case": case}
    if op in ("norm", "norm_bwd"):
        rows, cols = c["rows"], c["cols"]
        s["w"] = (1 + _normal(g, (cols,), 0.1, F32)).to(BF16)
        hot = torch.ones(cols, device="cuda")
        hot[torch.randint(0, cols, (max(1, cols // 512),), generator=g, device="cuda")] = 20.0   # outlier channels
        ld = c.get("ld", cols)
        wide = torch.zeros((rows, ld), dtype=BF16, device="cuda")
        wide[:, :cols] = (torch.randn((rows, cols), generator=g, device="cuda") * hot).to(BF16)
        if ld > cols:
            wide[:, cols:] = _normal(g, (rows, ld - cols), 30.0)
        s["x"] = wide[:, :cols]
        if op == "norm":
            s["res"] = _normal(g, (rows, cols), 2.0) if c["residual"] else None
        else:
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(-1) + 1e-6)
            s["dy"] = _normal(g, (rows, cols), 0.01)
            s["dres"] = _normal(g, (rows, cols), 0.01) if c["residual"] else None
    elif op in ("gate", "gate_bwd"):
        shape = (c["tokens"], c["experts"])
        dt = F32 if c["dtype"] == "f32" else BF16
        s["logits"] = (_normal(g, shape, 1.5, F32) + _normal(g, shape[1:], 0.5, F32)).to(dt)
        if op == "gate":
            steps = torch.randint(-60, 61, shape[1:], generator=g, device="cuda").float()
            s["bias"] = steps * 0.001 if c["bias"] else None
        else:
            s["ids"] = torch.topk(s["logits"].float(), c["topk"], dim=1).indices.to(torch.int32).contiguous()
            s["dweights"] = _normal(g, (c["tokens"], c["topk"]), 0.1, F32)
    elif op in ("combine", "combine_bwd"):
        t, h, k = c["tokens"], c["hidden"], c["topk"]
        s["rows"] = _rows_of(_choices(g, t, c["experts"], k))
        wt = torch.rand((t, k), generator=g, device="cuda") + 0.05
        s["weights"] = wt / wt.sum(1, keepdim=True)
        s["y"] = _normal(g, (t * k, h), 0.5)
        if op == "combine":
            s["add"] = _normal(g, (t, h), 0.5) if c["add"] else None
        else:
            s["dout"] = _normal(g, (t, h), 0.01)
    elif op == "gemv":
        s["x"] = _normal(g, (c["rows"], c["k"]))
        s["wq"], s["ws"], s["wg"] = _nvfp4(_normal(g, (c["n"], c["k"]), 0.02))
    else:
        s["x"] = _normal(g, (c["tokens"], c["k"]))
        s["ids"] = _choices(g, c["tokens"], c["experts"], c["topk"])
        parts = [_nvfp4(_normal(g, (c["n"], c["k"]), 0.02)) for _ in range(c["experts"])]
        s["wq"], s["ws"] = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
        s["wg"] = torch.cat([p[2] for p in parts])
    return s


# ------------------------------------------------------------------ plain forms

def _out_dtype(case):
    return F32 if case["out"] == "f32" else BF16


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    if s["res"] is not None:
        x = x + s["res"].float()
    rstd = torch.rsqrt(x.square().mean(-1) + 1e-6)
    y = x * rstd[:, None] * s["w"].float()
    out = {"rstd": rstd}
    if s["res"] is not None:
        out["h"] = x.to(BF16)
    if c["y"]:
        out["y"] = y.to(BF16)
    if c["fmt"] == "fp8":
        t = y.view(c["rows"], c["cols"] // 128, 128)
        scale = t.abs().amax(-1) / 448.0
        scale = torch.where(scale > 0, scale, torch.ones_like(scale))
        out["q"] = (t / scale[..., None]).view_as(y).to(torch.float8_e4m3fn)
        out["scales"] = scale
    elif c["fmt"] == "mxfp8":
        t = y.view(c["rows"], c["cols"] // 32, 32)
        mant, expo = torch.frexp(t.abs().amax(-1) / 448.0)          # amax/448 = mant 2^expo, mant in [0.5, 1)
        e = torch.where(mant > 0.5, expo, expo - 1).clamp(-127, 127)
        out["q"] = (t * torch.exp2(-e.float())[..., None]).view_as(y).to(torch.float8_e4m3fn)
        out["scales"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _plain_norm_bwd(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = x * rstd
    gy = dy * s["w"].float()
    dx = rstd * (gy - xhat * (gy * xhat).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(BF16), "dweight": (dy * xhat).sum(0)}


def _plain_gate(s):
    # keys in 64 bits: two experts' scores may lie closer than 32 bits tell apart
    c = s["case"]
    t, e, k, n_group = c["tokens"], c["experts"], c["topk"], c["groups"]
    lg = s["logits"].double()
    score = torch.sigmoid(lg) if c["score"] == "sigmoid" else torch.softmax(lg, -1)
    key = lg if s["bias"] is None else score + s["bias"].double()
    if n_group > 1:
        per = (score if s["bias"] is None else key).view(t, n_group, e // n_group)
        best = torch.sort(per, dim=-1, descending=True).values[..., :2].sum(-1)
        chosen = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros_like(best).scatter_(1, chosen, 1.0).repeat_interleave(e // n_group, dim=1)
        key = torch.where(keep > 0, key, torch.full_like(key, -math.inf))
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(score, 1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (w * 2.5).to(F32)}


def _plain_gate_bwd(s):
    c = s["case"]
    lg, ids, dw = s["logits"].float(), s["ids"].long(), s["dweights"] * 2.5
    score = torch.sigmoid(lg) if c["score"] == "sigmoid" else torch.softmax(lg, -1)
    sel = torch.gather(score, 1, ids)
    if c["renorm"]:
        total = sel.sum(-1, keepdim=True)
        dw = (dw - (dw * sel / total).sum(-1, keepdim=True)) / total
    ds = torch.zeros_like(score).scatter_(1, ids, dw)
    if c["score"] == "sigmoid":
        d = ds * score * (1 - score)
    else:
        d = score * (ds - (ds * score).sum(-1, keepdim=True))
    return {"dlogits": d.to(s["logits"].dtype)}


def _plain_combine(s):
    rows = s["y"][s["rows"].long()].float()                       # [tokens, topk, hidden]
    out = (rows * s["weights"][..., None]).sum(1)
    if s["add"] is not None:
        out = out + s["add"].float()
    return {"out": out.to(_out_dtype(s["case"]))}


def _plain_combine_bwd(s):
    d, rows = s["dout"].float(), s["rows"].long()
    dweights = (s["y"][rows].float() * d[:, None, :]).sum(-1)
    dy = torch.empty_like(s["y"])
    dy[rows.flatten()] = (s["weights"][..., None] * d[:, None, :]).to(BF16).flatten(0, 1)
    return {"dy": dy, "dweights": dweights}


def _decoded(wq, ws, wg):
    """fp32 weights of packed codes [..., n, k/2], E4M3 scales [..., n, k/16] and scales wg [...]."""
    levels = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), device=wq.device)
    code = torch.stack([wq & 15, wq >> 4], -1).flatten(-2).int()
    w = levels[code].unflatten(-1, (-1, 16)) * ws.view(torch.float8_e4m3fn).float()[..., None]
    return w.flatten(-2) * wg[..., None, None]


def _plain_gemv(s):
    w = _decoded(s["wq"], s["ws"], s["wg"][0])
    return {"y": (s["x"].float() @ w.T).to(_out_dtype(s["case"]))}


def _plain_gemv_moe(s):
    used, at = torch.unique(s["ids"].long(), return_inverse=True)       # each chosen expert decoded once
    w = _decoded(s["wq"][used], s["ws"][used], s["wg"][used])
    every = torch.einsum("tk,enk->ten", s["x"].float(), w)
    y = torch.gather(every, 1, at.view_as(s["ids"])[..., None].expand(-1, -1, w.shape[1]))
    return {"y": y.to(_out_dtype(s["case"]))}


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "gate": _plain_gate, "gate_bwd": _plain_gate_bwd,
          "combine": _plain_combine, "combine_bwd": _plain_combine_bwd, "gemv": _plain_gemv,
          "gemv_moe": _plain_gemv_moe}


# ------------------------------------------------------------------ the library's calls

def _own_run(s):
    import mxfp8_block_scaled_warp_b200 as fpq
    from mxfp8_block_scaled_warp_b200 import moe
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        fmt = {"fp8": fpq.FP8_1x128, "mxfp8": fpq.MXFP8, "none": None}[c["fmt"]]
        r = fpq.rmsnorm_quantize(s["x"], s["w"], fmt, eps=1e-6, residual=s["res"], want_y=c["y"], want_rstd=True)
        out = {"rstd": r.rstd}
        if s["res"] is not None:
            out["h"] = r.h
        if c["y"]:
            out["y"] = r.y
        if fmt is not None:
            out["q"] = r.q.view(torch.float8_e4m3fn)
            out["scales"] = r.scales if c["fmt"] == "fp8" else r.scales.view(torch.float8_e8m0fnu)
        return out
    if op == "norm_bwd":
        dx, dweight = fpq.rmsnorm_backward(s["dy"], s["x"], s["w"], s["rstd"], dres=s["dres"])
        return {"dx": dx, "dweight": dweight}
    if op in ("gate", "gate_bwd"):
        score = moe.SIGMOID if c["score"] == "sigmoid" else moe.SOFTMAX
        if op == "gate":
            ids, weights = moe.gate(s["logits"], c["topk"], bias=s["bias"], score=score, n_group=c["groups"],
                                    topk_group=c["topk_group"], group_top=2, renormalize=c["renorm"], scale=2.5)
            return {"ids": ids, "weights": weights}
        return {"dlogits": moe.gate_backward(s["dweights"], s["logits"], s["ids"], score=score,
                                             renormalize=c["renorm"], scale=2.5)}
    if op == "combine":
        return {"out": moe.combine(s["y"], s["weights"], rows=s["rows"], add=s["add"], out_dtype=_out_dtype(c))}
    if op == "combine_bwd":
        dy, dweights = moe.combine_backward(s["dout"], s["y"], s["weights"], rows=s["rows"])
        return {"dy": dy, "dweights": dweights}
    return {"y": fpq.gemv_nvfp4(s["x"], s["wq"], s["ws"], s["wg"], ids=s.get("ids"), out_dtype=_out_dtype(c))}


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    if op == "norm":
        n = c["rows"] * c["cols"]
        b = 2 * n * (1 + 2 * c["residual"] + c["y"]) + 2 * c["cols"] + 4 * c["rows"]
        b += {"fp8": n + n // 32, "mxfp8": n + n // 32, "none": 0}[c["fmt"]]
        return {"bytes": b, "flops": 8 * n}
    if op == "norm_bwd":
        n = c["rows"] * c["cols"]
        return {"bytes": 2 * n * (3 + c["residual"]) + 6 * c["cols"] + 4 * c["rows"], "flops": 12 * n}
    if op in ("gate", "gate_bwd"):
        n = c["tokens"] * c["experts"]
        size = 4 if c["dtype"] == "f32" else 2
        b = n * size + 8 * c["tokens"] * c["topk"]
        return {"bytes": b + (n * size if op == "gate_bwd" else 4 * c["experts"] * c["bias"]), "flops": 10 * n}
    if op == "combine":
        n = c["tokens"] * c["hidden"]
        size = 4 if c["out"] == "f32" else 2
        return {"bytes": 2 * n * (c["topk"] + c["add"]) + size * n + 8 * c["tokens"] * c["topk"],
                "flops": 2 * n * c["topk"]}
    if op == "combine_bwd":
        n = c["tokens"] * c["hidden"]
        return {"bytes": 2 * n * (1 + 2 * c["topk"]) + 12 * c["tokens"] * c["topk"], "flops": 3 * n * c["topk"]}
    size = 4 if c["out"] == "f32" else 2
    per = c["n"] * c["k"] * 9 // 16 + 4
    if op == "gemv":
        return {"bytes": per + c["rows"] * (2 * c["k"] + size * c["n"]), "flops": 2 * c["rows"] * c["n"] * c["k"]}
    seen = c["experts"] * (1 - (1 - c["topk"] / c["experts"]) ** c["tokens"]) if c["experts"] > c["topk"] else c["experts"]
    pairs = c["tokens"] * c["topk"]
    return {"bytes": int(seen * per) + c["tokens"] * 2 * c["k"] + pairs * (4 + size * c["n"]),
            "flops": 2 * pairs * c["n"] * c["k"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op == "norm":
        v = s["x"].to(F64)
        if c["residual"]:
            v = v + s["res"].to(F64)
        inv = 1 / (v.pow(2).sum(1) / c["cols"] + 1e-6).sqrt()
        y = torch.einsum("rc,r,c->rc", v, inv, s["w"].to(F64))
        out = {"rstd": inv}
        if c["residual"]:
            out["h"] = v
        if c["y"]:
            out["y"] = y
        if c["fmt"] != "none":
            width = 128 if c["fmt"] == "fp8" else 32
            top = y.reshape(-1, width).abs().max(1).values
            if c["fmt"] == "fp8":
                scale = torch.where(top == 0, torch.ones_like(top), top / 448)
            else:
                scale = torch.where(top == 0, torch.full_like(top, 2.0 ** -127), 2 ** torch.ceil(torch.log2(top / 448)))
            out["q"] = (y.reshape(-1, width) / scale[:, None]).reshape(y.shape)
            out["scales"] = scale.reshape(c["rows"], -1)
        return out
    if op == "norm_bwd":
        x, gy, r, w = (s[n].to(F64) for n in ("x", "dy", "rstd", "w"))
        # d/dx_j of sum_i gy_i w_i x_i r(x), with dr/dx_j = -r^3 x_j / cols
        dot = torch.einsum("rc,rc,c->r", gy, x, w)
        dx = torch.einsum("r,rc,c->rc", r, gy, w) - x * (r.pow(3) * dot / c["cols"])[:, None]
        if c["residual"]:
            dx += s["dres"].to(F64)
        return {"dx": dx, "dweight": torch.einsum("rc,rc,r->c", gy, x, r)}
    if op == "gate":
        lg = s["logits"].to(F64)
        p = 1 / (1 + torch.exp(-lg)) if c["score"] == "sigmoid" else torch.exp(lg - torch.logsumexp(lg, 1, True))
        # the greedy definition: take the best that is left, the lowest index among equals
        left = (lg if s["bias"] is None else p + s["bias"].to(F64)).clone()
        e, n = c["experts"], c["groups"]
        if n > 1:
            val = (p if s["bias"] is None else left).reshape(-1, n, e // n)
            rank = val.topk(2, dim=2).values.sum(2)
            open_ = torch.zeros_like(rank, dtype=torch.bool)
            for _ in range(c["topk_group"]):
                open_.scatter_(1, rank.argmax(1, keepdim=True), True)
                rank = rank.masked_fill(open_, -math.inf)
            left = left.masked_fill(~open_.repeat_interleave(e // n, 1), -math.inf)
        ids = []
        for _ in range(c["topk"]):
            best = left == left.max(1, keepdim=True).values
            first = torch.where(best, torch.arange(e, device=lg.device), e).min(1, keepdim=True).values
            ids.append(first)
            left = left.scatter(1, first, -math.inf)
        ids = torch.cat(ids, 1)
        w = p.gather(1, ids)
        return {"ids": ids.to(torch.int32), "weights": 2.5 * (w / w.sum(1, keepdim=True) if c["renorm"] else w)}
    if op == "gate_bwd":
        lg = s["logits"].to(F64).requires_grad_(True)
        with torch.enable_grad():
            p = 1 / (1 + torch.exp(-lg)) if c["score"] == "sigmoid" else torch.exp(lg - torch.logsumexp(lg, 1, True))
            w = p.gather(1, s["ids"].long())
            w = 2.5 * (w / w.sum(1, keepdim=True) if c["renorm"] else w)
            (w * s["dweights"].to(F64)).sum().backward()
        return {"dlogits": lg.grad}
    if op == "combine":
        out = torch.zeros((c["tokens"], c["hidden"]), dtype=F64, device="cuda")
        if c["add"]:
            out += s["add"]
        for j in range(c["topk"]):
            out += s["weights"][:, j:j + 1].to(F64) * s["y"].index_select(0, s["rows"][:, j].int())
        return {"out": out}
    if op == "combine_bwd":
        d = s["dout"].to(F64)
        dy = torch.zeros(s["y"].shape, dtype=F64, device="cuda")
        dw = []
        for j in range(c["topk"]):
            at = s["rows"][:, j].long()
            dy.index_copy_(0, at, d * s["weights"][:, j:j + 1].to(F64))
            dw.append(torch.einsum("th,th->t", d, s["y"].index_select(0, at).to(F64)))
        return {"dy": dy, "dweights": torch.stack(dw, 1)}

    def weight(q, sc, g):
        value = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=F64, device="cuda") / 2
        lo, hi = (q & 15).long(), (q >> 4).long()
        v = torch.stack([value[lo & 7] * (1 - 2 * (lo >> 3)), value[hi & 7] * (1 - 2 * (hi >> 3))], 2).reshape(q.shape[0], -1)
        return v * sc.view(torch.float8_e4m3fn).to(F64).repeat_interleave(16, 1) * g.to(F64)

    x = s["x"].to(F64)
    if op == "gemv":
        return {"y": torch.cat([x @ weight(s["wq"][i:i + 4096], s["ws"][i:i + 4096], s["wg"]).T
                                for i in range(0, c["n"], 4096)], 1)}
    y = torch.zeros((c["tokens"], c["topk"], c["n"]), dtype=F64, device="cuda")
    for e in s["ids"].unique().tolist():
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        y[t, j] = x[t] @ weight(s["wq"][e], s["ws"][e], s["wg"][e]).T
    return {"y": y}
