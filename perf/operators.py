"""Timed cases of the operators around the expert GEMMs of an MoE layer.

  router   scores (softmax or sigmoid), balance bias, expert groups, top-k, weights; with its gradient
  combine  the weighted sum of a token's expert rows; with its gradients
  norm     residual addition + root-mean-square norm, MXFP8 copy of the output; with its gradients
  mxfp4    quantisation of the grouped rows and their grouped product with MXFP4 weights

``listed`` and ``draw`` give cases, ``prepare`` their inputs on the GPU, ``run`` one pass (in plain
torch operations, or with ``own`` set the library's kernels), ``work`` what a pass has to move and
compute, ``exact`` the outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token's routing while decoding: latency of a launch
        dict(name="router one token", op="router", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8,
             keep=4, top2=True, renorm=True, scale=2.5, bf16=False, grad=False),
        # a prompt's routing over 256 experts, limited to 4 of 8 groups
        dict(name="router prompt", op="router", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8,
             keep=4, top2=True, renorm=True, scale=2.5, bf16=False, grad=False),
        # a training step's routing over 32 experts from bf16 logits, an odd token count, with its gradient
        dict(name="router train", op="router", T=8191, E=32, k=4, score="softmax", bias=False, groups=1,
             keep=1, top2=False, renorm=True, scale=1.0, bf16=True, grad=True),
        # a small decoding batch: the expert rows back to tokens, onto the residual
        dict(name="combine tokens", op="combine", T=16, k=4, H=2880, drop=0.0, residual=True, grad=False),
        # a training step's combine with 1% of the pairs dropped by capacity, and its gradients
        dict(name="combine train", op="combine", T=2047, k=8, H=7168, drop=0.01, residual=False, grad=True),
        # the norm before one decoded token's experts, with the MXFP8 rows their GEMM reads
        dict(name="norm one token", op="norm", T=1, H=7168, residual=True, mx=True, grad=False),
        # the same over a prompt
        dict(name="norm prompt", op="norm", T=16384, H=7168, residual=True, mx=True, grad=False),
        # a training step's norm and its gradients
        dict(name="norm train", op="norm", T=8191, H=2880, residual=True, mx=False, grad=True),
        # one decoded token: 8 experts' second product, bound by their weights
        dict(name="mxfp4 one token", op="mxfp4", rows=8, pad=0, E=32, N=7168, K=2048, a="fp4", skew=0.0),
        # 8 decoded tokens, 4 experts each: the first product (gate and up columns)
        dict(name="mxfp4 tokens", op="mxfp4", rows=32, pad=0, E=32, N=5760, K=2880, a="fp4", skew=0.5),
        # a prompt of 8192 tokens, 4 experts each, both operands in 4 bits
        dict(name="mxfp4 prompt", op="mxfp4", rows=32768, pad=0, E=32, N=5760, K=2880, a="fp4", skew=0.5),
        # an expert share with uneven groups, rows in 8 bits, and rows behind the last group
        dict(name="mxfp4 share", op="mxfp4", rows=16384, pad=100, E=32, N=4096, K=7168, a="fp8", skew=1.1),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["router", "combine", "norm", "mxfp4"])
    if op == "router":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _spread(rng, 4, 512 // groups)
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(16, keep * (E // groups)))
        return dict(op=op, T=_spread(rng, 1, 8192), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, keep=keep, top2=rng.random() < 0.5,
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), bf16=rng.random() < 0.4,
                    grad=rng.random() < 0.5)
    if op == "combine":
        k = rng.randint(1, 8)
        return dict(op=op, T=_spread(rng, 1, 16384 // k), k=k, H=8 * _spread(rng, 8, 896),
                    drop=rng.choice([0.0, 0.0, 0.05]), residual=rng.random() < 0.5, grad=rng.random() < 0.5)
    if op == "norm":
        mx = rng.random() < 0.5
        H = 32 * _spread(rng, 2, 224) if mx else 8 * _spread(rng, 8, 896)
        return dict(op=op, T=_spread(rng, 1, 16384), H=H, residual=rng.random() < 0.6, mx=mx,
                    grad=rng.random() < 0.5)
    E = _spread(rng, 1, 32)
    return dict(op=op, rows=_spread(rng, 1, 16384), pad=rng.choice([0, 0, 37]), E=E,
                N=64 * _spread(rng, 2, 64), K=32 * _spread(rng, 4, 224), a=rng.choice(["fp4", "fp8"]),
                skew=rng.choice([0.0, 0.5, 1.1]))


# ----------------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _group_sizes(rows, E, skew):
    """Group sizes that sum to ``rows``, the r-th in proportion to r^-skew (largest remainders up)."""
    w = [(r + 1) ** -skew for r in range(E)]
    quota = [rows * v / sum(w) for v in w]
    size = [int(q) for q in quota]
    for r in sorted(range(E), key=lambda r: (size[r] - quota[r], r))[:rows - sum(size)]:
        size[r] += 1
    return size


# e2m1 values by code; codes of normal values in units of the block scale, as 256 equally likely ones
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _codes_of_normal():
    q = torch.distributions.Normal(0.0, 2.0).icdf((torch.arange(256) + 0.5) / 256).clamp(-6, 6)
    code = (q.abs()[:, None] - torch.tensor(E2M1)[None]).abs().argmin(1)
    return (code + 8 * (q < 0)).to(torch.uint8)


def prepare(case, seed):
    c = case
    g = _generator(seed)
    s = {"case": c}
    if c["op"] == "router":
        T, E, k = c["T"], c["E"], c["k"]
        s["logits"] = _normal(g, T, E, std=1.5, dtype=BF16 if c["bf16"] else torch.float32)
        s["bias"] = _normal(g, E, std=0.1, dtype=torch.float32) if c["bias"] else None
        s["dw"] = _normal(g, T, k, dtype=torch.float32) if c["grad"] else None
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["w"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
        s["dlogits"] = torch.empty_like(s["logits"]) if c["grad"] else None
    elif c["op"] == "combine":
        T, k, H = c["T"], c["k"], c["H"]
        E = 32   # pairs grouped by expert, as the routing leaves them; the rows of dropped pairs stay unused
        e = torch.randn(T, E, generator=g, device=DEV).topk(k, 1).indices.flatten()
        order = e.sort(stable=True).indices
        dst = torch.empty(T * k, dtype=torch.int32, device=DEV)
        dst[order] = torch.arange(T * k, dtype=torch.int32, device=DEV)
        dst[torch.rand(T * k, generator=g, device=DEV) < c["drop"]] = -1
        s["dst"] = dst.view(T, k)
        s["y"] = _normal(g, T * k, H)
        s["w"] = torch.randn(T, k, generator=g, device=DEV).softmax(1)
        s["residual"] = _normal(g, T, H) if c["residual"] else None
        s["out"] = torch.empty(T, H, dtype=BF16, device=DEV)
        if c["grad"]:
            s["dout"] = _normal(g, T, H, std=0.01)
            s["dy"] = torch.zeros(T * k, H, dtype=BF16, device=DEV)
            s["dw"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
    elif c["op"] == "norm":
        T, H = c["T"], c["H"]
        s["x"] = _normal(g, T, H)
        s["residual"] = _normal(g, T, H, std=3.0) if c["residual"] else None
        s["weight"] = (1 + _normal(g, H, std=0.2, dtype=torch.float32)).to(BF16)
        s["h"] = torch.empty_like(s["x"]) if c["residual"] else s["x"]
        s["y"] = torch.empty_like(s["x"])
        s["rstd"] = torch.empty(T, dtype=torch.float32, device=DEV)
        if c["mx"]:
            s["q"] = torch.empty(T, H, dtype=torch.uint8, device=DEV)
            s["s"] = torch.empty(T, H // 32, dtype=torch.uint8, device=DEV)
        if c["grad"]:
            s["dy"] = _normal(g, T, H, std=0.01)
            s["dh"] = _normal(g, T, H, std=0.01)      # the gradient that comes down the residual
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"] = torch.empty(H, dtype=torch.float32, device=DEV)
            s["scratch"] = torch.empty(4 << 20, dtype=torch.float32, device=DEV)
    else:
        E, N, K = c["E"], c["N"], c["K"]
        cap = c["rows"] + c["pad"]
        sizes = _group_sizes(c["rows"], E, c["skew"])
        perm = torch.randperm(E, generator=g, device=DEV).tolist()
        s["sizes"] = [sizes[p] for p in perm]
        s["counts"] = torch.tensor(s["sizes"], dtype=torch.int32, device=DEV)
        s["x"] = _normal(g, cap, K)
        s["x"] *= torch.exp(torch.randn(cap, 1, generator=g, device=DEV)).to(BF16)   # rows of uneven size
        table = _codes_of_normal().to(DEV)
        lo = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        hi = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["wq"] = table[lo.int()] | (table[hi.int()] << 4)
        s["ws"] = torch.randint(118, 122, (E, N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
        s["aq"] = torch.empty(cap, K // 2 if c["a"] == "fp4" else K, dtype=torch.uint8, device=DEV)
        s["as"] = torch.empty(cap, K // 32, dtype=torch.uint8, device=DEV)
        s["out"] = torch.zeros(cap, N, dtype=BF16, device=DEV)
    return s


# ----------------------------------------------------------------------------- plain forms
def _router_plain(s, c):
    """ids by the choice value (score + bias, or the logit), ties to the lower id; the scores and the choice in
    64 bits, since one unit in the last place decides between neighbours."""
    x = s["logits"].double()
    if c["score"] == "softmax":
        score = torch.exp(x - x.max(1, keepdim=True).values)
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-x))
    choice = score + s["bias"].double() if c["bias"] else x
    if c["groups"] > 1:
        T, E, G = c["T"], c["E"], c["groups"]
        # a group's value: its two best scores (with the bias) together, or its best choice value
        if c["top2"]:
            value = (choice if c["bias"] else score).view(T, G, E // G)
            value = value.sort(2, descending=True).values[..., :2].sum(2)
        else:
            value = choice.view(T, G, E // G).max(2).values
        kept = value.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter(1, kept, True)
        choice = torch.where(open_.repeat_interleave(E // G, 1), choice, -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    sel = score.gather(1, ids)
    total = sel.sum(1, keepdim=True) if c["renorm"] else torch.ones_like(sel[:, :1])
    out = {"ids": ids.int(), "weights": (c["scale"] * sel / total).float()}
    if c["grad"]:
        dsel = c["scale"] * s["dw"].double() / total
        if c["renorm"]:
            dsel = dsel - (dsel * sel).sum(1, keepdim=True) / total
        if c["score"] == "softmax":
            dx = -score * (dsel * sel).sum(1, keepdim=True)
            dx = dx.scatter_add(1, ids, dsel * sel)
        else:
            dx = torch.zeros_like(x).scatter(1, ids, dsel * sel * (1 - sel))
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


def _combine_plain(s, c):
    there = (s["dst"] >= 0)[..., None]
    at = s["dst"].clamp(min=0).long()
    rows = torch.where(there, s["y"][at].float(), 0.0)          # [T, k, H]
    out = (rows * s["w"][..., None]).sum(1)
    if c["residual"]:
        out = out + s["residual"].float()
    got = {"out": out.to(BF16)}
    if c["grad"]:
        dout = s["dout"].float()
        got["dw"] = (rows * dout[:, None]).sum(2)
        dy = torch.zeros(s["y"].shape, dtype=BF16, device=DEV)
        # dropped pairs go to a row of their own, which is cut off
        dy = torch.cat([dy, dy[:1]])
        dy[torch.where(s["dst"] >= 0, s["dst"], len(dy) - 1).flatten().long()] = (
            dout[:, None] * s["w"][..., None]).to(BF16).flatten(0, 1)
        got["dy"] = dy[:-1]
    return got


def _mx_scale(amax, cut, exponent):
    """The smallest E with amax / 2^E <= cut * 2^exponent (amax = m 2^e, m in [0.5, 1)), cut in [0.5, 1)."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, e - exponent + (m > cut).int(), -127).clamp(-127, 127)


def _norm_plain(s, c):
    h = (s["x"].float() + s["residual"].float()).to(BF16) if c["residual"] else s["x"]
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(1, keepdim=True) + 1e-6)
    y = (f * rstd * s["weight"].float()).to(BF16)
    out = {"h": h, "y": y, "rstd": rstd[:, 0]}
    if c["mx"]:
        v = y.float().view(c["T"], -1, 32)
        e = _mx_scale(v.abs().amax(2), 0.875, 9)               # 448 = 0.875 * 2^9
        out["s"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
        out["q"] = torch.ldexp(v, -e[..., None]).flatten(1).to(torch.float8_e4m3fn)
    if c["grad"]:
        gw = s["dy"].float() * s["weight"].float()
        n = f * rstd
        dx = rstd * (gw - n * (gw * n).mean(1, keepdim=True)) + s["dh"].float()
        out["dx"] = dx.to(BF16)
        out["dweight"] = (s["dy"].double() * n.double()).sum(0).float()
    return out


def _round_e2m1(v):
    """v (at most 6 in size) to the nearest e2m1 value, ties to the even code."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, v)


def _e2m1_table(dtype):
    v = torch.tensor(E2M1 + [-x for x in E2M1], dtype=dtype, device=DEV)
    b = torch.arange(256, device=DEV)
    return torch.stack([v[b & 15], v[b >> 4]], 1)


def _mxfp4_plain(s, c):
    cap, K = s["x"].shape
    v = s["x"].float().view(cap, -1, 32)
    amax = v.abs().amax(2)
    if c["a"] == "fp4":
        e = _mx_scale(amax, 0.75, 3)[..., None]                # 6 = 0.75 * 2^3
        q = _round_e2m1(torch.ldexp(v, -e))
    else:
        e = _mx_scale(amax, 0.875, 9)[..., None]
        q = torch.ldexp(v, -e).to(torch.float8_e4m3fn).float()
    x = torch.ldexp(q, e).view(cap, K)
    w = _e2m1_table(torch.float32)[s["wq"].int()].view(c["E"], c["N"], K // 32, 32)
    w = (w * torch.exp2(s["ws"].float() - 127)[..., None]).view(c["E"], c["N"], K)
    out = torch.zeros(cap, c["N"], dtype=BF16, device=DEV)
    parts = [a @ b.t() for a, b in zip(x[:c["rows"]].split(s["sizes"]), w)]
    out[:c["rows"]] = torch.cat(parts).to(BF16)
    return out


# ----------------------------------------------------------------------------- one pass
def _run_own(s, c):
    import grouped_gemm_glu_amd as G
    if c["op"] == "router":
        r = G.router(c["score"], bias=s["bias"], n_groups=c["groups"], topk_groups=c["keep"],
                     group_score="top2" if c["top2"] else "max", renorm=c["renorm"], scale=c["scale"])
        G.moe_router_topk(s["logits"], c["T"], c["E"], c["k"], r, s["ids"], s["w"])
        out = {"ids": s["ids"], "weights": s["w"]}
        if c["grad"]:
            G.moe_router_topk_bwd(s["logits"], c["T"], c["E"], c["k"], r, s["ids"], s["dw"], s["dlogits"])
            out["dlogits"] = s["dlogits"]
        return out
    if c["op"] == "combine":
        M = s["y"].shape[0]
        G.moe_combine(s["y"], M, c["H"], s["dst"], c["T"], c["k"], s["out"], weights=s["w"],
                      residual=s["residual"])
        out = {"out": s["out"]}
        if c["grad"]:
            G.moe_combine_bwd(s["dout"], s["y"], M, c["H"], s["dst"], c["T"], c["k"], weights=s["w"],
                              dy=s["dy"], dweights=s["dw"])
            out |= {"dw": s["dw"], "dy": s["dy"]}
        return out
    if c["op"] == "norm":
        mx = G.mx_out(row_q=s["q"], row_s=s["s"]) if c["mx"] else None
        G.moe_add_rmsnorm(s["x"], s["weight"], c["T"], c["H"], 1e-6, residual=s["residual"],
                          h=s["h"] if c["residual"] else None, y=s["y"], rstd=s["rstd"], mx=mx)
        out = {"h": s["h"], "y": s["y"], "rstd": s["rstd"]}
        if c["mx"]:
            out |= {"q": s["q"].view(torch.float8_e4m3fn), "s": s["s"].view(torch.float8_e8m0fnu)}
        if c["grad"]:
            G.moe_add_rmsnorm_bwd(s["dy"], s["h"], s["weight"], s["rstd"], c["T"], c["H"], dh=s["dh"],
                                  dx=s["dx"], dweight=s["dweight"], workspace=s["scratch"])
            out |= {"dx": s["dx"], "dweight": s["dweight"]}
        return out
    cap, K = s["x"].shape
    grp = G.groups(s["counts"], cap)
    if c["a"] == "fp4":
        G.moe_mxfp4_quantize(s["x"], cap, K, grp, s["aq"], s["as"])
    else:
        G.moe_mxfp8_quantize(s["x"], cap, K, grp, G.mx_out(row_q=s["aq"], row_s=s["as"]))
    a = G.operand(s["aq"], dtype=G.DT_MXFP4 if c["a"] == "fp4" else G.DT_MXFP8, scales=s["as"])
    b = G.operand(s["wq"], dtype=G.DT_MXFP4, layout=G.B_NK, scales=s["ws"])
    G.moe_group_gemm_quant(a, b, c["N"], K, grp, s["out"])
    return s["out"]


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    plain = {"router": _router_plain, "combine": _combine_plain, "norm": _norm_plain, "mxfp4": _mxfp4_plain}
    return plain[c["op"]](state, c)


# ----------------------------------------------------------------------------- what a pass needs
def work(case):
    c = case
    if c["op"] == "router":
        T, E, k = c["T"], c["E"], c["k"]
        size = 2 if c["bf16"] else 4
        b = T * E * size + T * k * 8 + (4 * E if c["bias"] else 0)
        if c["grad"]:
            b += T * E * size + T * k * 4
        return {"bytes": b, "flops": T * E * (8 if c["grad"] else 5)}
    if c["op"] == "combine":
        T, k, H = c["T"], c["k"], c["H"]
        rows = T * k * (1 - c["drop"])
        b = rows * H * 2 + T * H * 2 * (2 if c["residual"] else 1) + T * k * 8
        f = 2 * rows * H
        if c["grad"]:
            b += T * H * 2 + rows * H * 2 + T * k * 4
            f *= 2.5
        return {"bytes": b, "flops": f}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        b = T * H * (8 if c["residual"] else 4) + 2 * H + T * 4
        if c["mx"]:
            b += T * H + T * H // 32
        if c["grad"]:
            b += T * H * 6 + 4 * H
        return {"bytes": b, "flops": T * H * (14 if c["grad"] else 5)}
    E, N, K, M = c["E"], c["N"], c["K"], c["rows"]
    active = sum(1 for m in _group_sizes(M, E, c["skew"]) if m)
    return {"bytes": M * K * 2 + active * N * K * (0.5 + 1 / 32) + M * N * 2, "flops": 2 * M * N * K}


# ----------------------------------------------------------------------------- the definitions in 64 bits
def _router_exact(s, c):
    x = s["logits"].double().requires_grad_(c["grad"])
    score = x.softmax(1) if c["score"] == "softmax" else torch.sigmoid(x)
    with torch.no_grad():
        value = score + s["bias"].double() if c["bias"] else score
        closed = torch.zeros_like(value, dtype=torch.bool)
        if c["groups"] > 1:
            per = value.unflatten(1, (c["groups"], -1))
            best = per.topk(2 if c["top2"] else 1, 2).values.sum(2)
            lowest = best.argsort(dim=1, descending=True, stable=True)[:, c["keep"]:]
            shut = torch.zeros_like(best, dtype=torch.bool)
            shut[torch.arange(len(best), device=DEV)[:, None], lowest] = True
            closed = shut[..., None].expand_as(per).flatten(1)
        ids = (value.masked_fill(closed, -math.inf)).argsort(dim=1, descending=True, stable=True)[:, :c["k"]]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    out = {"ids": None, "weights": w.detach()}
    if c["grad"]:
        out["dlogits"], = torch.autograd.grad(w, x, s["dw"].double())
    return out


def _combine_exact(s, c):
    T, k, H = c["T"], c["k"], c["H"]
    pair = torch.nonzero(s["dst"].flatten() >= 0)[:, 0]
    row, tok = s["dst"].flatten()[pair].long(), pair // k
    w = s["w"].double().flatten()
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    out.index_add_(0, tok, s["y"].double()[row] * w[pair, None])
    if c["residual"]:
        out += s["residual"].double()
    got = {"out": out}
    if c["grad"]:
        d = s["dout"].double()[tok]
        dw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
        dw[pair] = torch.linalg.vecdot(d, s["y"].double()[row])
        dy = torch.zeros(T * k, H, dtype=torch.float64, device=DEV)
        dy[row] = d * w[pair, None]
        got |= {"dw": dw.view(T, k), "dy": dy}
    return got


def _norm_exact(s, c):
    h = s["x"].double()
    if c["residual"]:
        h = (h + s["residual"].double()).to(BF16).double()     # the residual stream is kept in bf16
    h.requires_grad_(c["grad"])
    weight = s["weight"].double().requires_grad_(c["grad"])
    rstd = 1 / torch.sqrt((h * h).mean(1) + 1e-6)
    y = h * rstd[:, None] * weight
    out = {"h": h.detach(), "y": y.detach(), "rstd": rstd.detach()}
    if c["mx"]:
        v = y.detach().to(BF16).double().unflatten(1, (-1, 32))
        amax = v.abs().amax(2)
        e = torch.floor(torch.log2(amax)) - 8
        e = e + (amax > 448 * torch.exp2(e))
        a = v.abs() / torch.exp2(e)[..., None]
        step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
        out |= {"s": torch.exp2(e), "q": (torch.sign(v) * torch.round(a / step) * step).flatten(1)}
    if c["grad"]:
        dx, dweight = torch.autograd.grad(y, (h, weight), s["dy"].double())
        out |= {"dx": dx + s["dh"].double(), "dweight": dweight}
    return out


def _mxfp4_exact(s, c):
    cap, K = s["x"].shape
    v = s["x"].double().unflatten(1, (-1, 32))
    amax = v.abs().amax(2)
    top, low = (6.0, 2) if c["a"] == "fp4" else (448.0, 8)
    e = torch.floor(torch.log2(amax)) - low
    e = e + (amax > top * torch.exp2(e))
    a = v.abs() / torch.exp2(e)[..., None]
    bits, least = (1, 0) if c["a"] == "fp4" else (3, -6)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** least))) - bits)
    x = (torch.sign(v) * torch.round(a / step) * step * torch.exp2(e)[..., None]).flatten(1)
    out = torch.zeros(cap, c["N"], dtype=torch.float64, device=DEV)
    value = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    at = 0
    for wq, ws, m in zip(s["wq"], s["ws"], s["sizes"]):
        code = torch.stack([wq % 16, wq // 16], 2).int()
        w = value[code % 8] * (1 - 2 * (code // 8))
        w = w.view(c["N"], -1, 32) * torch.exp2(ws.double() - 127)[..., None]
        out[at:at + m] = x[at:at + m] @ w.view(c["N"], K).t()
        at += m
    return out


def exact(case, seed):
    s = prepare(case, seed)
    form = {"router": _router_exact, "combine": _combine_exact, "norm": _norm_exact, "mxfp4": _mxfp4_exact}
    return form[case["op"]](s, case)
