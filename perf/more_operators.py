"""Timed cases of what adapts and trains the weights of the library's products.

  lora   low-rank adapters of many requests beside a shared projection, with their gradients
  adamw  an AdamW step over many tensors at once, states in 32 or in 8 bits
  norm   the norm of all gradients, and the factor that clips them

``listed`` and ``draw`` give cases, ``prepare`` their inputs on the GPU, ``run`` one pass (in plain
torch operations, or with ``own`` set the library's kernels), ``work`` what a pass has to move and
compute, ``exact`` the outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16
BLOCK = 128        # elements that share the scales of an 8-bit state
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.01, 20


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one request decoding with an adapter: latency of a call
        dict(name="lora one token", op="lora", T=1, L=8, r=16, K=7168, N=4096, none=0.0, skew=0.0, direct=False,
             grad=False),
        # a decoding batch of 64 requests over 32 adapters, some without one
        dict(name="lora tokens", op="lora", T=64, L=32, r=16, K=2880, N=5760, none=0.1, skew=0.5, direct=False,
             grad=False),
        # prompts of several requests, 8 adapters of rank 64
        dict(name="lora prompt", op="lora", T=16384, L=8, r=64, K=7168, N=4096, none=0.1, skew=0.5, direct=False,
             grad=False),
        # fine-tuning one adapter, an odd token count, forward and backward
        dict(name="lora train", op="lora", T=8191, L=1, r=16, K=2880, N=5760, none=0.0, skew=0.0, direct=False,
             grad=True),
        # an adapter for each of 32 experts, on the grouped rows themselves, forward and backward
        dict(name="lora experts train", op="lora", T=16384, L=32, r=32, K=7168, N=4096, none=0.0, skew=1.1,
             direct=True, grad=True),
        # the step over the adapters of one projection (16 tensors), bf16 weights with fp32 masters
        dict(name="adamw adapters", op="adamw", tensors=16, low=46080, high=92160, bits=32, param="master",
             bf16_grad=False),
        # a model's small tensors, of any size, states in 8 bits
        dict(name="adamw many 8 bits", op="adamw", tensors=300, low=1, high=60000, bits=8, param="bf16",
             bf16_grad=True),
        # the first weights of 32 experts
        dict(name="adamw experts", op="adamw", tensors=32, low=16588800, high=16588800, bits=32, param="master",
             bf16_grad=False),
        # the second weights of 32 experts, states in 8 bits
        dict(name="adamw experts 8 bits", op="adamw", tensors=32, low=8294400, high=8294400, bits=8, param="master",
             bf16_grad=False),
        # the norm of many small gradients
        dict(name="norm many", op="norm", tensors=300, low=1, high=60000, bf16_grad=True),
        # the norm of the gradients of 32 experts' second weights
        dict(name="norm experts", op="norm", tensors=32, low=8294400, high=8294400, bf16_grad=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["lora", "lora", "adamw", "norm"])
    if op == "lora":
        return dict(op=op, T=_spread(rng, 1, 16384), L=_spread(rng, 1, 32), r=rng.choice([8, 16, 24, 32, 64, 128]),
                    K=8 * _spread(rng, 8, 896), N=8 * _spread(rng, 8, 896), none=rng.choice([0.0, 0.1, 0.5]),
                    skew=rng.choice([0.0, 0.5, 1.1]), direct=rng.random() < 0.3, grad=rng.random() < 0.6)
    low, high = sorted((_spread(rng, 1, 200000), _spread(rng, 1, 200000)))
    c = dict(op=op, tensors=_spread(rng, 1, 400), low=low, high=high, bf16_grad=rng.random() < 0.5)
    if op == "adamw":
        c |= dict(bits=rng.choice([8, 32]), param=rng.choice(["bf16", "fp32", "master"]))
    return c


def _group_sizes(rows, L, skew):
    """Group sizes that sum to ``rows``, the i-th in proportion to (i + 1)^-skew (largest remainders up)."""
    w = [(i + 1) ** -skew for i in range(L)]
    quota = [rows * v / sum(w) for v in w]
    size = [int(q) for q in quota]
    for i in sorted(range(L), key=lambda i: (size[i] - quota[i], i))[:rows - sum(size)]:
        size[i] += 1
    return size


def _adapted(c):
    """Rows that have an adapter; at least one."""
    return max(1, c["T"] - int(c["none"] * c["T"]))


def _tensor_sizes(c):
    """Sizes from low to high, spread over their logarithm, in no order."""
    ratio = math.log(c["high"] / c["low"])
    return [min(c["high"], int(c["low"] * math.exp(ratio * (i * 0.6180339887498949 % 1.0)) + 0.5))
            for i in range(c["tensors"])]


# ----------------------------------------------------------------------------- inputs
def _normal(g, *shape, std=1.0, dtype=BF16):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "lora":
        T, L, r, K, N = c["T"], c["L"], c["r"], c["K"], c["N"]
        M = _adapted(c)
        sizes = _group_sizes(M, L, c["skew"])
        s["sizes"] = [sizes[p] for p in torch.randperm(L, generator=g, device=DEV).tolist()]
        s["counts"] = torch.tensor(s["sizes"], dtype=torch.int32, device=DEV)
        # the rows of each adapter in ascending order, as the grouping leaves them; behind them none
        at = torch.arange(T, device=DEV) if c["direct"] else torch.randperm(T, generator=g, device=DEV)
        at = torch.cat([p.sort().values for p in at[:M].split(s["sizes"])])
        s["rows"] = at
        s["src"] = torch.full((T,), -1, dtype=torch.int32, device=DEV)
        s["src"][:M] = at.int()
        s["x"] = _normal(g, T, K)
        s["A"] = _normal(g, L, r, K, std=K ** -0.5)
        s["B"] = _normal(g, L, N, r, std=0.3 * r ** -0.5)
        s["scale"] = torch.rand(L, generator=g, device=DEV) + 0.5
        s["base"] = _normal(g, T, N)                    # the shared projection's output
        s["y"] = s["base"].clone()                      # rows without an adapter stay
        s["u"] = torch.zeros(T, r, dtype=torch.float32, device=DEV)
        if c["grad"]:
            s["dy"] = _normal(g, T, N, std=0.01)
            s["dx_base"] = _normal(g, T, K, std=0.01)   # the gradient through the shared projection
            s["dx"] = s["dx_base"].clone()
            s["dA"] = torch.empty(L, r, K, dtype=torch.float32, device=DEV)
            s["dB"] = torch.empty(L, N, r, dtype=torch.float32, device=DEV)
        if own:
            import grouped_gemm_glu_amd as G
            need = G.moe_lora_fwd_workspace_bytes(T, L, r, K, N)
            if c["grad"]:
                need = max(need, G.moe_lora_bwd_workspace_bytes(T, L, r, K, N))
            s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
        return s
    # the tensors lie in flat buffers, each from a block's start; what is between them is zero
    sizes = _tensor_sizes(c)
    blocks = [-(-n // BLOCK) for n in sizes]
    total = BLOCK * sum(blocks)
    start, at = [], 0
    for b in blocks:
        start.append(at)
        at += BLOCK * b
    begin = torch.tensor(start, device=DEV).repeat_interleave(torch.tensor(blocks, device=DEV), output_size=total // BLOCK)
    end = torch.tensor([a + n for a, n in zip(start, sizes)], device=DEV).repeat_interleave(
        torch.tensor(blocks, device=DEV), output_size=total // BLOCK)
    inside = (torch.arange(total, device=DEV).view(-1, BLOCK) < end[:, None]).view(-1) if total != sum(sizes) else None
    fill = (lambda t: t) if inside is None else (lambda t: t.mul_(inside))
    spread = torch.exp(torch.randn(total // BLOCK, 1, generator=g, device=DEV))   # gradients of uneven size
    grad = fill(torch.randn(total, generator=g, device=DEV).view(-1, BLOCK).mul_(1e-3 * spread).view(-1))
    s["grad"] = grad.to(BF16) if c["bf16_grad"] else grad
    pieces = [(a, n) for a, n in zip(start, sizes)]
    if c["op"] == "norm":
        s["out"] = torch.zeros(2, dtype=torch.float32, device=DEV)
    s["grad_scale"] = torch.rand(1, generator=g, device=DEV) * 0.5 + 0.5          # as clipping leaves it
    p = fill(_normal(g, total, std=0.02, dtype=torch.float32)) if c["op"] == "adamw" else None
    if c["op"] == "adamw":
        s["decay"] = torch.tensor([DECAY if n > 1000 else 0.0 for n in sizes], device=DEV).repeat_interleave(
            torch.tensor(blocks, device=DEV), output_size=total // BLOCK)[:, None]  # small tensors: none
        if c["param"] == "fp32":
            s["param"], s["master"] = p, None
        else:
            s["param"] = p.to(BF16)
            s["master"] = p if c["param"] == "master" else None
        m = fill(torch.randn(total, generator=g, device=DEV).view(-1, BLOCK).mul_(3e-4 * spread).view(-1))
        v = torch.randn(total, generator=g, device=DEV).square_().view(-1, BLOCK).mul_(1e-6 * spread * spread).view(-1)
        v = fill(v)
        if c["bits"] == 32:
            s["m"], s["v"], s["m_scale"], s["v_scale"] = m, v, None, None
        else:
            s["m"], s["v"], s["m_scale"], s["v_scale"] = _encode(m.double(), v.double())
            del m, v
            s["m_out"] = torch.empty(total, dtype=torch.float32, device=DEV)
            s["v_out"] = torch.empty(total, dtype=torch.float32, device=DEV)
    if own:
        import grouped_gemm_glu_amd as G
        cut = lambda name, a, n: None if s.get(name) is None else s[name][a:a + n]  # noqa: E731
        scales = lambda name, a, n: None if s.get(name) is None else s[name][a // BLOCK:-(-(a + n) // BLOCK)]  # noqa: E731
        if c["op"] == "adamw":
            tensors = [G.adamw_tensor(cut("param", a, n), cut("grad", a, n), cut("m", a, n), cut("v", a, n),
                                      master=cut("master", a, n), m_scale=scales("m_scale", a, n),
                                      v_scale=scales("v_scale", a, n), weight_decay=DECAY if n > 1000 else 0.0)
                       for a, n in pieces]
        else:
            tensors = [G.adamw_tensor(None, cut("grad", a, n), None, None) for a, n in pieces]
            s["workspace"] = torch.empty(G.moe_grad_norm_workspace_bytes(), dtype=torch.uint8, device=DEV)
        s["plan"] = G.adamw_plan(tensors)
    return s


# ----------------------------------------------------------------------------- plain forms
def _lora_plain(s, c):
    at, sizes = s["rows"], s["sizes"]
    scale = s["scale"].repeat_interleave(s["counts"], output_size=len(at))[:, None]
    groups = [e for e in range(c["L"]) if sizes[e]]
    x = s["x"][at].float()
    cut = [p for p in x.split(sizes) if len(p)]
    A, B = s["A"].float(), s["B"].float()
    u = torch.cat([p @ A[e].t() for e, p in zip(groups, cut)])
    cut_u = [p for p in u.split(sizes) if len(p)]
    add = torch.cat([p @ B[e].t() for e, p in zip(groups, cut_u)])
    s["y"][at] = (s["base"][at].float() + scale * add).to(BF16)
    s["u"][:len(at)] = u
    out = {"y": s["y"], "u": s["u"]}
    if c["grad"]:
        dy = s["dy"][at].float() * scale
        cut_dy = [p for p in dy.split(sizes) if len(p)]
        w = [p @ B[e] for e, p in zip(groups, cut_dy)]
        s["dx"][at] = (s["dx_base"][at].float() + torch.cat([p @ A[e] for e, p in zip(groups, w)])).to(BF16)
        where = torch.tensor(groups, device=DEV)
        s["dA"].zero_()[where] = torch.stack([p.t() @ q for p, q in zip(w, cut)])
        s["dB"].zero_()[where] = torch.stack([p.t() @ q for p, q in zip(cut_dy, cut_u)])
        out |= {"dx": s["dx"], "dA": s["dA"], "dB": s["dB"]}
    return out


def _decode(s):
    """The states in 64 bits from their codes: m = sign(c) (c / 127)^2 m_scale, sqrt(v) = (c / 255)^2 v_scale."""
    cm, cv = s["m"].view(-1, BLOCK).double(), s["v"].view(-1, BLOCK).double()
    m = cm * cm.abs() / 127 ** 2 * s["m_scale"].double()[:, None]
    root = cv.square() / 255 ** 2 * s["v_scale"].double()[:, None]
    return m.view(-1), root.square().view(-1)


def _encode(m, v):
    """Codes and scales of states in 64 bits: the nearest code under the square root, the lower one of two as near;
    a v above zero never gets code 0."""
    m, root = m.view(-1, BLOCK), torch.sqrt(v).view(-1, BLOCK)
    m_scale, v_scale = m.abs().amax(1).float(), root.amax(1).float()

    def nearest(value, scale, top):
        x = torch.sqrt(value / torch.where(scale > 0, scale, 1.0).double()[:, None]) * top
        return torch.ceil(x - 0.5).clamp(0, top)
    cm = nearest(m.abs(), m_scale, 127) * torch.sign(m)
    cv = torch.where((root > 0) & (v_scale > 0)[:, None], nearest(root, v_scale, 255).clamp(min=1), 0.0)
    return cm.to(torch.int8).view(-1), cv.to(torch.uint8).view(-1), m_scale, v_scale


def _adamw_plain(s, c):
    wide = c["bits"] == 8          # 64 bits where they decide between two codes
    f = torch.float64 if wide else torch.float32
    m, v = _decode(s) if wide else (s["m"], s["v"])
    g = s["grad"].to(f) * s["grad_scale"].to(f)
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    del g
    if wide:
        s["m"][:], s["v"][:], s["m_scale"][:], s["v_scale"][:] = _encode(m, v)
    else:
        s["m"][:], s["v"][:] = m, v
    update = m.float() * (LR / (1 - BETA1 ** STEP)) / (torch.sqrt(v.float() * (1 / (1 - BETA2 ** STEP))) + EPS)
    p = (s["param"] if s["master"] is None else s["master"]).float().view(-1, BLOCK)
    p = (p * (1 - LR * s["decay"])).view(-1) - update
    if s["master"] is not None:
        s["master"][:] = p
    s["param"][:] = p.to(s["param"].dtype)
    out = {"param": s["param"], "m": s["m"], "v": s["v"]}
    if s["master"] is not None:
        out["master"] = s["master"]
    if wide:
        m, v = _decode(s)
        s["m_out"][:], s["v_out"][:] = m.float(), v.float()
        out |= {"m": s["m_out"], "v": s["v_out"]}
    return out


def _norm_plain(s, c):
    norm = torch.sqrt(s["grad"].double().square().sum())
    s["out"][0] = norm
    s["out"][1] = (1.0 / (norm + 1e-6)).clamp(max=1.0)
    return {"norm": s["out"][:1], "factor": s["out"][1:]}


# ----------------------------------------------------------------------------- one pass
def _run_own(s, c):
    import grouped_gemm_glu_amd as G
    if c["op"] == "lora":
        grp = G.groups(s["counts"], c["T"])
        src = None if c["direct"] else s["src"]
        lora = G.lora(s["A"], s["B"], c["r"], c["K"], c["N"], scale=s["scale"])
        G.moe_lora_fwd(s["x"], c["T"], grp, lora, s["y"], base=s["base"], src=src, u=s["u"],
                       workspace=s["workspace"])
        out = {"y": s["y"], "u": s["u"]}
        if c["grad"]:
            G.moe_lora_bwd(s["dy"], s["x"], c["T"], grp, lora, s["u"], dx=s["dx"], dx_base=s["dx_base"], dA=s["dA"],
                           dB=s["dB"], src=src, workspace=s["workspace"])
            out |= {"dx": s["dx"], "dA": s["dA"], "dB": s["dB"]}
        return out
    if c["op"] == "adamw":
        G.moe_adamw_step(s["plan"], G.adamw(LR, BETA1, BETA2, EPS, step=STEP, grad_scale=s["grad_scale"]))
        out = {"param": s["param"], "m": s["m"], "v": s["v"]}
        if s["master"] is not None:
            out["master"] = s["master"]
        if c["bits"] == 8:
            G.moe_adamw_unpack(s["m"], s["m_scale"], s["v"], s["v_scale"], s["m"].numel(), s["m_out"], s["v_out"])
            out |= {"m": s["m_out"], "v": s["v_out"]}
        return out
    G.moe_grad_norm(s["plan"], 1.0, s["out"], s["workspace"])
    return {"norm": s["out"][:1], "factor": s["out"][1:]}


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    plain = {"lora": _lora_plain, "adamw": _adamw_plain, "norm": _norm_plain}
    return plain[c["op"]](state, c)


# ----------------------------------------------------------------------------- what a pass needs
def work(case):
    c = case
    if c["op"] == "lora":
        r, K, N, M = c["r"], c["K"], c["N"], _adapted(c)
        active = sum(1 for m in _group_sizes(M, c["L"], c["skew"]) if m)
        weights = active * r * (K + N)
        b = 2 * M * K + 4 * M * N + 2 * weights + 4 * M * r + 4 * M
        f = 2 * M * r * (K + N)
        if c["grad"]:
            b += 2 * M * N + 6 * M * K + 2 * weights + 4 * c["L"] * r * (K + N) + 4 * M * r
            f *= 3
        return {"bytes": b, "flops": f}
    n = sum(_tensor_sizes(c))
    b = n * (2 if c["bf16_grad"] else 4)
    if c["op"] == "norm":
        return {"bytes": b, "flops": 2 * n}
    b += n * {"bf16": 4, "fp32": 8, "master": 10}[c["param"]]
    # states read and written; those of 8 bits read out once more, in 32
    b += n * (16 if c["bits"] == 32 else 4 + 16 / BLOCK + 8)
    return {"bytes": b, "flops": 16 * n}


# ----------------------------------------------------------------------------- the definitions in 64 bits
def _lora_exact(s, c):
    M = len(s["rows"])
    y, u = s["base"].double(), s["u"].double()
    out = {"y": y, "u": u}
    if c["grad"]:
        out |= {"dx": s["dx_base"].double(), "dA": torch.zeros(s["dA"].shape, dtype=torch.float64, device=DEV),
                "dB": torch.zeros(s["dB"].shape, dtype=torch.float64, device=DEV)}
    first = 0
    for e, m in enumerate(s["sizes"]):
        if m == 0:
            continue
        rows = s["rows"][first:first + m]
        x, a, b = s["x"][rows].double(), s["A"][e].double(), s["B"][e].double()
        k = s["scale"][e].double()
        low = torch.matmul(x, a.transpose(0, 1))
        u[first:first + m] = low
        y[rows] += k * torch.matmul(low, b.transpose(0, 1))
        if c["grad"]:
            dy = s["dy"][rows].double()
            back = k * torch.matmul(dy, b)
            out["dx"][rows] += torch.matmul(back, a)
            out["dA"][e] = torch.matmul(back.transpose(0, 1), x)
            out["dB"][e] = k * torch.matmul(dy.transpose(0, 1), low)
        first += m
    assert first == M
    return out


def _adamw_exact(s, c):
    g = s["grad"].double() * s["grad_scale"].double()
    if c["bits"] == 8:
        level = torch.arange(256, dtype=torch.float64, device=DEV)
        m = (level.square() / 127.0 ** 2)[s["m"].int().abs()] * torch.sign(s["m"].double())
        m = m * s["m_scale"].double().repeat_interleave(BLOCK)
        v = ((level / 255.0) ** 4)[s["v"].int()] * s["v_scale"].double().square().repeat_interleave(BLOCK)
    else:
        m, v = s["m"].double(), s["v"].double()
    m, v = m * BETA1 + g * (1.0 - BETA1), v * BETA2 + g.square() * (1.0 - BETA2)
    old = (s["master"] if c["param"] == "master" else s["param"]).double()
    denominator = torch.sqrt(v / (1.0 - BETA2 ** STEP)) + EPS
    p = old - LR * s["decay"].double().expand(-1, BLOCK).reshape(-1) * old - LR * (m / (1.0 - BETA1 ** STEP)) / denominator
    out = {"param": p}
    if c["param"] == "master":
        out["master"] = p
    if c["bits"] == 8:
        # the nearest of the code's values, measured under the square root, by the borders between neighbours
        def held(value, top, least):
            per = value.view(-1, BLOCK)
            scale = per.amax(1, keepdim=True).float().double()
            border = ((torch.arange(top, dtype=torch.float64, device=DEV) + 0.5) / top).square()
            code = torch.bucketize(per / torch.where(scale > 0, scale, torch.ones_like(scale)), border)
            code = torch.where(per > 0, code.clamp(min=least), 0)
            return ((code.double() / top).square() * scale).view(-1)
        out["m"] = held(m.abs(), 127, 0) * torch.sign(m)
        out["v"] = held(torch.sqrt(v), 255, 1).square()
    else:
        out["m"], out["v"] = m, v
    return out


def _norm_exact(s, c):
    norm = torch.linalg.vector_norm(s["grad"].double())
    return {"norm": norm.reshape(1), "factor": torch.clamp(1.0 / (norm + 1e-6), max=1.0).reshape(1)}


def exact(case, seed):
    s = prepare(case, seed)
    form = {"lora": _lora_exact, "adamw": _adamw_exact, "norm": _norm_exact}
    return form[case["op"]](s, case)
