"""A step of fine-tuning adapters beside a shared projection: grouping by adapter
ids, the projection, the adapters onto it, their gradients onto the projection's,
the norm of the gradients and the AdamW step; eagerly, in replayed graphs and on
two streams at once.

Each call is checked against the float64 oracle on the inputs that it had on the
GPU, with the tolerances of the operators' own tests (U = 2^-24, half a bf16 step
2^-8); replays and streams against the eager run from the same state, to the bit."""
import numpy as np
import pytest

import workloads as W
from oracle import formats as F
from oracle import training as P
from tests.gpu_util import dev_bits, host_bits
from tests.test_gpu_lora import G, TINY, U, bits  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
T_, L_, R_, K_, N_ = 192, 5, 16, 256, 192
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8)


class Step:
    """Weights, states and buffers of one adapted projection."""

    def __init__(self, G, seed, bits8):  # noqa: F811
        import torch
        rng = np.random.default_rng(seed)
        f32 = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
        bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        put = lambda a: dev_bits(a).view(torch.bfloat16)  # noqa: E731
        self.G, self.bits8 = G, bits8
        self.w = put(bits(rng, 1, K_, N_, std=K_ ** -0.5))
        self.master = {"A": torch.from_numpy((rng.standard_normal((L_, R_, K_)) * K_ ** -0.5).astype(np.float32)).cuda(),
                       "B": torch.from_numpy((rng.standard_normal((L_, N_, R_)) * 0.1).astype(np.float32)).cuda()}
        self.p = {k: m.bfloat16() for k, m in self.master.items()}
        self.g = {k: torch.empty_like(m) for k, m in self.master.items()}
        self.scale = torch.full((L_,), 0.5, device="cuda")
        self.x, self.dy, self.ids = bf(T_, K_), bf(T_, N_), i32(T_, 1)
        self.y, self.dx, self.u = bf(T_, N_), bf(T_, K_), f32(T_, R_)
        self.ids_out, self.counts, self.offsets, self.dst, self.src = i32(T_, 1), i32(L_), i32(L_ + 1), i32(T_, 1), i32(T_)
        self.all = torch.tensor([T_], dtype=torch.int32, device="cuda")
        need = max(G.moe_lora_fwd_workspace_bytes(T_, L_, R_, K_, N_), G.moe_lora_bwd_workspace_bytes(T_, L_, R_, K_, N_),
                   G.moe_grad_norm_workspace_bytes())
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        self.state, tensors = {}, []
        for k, m in self.master.items():
            n = m.numel()
            if bits8:
                st = dict(m=torch.zeros(n, dtype=torch.int8, device="cuda"), v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                          m_scale=f32((n + 127) // 128), v_scale=f32((n + 127) // 128))
            else:
                st = dict(m=f32(n), v=f32(n))
            self.state[k] = st
            tensors.append(G.adamw_tensor(self.p[k], self.g[k], st["m"], st["v"], master=m, m_scale=st.get("m_scale"),
                                          v_scale=st.get("v_scale"), weight_decay=0.1))
        self.plan = G.adamw_plan(tensors)
        self.step, self.out = torch.ones(1, dtype=torch.int32, device="cuda"), f32(2)
        self.hyper = G.adamw(**HYPER, step_dev=self.step, grad_scale=self.out[1:])
        self.groups, self.one = G.groups(self.counts, T_), G.groups(self.all, T_)
        self.lora = G.lora(self.p["A"], self.p["B"], R_, K_, N_, scale=self.scale)

    def feed(self, seed):
        import torch
        rng = np.random.default_rng(seed)
        self.x.copy_(dev_bits(bits(rng, T_, K_)).view(torch.bfloat16))
        self.dy.copy_(dev_bits(bits(rng, T_, N_, std=0.2)).view(torch.bfloat16))
        ids = rng.integers(-1, L_ - 1, T_)               # some without an adapter; the last adapter has no rows
        self.ids.copy_(torch.from_numpy(ids.astype(np.int32).reshape(T_, 1)))

    def __call__(self, stream=None):
        G, s = self.G, stream  # noqa: F811
        G.moe_route_group(None, self.ids, T_, L_, 1, self.ids_out, self.counts, self.offsets, self.dst, self.src, stream=s)
        G.moe_group_gemm_quant(G.operand(self.x), G.operand(self.w, layout=G.B_KN), N_, K_, self.one, self.y, stream=s)
        G.moe_lora_fwd(self.x, T_, self.groups, self.lora, self.y, base=self.y, src=self.src, u=self.u, workspace=self.ws, stream=s)
        G.moe_group_gemm_quant(G.operand(self.dy), G.operand(self.w, layout=G.B_NK), K_, N_, self.one, self.dx, stream=s)
        G.moe_lora_bwd(self.dy, self.x, T_, self.groups, self.lora, self.u, dx=self.dx, dx_base=self.dx, dA=self.g["A"],
                       dB=self.g["B"], src=self.src, workspace=self.ws, stream=s)
        G.moe_grad_norm(self.plan, 1.0, self.out, self.ws, stream=s)
        G.moe_adamw_step(self.plan, self.hyper, stream=s)

    def tensors(self):
        out = [self.y, self.dx, self.u, self.out, self.counts, self.src]
        for k in ("A", "B"):
            out += [self.p[k], self.master[k], self.g[k]] + list(self.state[k].values())
        return out

    def snapshot(self):
        import torch
        torch.cuda.synchronize()
        return [t.clone().view(torch.uint8) if t.dim() else t.clone() for t in self.tensors()]


def _same(a, b):
    import torch
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), i


def _u16(t):
    import torch
    return host_bits(t.view(torch.int16))


@pytest.mark.parametrize("bits8", [False, True])
def test_step_by_step(G, bits8):  # noqa: F811
    """Three steps, each call against the oracle."""
    import torch
    s = Step(G, 1, bits8)
    for step in range(1, 4):
        s.feed(step)
        before = {k: (s.master[k].cpu().numpy().ravel().astype(np.float64), {n: t.cpu().numpy() for n, t in s.state[k].items()})
                  for k in ("A", "B")}
        A, B = _u16(s.p["A"]), _u16(s.p["B"])
        s()
        torch.cuda.synchronize()
        counts, src, x, dy = s.counts.cpu().numpy(), s.src.cpu().numpy(), _u16(s.x), _u16(s.dy)
        ids = s.ids.cpu().numpy()[:, 0]
        assert counts.tolist() == [int(np.sum(ids == e)) for e in range(L_)] and counts[-1] == 0
        # projection and adapters: the projection's output is rounded to bf16 once before the adapters' sum
        w = F.bf16_bits_to_f64(_u16(s.w))[0]
        sc = np.full(L_, 0.5, np.float32)
        u, add = P.lora_fwd(x, A, B, sc, counts, T_, src)
        plain = F.bf16_bits_to_f64(x) @ w
        mag_u, mag_add = P.lora_fwd(x & 0x7FFF, A & 0x7FFF, B & 0x7FFF, sc, counts, T_, src)
        add, mag_add = np.nan_to_num(add), np.nan_to_num(mag_add)
        tol = (2.0 ** -8 * np.abs(plain) + 2.0 ** -8 * np.abs(plain + add)) * 1.02 + (2.0 ** -17 + 2 * K_ * U) * mag_add \
            + K_ * U * (np.abs(F.bf16_bits_to_f64(x)) @ np.abs(w)) + TINY
        assert np.all(np.abs(F.bf16_bits_to_f64(_u16(s.y)) - plain - add) <= tol)
        held = ~np.isnan(u[:, 0])
        got_u = s.u.cpu().numpy()
        assert np.all(np.abs(got_u - u)[held] <= ((K_ + 8) * U * mag_u + TINY)[held])
        # gradients, from the u that the call had
        ug = np.where(held[:, None], got_u, 0).astype(np.float32)
        dadd, dA, dB, wv = P.lora_bwd(dy, x, A, B, sc, counts, T_, ug, src)
        m_dx, m_dA, m_dB, m_w = P.lora_bwd(dy & 0x7FFF, x & 0x7FFF, A & 0x7FFF, B & 0x7FFF, sc, counts, T_, np.abs(ug), src)
        dplain = F.bf16_bits_to_f64(dy) @ w.T
        dadd, m_dx = np.nan_to_num(dadd), np.nan_to_num(m_dx)
        tol = (2.0 ** -8 * np.abs(dplain) + 2.0 ** -8 * np.abs(dplain + dadd)) * 1.02 + (2.0 ** -17 + 2 * N_ * U) * m_dx \
            + N_ * U * (np.abs(F.bf16_bits_to_f64(dy)) @ np.abs(w.T)) + TINY
        assert np.all(np.abs(F.bf16_bits_to_f64(_u16(s.dx)) - dplain - dadd) <= tol)
        m = counts[:, None, None].astype(np.float64)
        gA, gB = s.g["A"].cpu().numpy().astype(np.float64), s.g["B"].cpu().numpy().astype(np.float64)
        assert np.all(np.abs(gA - dA) <= (3 * m + N_ + 32) * U * m_dA + TINY)
        assert np.all(np.abs(gB - dB) <= (3 * m + 16) * U * m_dB + TINY)
        assert np.all(gA[-1] == 0) and np.all(gB[-1] == 0)
        # norm and step, from the gradients that they had
        norm, factor = P.grad_norm([gA, gB], 1.0)
        out = s.out.cpu().numpy()
        assert abs(out[0] - norm) <= 1.01 * U * norm and abs(out[1] - factor) <= 2.01 * U * factor and factor < 1
        for k, g in (("A", gA), ("B", gB)):
            p0, st = before[k]
            m0, v0 = P.state8_decode(st["m"], st["m_scale"], st["v"], st["v_scale"]) if bits8 else \
                (st["m"].astype(np.float64), st["v"].astype(np.float64))
            decay = float(np.float32(0.1))
            p, m1, v1 = P.adamw(p0, g.ravel(), m0, v0, HYPER["lr"], 0.9, 0.99, 1e-8, step, decay, float(out[1]))
            denom = np.sqrt(v1 / (1 - 0.99 ** step)) + 1e-8
            coef = HYPER["lr"] / (1 - 0.9 ** step)
            tol_m = 4 * U * (np.abs(0.9 * m0) + np.abs(0.1 * g.ravel() * float(out[1]))) + 1e-44
            update = np.abs(p0 * (1 - HYPER["lr"] * decay) - p)
            tol = 4 * U * np.abs(p0) + coef * tol_m / denom + 20 * U * update + U * np.abs(p) + 1e-44
            got = s.master[k].cpu().numpy().ravel()
            assert np.all(np.abs(got - p) <= tol), k
            assert np.array_equal(_u16(s.p[k]).ravel(), W.to_bf16_bits(got))
        s.step += 1


@pytest.mark.parametrize("bits8", [False, True])
def test_replayed_graph(G, bits8):  # noqa: F811
    """The whole step captured once and replayed on new inputs, with eager work between the replays, against the eager
    step from the same state."""
    import torch
    eager, graphed = Step(G, 2, bits8), Step(G, 2, bits8)
    for s in (eager, graphed):
        s.feed(100)
        s()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            graphed(stream=side.cuda_stream)
    torch.cuda.synchronize()
    for i in range(5):
        for s in (eager, graphed):
            s.feed(200 + i)
            s.step += 1
        eager()
        g.replay()
        a, b = eager.snapshot(), graphed.snapshot()
        _same(a, b)
        torch.randn(1000, 1000, device="cuda").sum().item()


def test_two_streams(G):  # noqa: F811
    """Two steps of their own at the same time, and each alone, give the same bits."""
    import torch
    alone = []
    for seed in (3, 4):
        s = Step(G, seed, seed == 4)
        for i in range(6):
            s.feed(10 * seed + i)
            s()
            s.step += 1
            torch.cuda.synchronize()
        alone.append(s.snapshot())
    both = [Step(G, 3, False), Step(G, 4, True)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(6):
        for s, st, seed in zip(both, streams, (3, 4)):
            with torch.cuda.stream(st):
                s.feed(10 * seed + i)
                s()
                s.step += 1
    torch.cuda.synchronize()
    for s, a in zip(both, alone):
        _same(s.snapshot(), a)


def test_adapters_of_experts(G):  # noqa: F811
    """One adapter for each expert on the grouped rows: the expert products' own counts, no src."""
    import torch
    rng = np.random.default_rng(5)
    E, M, K, N, r = 4, 150, 128, 192, 24
    counts = np.array([70, 0, 50, 20], np.int32)
    x, w = bits(rng, M, K), bits(rng, E, K, N, std=K ** -0.5)
    A, B = bits(rng, E, r, K, std=K ** -0.5), bits(rng, E, N, r, std=r ** -0.5)
    grp = G.groups(torch.from_numpy(counts).cuda(), M)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    G.moe_group_gemm_quant(G.operand(dev_bits(x)), G.operand(dev_bits(w), layout=G.B_KN), N, K, grp, y)
    base = _u16(y)
    ws = torch.empty(G.moe_lora_fwd_workspace_bytes(M, E, r, K, N), dtype=torch.uint8, device="cuda")
    G.moe_lora_fwd(dev_bits(x), M, grp, G.lora(dev_bits(A), dev_bits(B), r, K, N), y, base=y, workspace=ws)
    torch.cuda.synchronize()
    _, want = P.lora_fwd(x, A, B, None, counts, M, None, base)
    _, mag = P.lora_fwd(x & 0x7FFF, A & 0x7FFF, B & 0x7FFF, None, counts, M)
    got = F.bf16_bits_to_f64(_u16(y))
    assert np.all(np.abs(got - want)[:140] <= (2.0 ** -8 * 1.01 * np.abs(want) + (2.0 ** -17 + 2 * K * U) * mag + TINY)[:140])
    assert np.all(got[140:] == 7)
