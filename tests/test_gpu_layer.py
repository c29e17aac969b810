"""The operators together, as a layer uses them: residual addition + norm,
router, grouping, expert products, combine onto the residual; with MXFP4
experts for serving, and with the gradients of every step for training.

Each step is checked against the float64 oracle on the inputs that the step
had on the GPU, so that the tolerances are those of one step (u = 2^-24): the
norm's, the router's, the product's and the combine's as in the operators' own
tests, the GLU's that of gpu_util.  The gradient of the whole chain is checked
against float64 differentiation with the routing held: a path passes at most 12
roundings to bf16, each of at most 2^-8 of the vector it rounds, so the
vectors' errors stay within 12 * 2^-8 of the sizes that the formulas add up."""
import numpy as np
import pytest

import workloads as W
from oracle import formats as F
from oracle import moe as O
from oracle import operators as P
from tests.gpu_util import BF16_NAN_SENTINEL, assert_bf16_close, dev_bits, empty_bits, empty_bytes, host_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
E_, K_, H_, I_ = 16, 3, 256, 192
EPS = 1e-5
ROUTER = dict(score="sigmoid", n_groups=4, topk_groups=2, group_score="top2", renorm=True, scale=2.5)


@pytest.fixture(scope="module")
def G():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_gemm_glu_amd as G
    G.moe_init(0)
    return G


def _bits(rng, *shape, std=1.0):
    return W.to_bf16_bits((rng.standard_normal(shape) * std).astype(np.float32))


class Weights:
    def __init__(self, G):
        rng = np.random.default_rng(5)
        E, H, I = E_, H_, I_
        self.norm_h = _bits(rng, H, std=0.3)
        self.w1_h, self.w2_h = _bits(rng, E, H, 2 * I, std=0.08), _bits(rng, E, I, H, std=0.08)
        self.bias_h = (rng.standard_normal(E) * 0.1).astype(np.float32)
        import torch
        self.norm, self.w1, self.w2 = dev_bits(self.norm_h), dev_bits(self.w1_h), dev_bits(self.w2_h)
        self.bias = torch.from_numpy(self.bias_h).cuda()
        self.router = G.router(bias=self.bias, **ROUTER)
        self.ep = G.epilogue("swiglu")
        self.q1, self.s1 = empty_bytes((E, 2 * I, H // 2)), empty_bytes((E, 2 * I, H // 32))
        self.q2, self.s2 = empty_bytes((E, H, I // 2)), empty_bytes((E, H, I // 32))
        G.moe_pack_weight_mxfp4(self.w1, E, 2 * I, H, G.B_KN, self.q1, self.s1)
        G.moe_pack_weight_mxfp4(self.w2, E, H, I, G.B_KN, self.q2, self.s2)
        torch.cuda.synchronize()
        self.v1 = P.mxfp4_dequantize_rows(self.q1.cpu().numpy(), self.s1.cpu().numpy())
        self.v2 = P.mxfp4_dequantize_rows(self.q2.cpu().numpy(), self.s2.cpu().numpy())


@pytest.fixture(scope="module")
def weights(G):
    return Weights(G)


class Serving:
    """One layer's buffers for T tokens, the last `pad` of them padding."""

    def __init__(self, G, w, T, pad, seed):
        import torch
        self.G, self.w, self.T, self.pad = G, w, T, pad
        E, k, H, I, M = E_, K_, H_, I_, T * K_
        self.x, self.res, self.logits = empty_bits((T, H)), empty_bits((T, H)), torch.empty(T, E, device="cuda")
        self.h, self.y = empty_bits((T, H)), empty_bits((T, H))
        self.ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
        self.pairs = torch.empty(T, k, dtype=torch.int32, device="cuda")
        self.used = torch.empty(T, k, dtype=torch.int32, device="cuda")
        self.p = torch.empty(T, k, device="cuda")
        self.counts = torch.empty(E, dtype=torch.int32, device="cuda")
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        self.dst = torch.empty(T, k, dtype=torch.int32, device="cuda")
        self.src = torch.empty(M, dtype=torch.int32, device="cuda")
        self.no_id = torch.tensor(-1, dtype=torch.int32, device="cuda")
        self.keep = (torch.arange(T, device="cuda") < T - pad)[:, None]
        self.xg, self.z, self.a, self.y2 = (empty_bits((M, n)) for n in (H, 2 * I, I, H))
        self.xq, self.xs = empty_bytes((M, H // 2)), empty_bytes((M, H // 32))
        self.aq, self.as_ = empty_bytes((M, I // 2)), empty_bytes((M, I // 32))
        self.out = empty_bits((T, H))
        self.grp = G.groups(self.counts, M)
        op = lambda q, s, **kw: G.operand(q, dtype=G.DT_MXFP4, scales=s, **kw)  # noqa: E731
        self.ops = (op(self.xq, self.xs), op(w.q1, w.s1, layout=G.B_NK), op(self.aq, self.as_), op(w.q2, w.s2, layout=G.B_NK))
        self.load(seed)

    def load(self, seed):
        import torch
        rng = np.random.default_rng(seed)
        self.x_h, self.res_h = _bits(rng, self.T, H_), _bits(rng, self.T, H_, std=2.0)
        self.lg_h = rng.standard_normal((self.T, E_)).astype(np.float32)
        if seed % 2:
            self.lg_h[0] = -np.inf                  # a row whose mask leaves nothing
            self.lg_h[:, 7] = -np.inf               # an expert that nobody scores
        self.x.copy_(dev_bits(self.x_h))
        self.res.copy_(dev_bits(self.res_h))
        self.logits.copy_(torch.from_numpy(self.lg_h))

    def step(self):
        import torch
        G, w, T, M = self.G, self.w, self.T, self.T * K_
        xq, w1, aq, w2 = self.ops
        G.moe_add_rmsnorm(self.x, w.norm, T, H_, EPS, residual=self.res, h=self.h, y=self.y)
        G.moe_router_topk(self.logits, T, E_, K_, w.router, self.ids, self.p)
        torch.where(self.keep, self.ids, self.no_id, out=self.pairs)    # padding goes to no expert
        self.dst.fill_(-1)
        G.moe_route_group(None, self.pairs, T, E_, K_, self.used, self.counts, self.offsets, self.dst, self.src, self.y,
                          H_, self.xg)
        G.moe_mxfp4_quantize(self.xg, M, H_, self.grp, self.xq, self.xs)
        G.moe_group_gemm_quant(xq, w1, 2 * I_, H_, self.grp, self.z)
        G.moe_glu_unfused(self.z, self.grp, I_, w.ep, self.a)
        G.moe_mxfp4_quantize(self.a, M, I_, self.grp, self.aq, self.as_)
        G.moe_group_gemm_quant(aq, w2, H_, I_, self.grp, self.y2)
        G.moe_combine(self.y2, M, H_, self.dst, T, K_, self.out, weights=self.p, residual=self.h)

    def check(self, what):
        T, live = self.T, self.T - self.pad
        f64 = F.bf16_bits_to_f64
        hb, rstd, yv = P.add_rmsnorm(self.x_h, self.w.norm_h, EPS, self.res_h)
        assert np.array_equal(host_bits(self.h), hb), what
        y = host_bits(self.y)
        assert np.all(np.abs(f64(y) - yv) <= (2.0 ** -8 + (H_ / 64 + 32) * U) * np.abs(yv)), what
        rid, rp = P.router_topk(self.lg_h, K_, bias=self.w.bias_h, **ROUTER)
        assert np.array_equal(self.ids.cpu().numpy(), rid), what
        p = self.p.cpu().numpy()
        assert np.all(np.abs(p - rp) <= (2 * 8 + 32) * U * np.abs(rp)), what     # (|logit| < 8)
        pairs = np.where(np.arange(T)[:, None] < live, rid, -1)
        counts, offsets, dst, src = O.group_pairs(pairs, E_)
        M = int(offsets[-1])
        assert np.array_equal(self.counts.cpu().numpy(), counts) and np.array_equal(self.dst.cpu().numpy(), dst), what
        xg = host_bits(self.xg)[:M]
        assert np.array_equal(xg, y[src]), what

        def product(q, s, rows, values, got, K):
            rq, rs = P.mxfp4_quantize_rows(rows)
            assert np.array_equal(q.cpu().numpy()[:M], rq) and np.array_equal(s.cpu().numpy()[:M], rs), what
            want, mag = P.group_gemm_values(P.mxfp4_dequantize_rows(rq, rs), counts, values)
            got = host_bits(got)
            err = np.abs(f64(got[:M]) - want)
            assert np.all(err <= 2.0 ** -8 * np.abs(want) + (K / 128 + 16) * 4 * U * mag + 1e-37), what
            assert np.all(got[M:] == BF16_NAN_SENTINEL), what
            return got[:M]
        if M:
            z = product(self.xq, self.xs, xg, self.w.v1, self.z, H_)
            a = host_bits(self.a)[:M]
            assert_bf16_close(a, F.f64_to_bf16_bits(O.glu_from_preact(f64(z), O.Epilogue())), what=what, normwise=1e-2)
            product(self.aq, self.as_, a, self.w.v2, self.y2, I_)
        y2 = host_bits(self.y2)
        want = P.combine(y2, dst, p, hb)
        mag = np.abs(f64(hb))
        for j in range(K_):
            on = dst[:, j] >= 0
            mag[on] += np.abs(p[on, j, None] * f64(y2[dst[on, j]]))
        out = host_bits(self.out)
        assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + (K_ + 2) * U * mag), what
        assert np.array_equal(out[live:], hb[live:]), what          # padding: the residual alone


@pytest.mark.parametrize("T,pad", [(1, 0), (5, 2), (70, 6), (900, 0)])
def test_serving_layer(G, weights, T, pad):
    import torch
    s = Serving(G, weights, T, pad, seed=T + 1)
    for seed in (T + 1, T + 2):
        s.load(seed)
        s.step()
        torch.cuda.synchronize()
        s.check(f"T={T} seed={seed}")


def test_serving_layer_of_padding_alone(G, weights):
    import torch
    s = Serving(G, weights, 4, 4, seed=9)
    s.step()
    torch.cuda.synchronize()
    s.check("padding alone")


@pytest.mark.parametrize("T,pad", [(1, 0), (70, 6), (900, 3)])
def test_serving_layer_graph_replays(G, weights, T, pad):
    import torch
    s = Serving(G, weights, T, pad, seed=20)
    other = Serving(G, weights, 33, 1, seed=50)       # the eager work between the replays
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.step()
    for replay in range(4):
        s.load(21 + replay)
        other.load(51 + replay)
        other.step()
        torch.cuda.synchronize()
        g.replay()
        other.step()
        torch.cuda.synchronize()
        s.check(f"replay {replay}")
        other.check(f"eager {replay}")
        kept = s.out.clone()
        s.step()
        torch.cuda.synchronize()
        assert torch.equal(kept, s.out), replay       # eager and replayed: the same bits


def test_serving_layers_on_two_streams(G, weights):
    """Two layers at once, each on a stream of its own, against each alone."""
    import torch
    a, b = Serving(G, weights, 700, 0, seed=61), Serving(G, weights, 3, 0, seed=62)
    want = []
    for s in (a, b):
        s.step()
        torch.cuda.synchronize()
        want.append(s.out.clone())
        s.out.fill_(0)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for st, s in zip(streams, (a, b)):
            with torch.cuda.stream(st):
                s.step()
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


class Training(Serving):
    """The same layer with bf16 experts, forward and backward."""

    def __init__(self, G, w, T, seed):
        import torch
        super().__init__(G, w, T, 0, seed)
        E, k, H, I, M = E_, K_, H_, I_, T * K_
        self.w1p = empty_bits((G.moe_packed_w1_bytes(E, H, I) // 2,))
        self.w1x = empty_bits((G.moe_packed_weight_bytes(E, H, 2 * I) // 2,))
        self.w2f = empty_bits((G.moe_packed_weight_bytes(E, H, I) // 2,))
        self.w2d = empty_bits((G.moe_packed_weight_bytes(E, I, H) // 2,))
        G.moe_repack_gate_up(w.w1, E, H, I, self.w1p)
        G.moe_pack_weight(w.w1, E, H, 2 * I, G.B_NK, self.w1x)
        G.moe_pack_weight(w.w2, E, H, I, G.B_KN, self.w2f)
        G.moe_pack_weight(w.w2, E, I, H, G.B_NK, self.w2d)
        self.rstd, self.dp = torch.empty(T, device="cuda"), torch.empty(T, k, device="cuda")
        self.dlogits, self.dnorm = torch.empty(T, E, device="cuda"), torch.empty(H, device="cuda")
        self.dy2, self.dgu, self.dxg = (empty_bits((M, n)) for n in (H, 2 * I, H))
        self.dy, self.dx = empty_bits((T, H)), empty_bits((T, H))
        self.dout_h = _bits(np.random.default_rng(seed + 7), T, H)
        self.dout = dev_bits(self.dout_h)
        self.ws = torch.empty(max(G.moe_add_rmsnorm_bwd_workspace_bytes(T, H), 4) // 4, device="cuda")

    def step(self):
        G, w, T, M = self.G, self.w, self.T, self.T * K_
        packed = lambda t, b: (G.operand(t), G.operand(b, layout=G.B_PACKED))  # noqa: E731
        G.moe_add_rmsnorm(self.x, w.norm, T, H_, EPS, residual=self.res, h=self.h, y=self.y, rstd=self.rstd)
        G.moe_router_topk(self.logits, T, E_, K_, w.router, self.ids, self.p)
        G.moe_route_group(None, self.ids, T, E_, K_, self.used, self.counts, self.offsets, self.dst, self.src, self.y,
                          H_, self.xg)
        G.moe_group_gemm_glu_fwd(self.xg, self.grp, self.w1p, H_, I_, w.ep, self.a, self.z)
        G.moe_group_gemm_quant(*packed(self.a, self.w2f), H_, I_, self.grp, self.y2)
        G.moe_combine(self.y2, M, H_, self.dst, T, K_, self.out, weights=self.p, residual=self.h)
        # backward from dout; h takes part in the residual and in the norm
        G.moe_combine_bwd(self.dout, self.y2, M, H_, self.dst, T, K_, weights=self.p, dy=self.dy2, dweights=self.dp)
        G.moe_router_topk_bwd(self.logits, T, E_, K_, w.router, self.ids, self.dp, self.dlogits)
        G.moe_group_gemm_dglu_bwd(self.dy2, packed(self.a, self.w2d)[1], H_, I_, self.grp, self.z, w.ep, self.dgu)
        G.moe_group_gemm_quant(*packed(self.dgu, self.w1x), H_, 2 * I_, self.grp, self.dxg)
        G.moe_combine(self.dxg, M, H_, self.dst, T, K_, self.dy)        # the gather's gradient
        G.moe_add_rmsnorm_bwd(self.dy, self.h, w.norm, self.rstd, T, H_, dh=self.dout, dx=self.dx, dweight=self.dnorm,
                              workspace=self.ws)

    def results(self):
        return [t.clone() for t in (self.out, self.dx, self.dlogits, self.dnorm, self.dgu)]

    def check(self, what):
        """The gradients of sum(dout * out) by float64 differentiation."""
        import torch
        f = lambda b: torch.from_numpy(F.bf16_bits_to_f64(b))  # noqa: E731
        x, lg, nw = f(self.x_h), torch.from_numpy(self.lg_h.astype(np.float64)), f(self.w.norm_h)
        for t in (x, lg, nw):
            t.requires_grad_(True)
        ids = torch.from_numpy(P.router_topk(self.lg_h, K_, bias=self.w.bias_h, **ROUTER)[0].astype(np.int64))
        assert torch.equal(self.ids.cpu().long(), ids), what
        h = x + f(self.res_h)
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * nw
        s = torch.sigmoid(lg).gather(1, ids)
        p = ROUTER["scale"] * s / s.sum(1, keepdim=True)
        w1, w2 = f(self.w.w1_h), f(self.w.w2_h)
        rows = []
        for t in range(self.T):
            for j in range(K_):
                z = y[t] @ w1[ids[t, j]]
                rows.append((torch.nn.functional.silu(z[:I_]) * z[I_:]) @ w2[ids[t, j]])
        y2 = torch.stack(rows).view(self.T, K_, H_)
        out = h + (p[..., None] * y2).sum(1)
        dout = f(self.dout_h)
        (dout * out).sum().backward()
        eps = 12 * 2.0 ** -8
        got = lambda t: torch.from_numpy(F.bf16_bits_to_f64(host_bits(t)))  # noqa: E731
        assert (got(self.out) - out).norm() <= eps * (h.norm() + (p[..., None] * y2).norm()), what
        assert (got(self.dx) - x.grad).norm() <= eps * (dout.norm() + (x.grad - dout).norm()), what
        # dp = <dout, y2>, off by eps of the two vectors' sizes; dlogits: s'(x) / S of it, less its mean
        size = p * dout.norm(dim=1)[:, None] * y2.norm(dim=2)
        bound = 2 * eps * size.sum(1).detach().numpy()
        err = np.abs(self.dlogits.double().cpu().numpy() - lg.grad.numpy()).sum(1)
        assert np.all(err <= bound), what
        # dweight: sum of dy * n over the tokens
        n = (y / nw).detach()
        dy = got(self.dy)
        assert (self.dnorm.double().cpu() - nw.grad).norm() <= eps * (dy.norm(dim=0) * n.norm(dim=0)).norm(), what


def test_training_layer_gradients(G, weights):
    import torch
    s = Training(G, weights, 40, seed=80)
    s.step()
    torch.cuda.synchronize()
    s.check("eager")


def test_training_layer_graph_replays(G, weights):
    import torch
    s = Training(G, weights, 24, seed=90)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.step()
    for replay in range(3):
        s.load(92 + 2 * replay)
        scratch = torch.ones(1 << 18, device="cuda") * 3.0
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert float(scratch.sum()) == 3.0 * (1 << 18)
        s.check(f"replay {replay}")
        kept = s.results()
        s.step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, s.results())), replay
