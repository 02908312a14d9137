"""A block of the operators as a user runs them: norm, route, sort, dispatch, 4-bit
products with SwiGLU between, combine, norm - eager, on its own stream, captured and
replayed; the training direction's rows."""
import numpy as np
import pytest
import torch

import int4_routed_expert_top_b200 as cm
from tests import fp4_format as ff

pytestmark = pytest.mark.gpu

H, I, E, K = 512, 256, 16, 4


class Block:
    """Weights, descriptors and every buffer of one block for up to T tokens."""

    def __init__(self, T, fmt, seed=0):
        rng = np.random.default_rng(seed)

        def rand(*shape, scale=1.0):
            return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).cuda()
        self.T, self.fmt, self.f = T, fmt, {"mx": cm.COLI_MXFP4, "nv": cm.COLI_NVFP4}[fmt]
        self.gate_up, self.down = rand(E * 2 * I, H, scale=0.05), rand(E * H, I, scale=0.05)
        self.g = {n: torch.tensor([v], device="cuda") for n, v in (("x", 0.002), ("h", 0.001), ("w", 1e-4))}
        self.wq = [self.quantize(w, w.shape[0], w.shape[1], self.g["w"]) for w in (self.gate_up, self.down)]
        nv = fmt == "nv"
        self.alpha = [(self.g[n] * self.g["w"]).repeat(E) if nv else None for n in ("x", "h")]
        self.router_w, self.router_b = rand(E, H, scale=0.05), rand(E, scale=0.01)
        blob = torch.zeros(cm.coli_moe_expert_bytes(H, I, 0) * E, dtype=torch.uint8, device="cuda")
        self.blob = blob
        self.layer = cm.coli_moe_layer_create(cm.Desc(H, I, E, K, 0, 0, 1.0, 1, self.router_w.data_ptr(),
                                                      self.router_b.data_ptr(), blob.data_ptr(), 0))
        self.gain = [rand(H, scale=0.1) + 1.0 for _ in range(3)]
        self.desc = cm.NormDesc(H, cm.COLI_F32, cm.COLI_BF16, 1, cm.COLI_GATE_CHANNEL, 0.5, 1e-5,
                                self.gain[0].data_ptr(), self.gain[1].data_ptr())
        P = T * K
        i32 = dict(dtype=torch.int32, device="cuda")
        self.x = rand(T, H)
        self.n = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
        self.idx, self.w = torch.zeros(T, K, **i32), torch.zeros(T, K, device="cuda")
        self.off, self.tok, self.slot, self.inv = (torch.zeros(s, **i32) for s in (E + 1, P, P, (T, K)))
        self.xs = torch.zeros(P, H, dtype=torch.bfloat16, device="cuda")
        self.xq, self.hq = self.space(P, H), self.space(P, I)
        self.gu = torch.zeros(P, 2 * I, dtype=torch.bfloat16, device="cuda")
        self.o = torch.zeros(P, H, dtype=torch.bfloat16, device="cuda")
        self.y = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
        self.x_out, self.n_out = torch.zeros_like(self.x), torch.zeros_like(self.n)
        self.rws = torch.empty(cm.coli_moe_workspace_size(self.layer, T), dtype=torch.uint8, device="cuda")
        self.sws = torch.empty(max(cm.coli_moe_sort_workspace_size(T, K, E), 16), dtype=torch.uint8, device="cuda")
        need = max(cm.coli_moe_fp4_product_workspace_size(self.f, P, H, E, 2 * I),
                   cm.coli_moe_fp4_product_workspace_size(self.f, P, I, E, H))
        self.pws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def space(self, rows, cols):
        return tuple(torch.zeros(n, dtype=torch.uint8, device="cuda") for n in cm.coli_moe_fp4_bytes(self.f, rows, cols))

    def quantize(self, w, rows, cols, g):
        q = self.space(rows, cols)
        cm.coli_moe_fp4_quantize(self.f, w, rows, cols, *q, gscale=g if self.fmt == "nv" else None)
        return q

    def run(self):
        T, P = self.T, self.T * K
        nv = self.fmt == "nv"
        cm.coli_moe_block_norm(self.desc, self.x, None, T, None, self.n)
        cm.coli_moe_route(self.layer, self.n, T, self.idx, self.w, self.rws)
        cm.coli_moe_sort(self.idx, T, K, E, self.off, self.tok, self.slot, self.inv, self.sws)
        cm.coli_moe_dispatch(self.n, T, H, K, self.inv, self.xs)
        cm.coli_moe_fp4_quantize(self.f, self.xs, P, H, *self.xq, count=self.off[E:],
                                 gscale=self.g["x"] if nv else None)
        cm.coli_moe_fp4_product(self.f, *self.xq, P, H, *self.wq[0], E, 2 * I, self.gu, self.pws, offsets=self.off,
                                alpha=self.alpha[0])
        cm.coli_moe_fp4_quantize(self.f, self.gu, P, I, *self.hq, act=cm.COLI_ACT_SWIGLU, count=self.off[E:],
                                 gscale=self.g["h"] if nv else None)
        cm.coli_moe_fp4_product(self.f, *self.hq, P, I, *self.wq[1], E, H, self.o, self.pws, offsets=self.off,
                                alpha=self.alpha[1])
        cm.coli_moe_combine(self.o, T, H, K, self.inv, self.w, self.y)
        cm.coli_moe_block_norm(self.desc, self.x, self.y, T, self.x_out, self.n_out, gate=self.gain[2])

    def results(self):
        return [t.clone() for t in (self.off, self.inv, self.gu, self.o, self.y, self.x_out, self.n_out)]


def plain_check(b):
    """Every step in 64 bits from the step before as the library left it."""
    T, P = b.T, b.T * K
    n = b.x.double() / torch.sqrt(b.x.double().square().mean(1, keepdim=True) + 1e-5) * b.gain[1].double()
    assert ((b.n.double() - n).abs() <= 2.0 ** -7 * n.abs()).all()
    z = torch.sigmoid(b.n.double() @ b.router_w.double().T)
    sel = z + b.router_b.double()
    top = torch.topk(sel, K + 1, dim=1)
    sure = top.values[:, K - 1] - top.values[:, K] > 1e-5
    assert torch.equal(b.idx.long().sort(1)[0][sure], top.indices[:, :K].sort(1)[0][sure])
    w = torch.gather(z, 1, b.idx.long())
    assert ((b.w.double() - w / w.sum(1, keepdim=True)).abs() <= 1e-5).all()
    order = torch.sort(b.idx.view(-1).long(), stable=True)[1]
    assert torch.equal(b.tok.long(), order // K)
    assert torch.equal(b.xs, b.n[order // K])
    off = b.off.tolist()

    def values(q, rows, cols):
        nb = cols // ff.BLOCK[b.fmt]
        byte = ff.untile_scales(q[1].cpu().numpy(), rows, nb)[:, :nb]
        return torch.from_numpy(ff.values(q[0].cpu().numpy().reshape(rows, cols // 2), byte, b.fmt)).cuda()

    def grouped(xq, wq, R, cols, out, alpha):
        X, W = values(xq, P, cols), values(wq, E * R, cols).view(E, R, cols)
        for e in range(E):
            a = 1.0 if alpha is None else float(alpha[e])
            want = a * (X[off[e]:off[e + 1]] @ W[e].T)
            size = a * (X[off[e]:off[e + 1]].abs() @ W[e].abs().T)
            bound = (cols // 64 + 24) * 2.0 ** -22 * size + 2.0 ** -8 * want.abs()
            assert ((out[off[e]:off[e + 1]].double() - want).abs() <= bound).all()
    want = ff.quantize(b.xs.float().cpu().numpy(), b.fmt, float(b.g["x"]))
    np.testing.assert_array_equal(b.xq[0].cpu().numpy().reshape(P, -1), want[0])
    grouped(b.xq, b.wq[0], 2 * I, H, b.gu, b.alpha[0])
    a, u = b.gu[:, :I].float(), b.gu[:, I:].float()
    want = ff.quantize((a / (1 + torch.exp(-a)) * u).cpu().numpy(), b.fmt, float(b.g["h"]))
    # silu's own rounding may move a value across a tie
    assert (b.hq[0].cpu().numpy().reshape(P, -1) != want[0]).mean() <= 0.01
    grouped(b.hq, b.wq[1], H, I, b.o, b.alpha[1])
    rows = b.o.double()[b.inv.long()]
    y = (rows * b.w.double()[..., None]).sum(1)
    size = (rows * b.w.double()[..., None]).abs().sum(1)
    assert ((b.y.double() - y).abs() <= (K + 1) * 2.0 ** -24 * size + 2.0 ** -8 * y.abs()).all()
    o = b.y.double()
    x1 = b.x.double() + 0.5 * b.gain[2].double() * o / torch.sqrt(o.square().mean(1, keepdim=True) + 1e-5) * b.gain[0].double()
    assert ((b.x_out.double() - x1).abs() <= 64 * 2.0 ** -24 * (x1.abs() + b.x.double().abs())).all()
    n = b.x_out.double()
    n = n / torch.sqrt(n.square().mean(1, keepdim=True) + 1e-5) * b.gain[1].double()
    assert ((b.n_out.double() - n).abs() <= 2.0 ** -7 * n.abs()).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T", [1, 3, 64, 700])
def test_block(T, fmt):
    b = Block(T, fmt, seed=T)
    b.run()
    assert cm.coli_moe_fp4_product_status(b.pws) == 0
    plain_check(b)


@pytest.mark.parametrize("T", [1, 64, 400])
def test_block_captured_replayed_and_on_another_stream(T):
    b = Block(T, "mx", seed=5)
    b.run()
    eager = b.results()
    x0 = b.x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(b.results(), eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.run()
    torch.cuda.synchronize()
    b.x.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(1)).cuda())
    graph.replay()
    torch.cuda.synchronize()
    plain_check(b)                       # other tokens, other routing, the same graph
    b.x.copy_(x0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(b.results(), eager))


def test_two_graphs_share_the_workspaces_one_after_the_other():
    b, c = Block(50, "nv", seed=1), Block(50, "nv", seed=2)
    c.pws, c.sws, c.rws = b.pws, b.sws, b.rws
    for blk in (b, c):
        blk.run()
    torch.cuda.synchronize()
    want = [b.results(), c.results()]
    graphs = []
    for blk in (b, c):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            blk.run()
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for blk, w in zip((b, c), want):
        assert all(torch.equal(p, q) for p, q in zip(blk.results(), w))


def test_rows_through_a_training_step():
    """dispatch -> rows times a matrix -> combine -> norm, and back, against autograd in 64 bits."""
    T, k, h = 37, 3, 96
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, h, generator=g).cuda()
    m = (torch.randn(h, h, generator=g) / h ** 0.5).cuda()
    idx = torch.stack([torch.randperm(5, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    idx[4, 1] = -1
    w = torch.rand(T, k, generator=g).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    off, inv = torch.empty(6, **i32), torch.empty(T, k, **i32)
    cm.coli_moe_sort(idx, T, k, 5, off, None, None, inv, None)
    xs = torch.zeros(T * k, h, device="cuda")
    cm.coli_moe_dispatch(x, T, h, k, inv, xs)
    o = xs @ m
    y = torch.empty(T, h, device="cuda")
    cm.coli_moe_combine(o, T, h, k, inv, w, y)
    desc = cm.NormDesc(h, cm.COLI_F32, cm.COLI_F32, 1, cm.COLI_GATE_NONE, 0.5, 1e-5, None, None)
    xo, n, rp, rx = (torch.empty(s, device="cuda") for s in ((T, h), (T, h), T, T))
    cm.coli_moe_block_norm(desc, x, y, T, xo, n, rstd_post=rp, rstd_pre=rx)
    cot = torch.randn(T, h, generator=g).cuda()
    dxr, dy = torch.empty_like(x), torch.empty_like(y)
    cm.coli_moe_block_norm_backward(desc, xo, y, T, None, cot, dxr, dy, None, rstd_post=rp, rstd_pre=rx)
    do, dw, dx = torch.zeros_like(o), torch.empty_like(w), torch.empty_like(x)
    cm.coli_moe_combine_backward(dy, o, T, h, k, inv, w, do, dw)
    cm.coli_moe_dispatch_backward(do @ m.T, T, h, k, inv, dx)
    X, M, W = (t.double().requires_grad_(True) for t in (x, m, w))
    live = (idx >= 0).double()
    Y = ((X @ M)[:, None] * (W * live)[..., None]).sum(1)
    X1 = X + 0.5 * Y / torch.sqrt(Y.square().mean(1, keepdim=True) + 1e-5)
    N = X1 / torch.sqrt(X1.square().mean(1, keepdim=True) + 1e-5)
    gx, gm, gw = torch.autograd.grad(N, (X, M, W), cot.double())
    for got, want in ((dxr + dx, gx), (xs.T @ do, gm)):
        # f32 sums of at most 111 x 96 terms: 1e-5 is 170 half-steps, and the products by
        # the library take the plain f32 path
        assert (got.double() - want).norm() <= 1e-5 * want.norm()
    # All rows of a token are x m here, so y lies along them, and a norm's gradient dy is
    # orthogonal to its input y up to eps / mean(y^2): dw = <o, dy> cancels to about 1e-5 of
    # its terms.  What rounding allows is relative to the terms: |dw - exact| <= sum_h |o| times
    # the error of dy (f32, relative to |dy|-sized terms) + |dy| times the error of o, each
    # within the 170 half-steps above.
    size = (o.double()[inv.long().clamp(min=0)].abs() * dy.double().abs()[:, None]).sum(2)
    assert ((dw.double() - gw).abs() <= 2e-5 * size).all()
