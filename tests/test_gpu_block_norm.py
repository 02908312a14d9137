"""The step between two blocks (norm, gate, residual scale, sum, norm) and its
gradient against the formula in 64 bits."""
import itertools

import numpy as np
import pytest
import torch

import int4_routed_expert_top_b200 as cm

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
KIND = {"none": cm.COLI_GATE_NONE, "channel": cm.COLI_GATE_CHANNEL, "token": cm.COLI_GATE_TOKEN,
        "full": cm.COLI_GATE_FULL}
F, B = torch.float32, torch.bfloat16
CODE = {F: cm.COLI_F32, B: cm.COLI_BF16}
ALPHA, EPS = 0.7, 1e-5


def chain(H):
    """Roundings on the way of one term into a sum over the row: at most 32 of a thread (four
    vectors of eight), 5 in a warp, 5 across warps, and a few of the factors."""
    return 32 + 5 + 5 + 6


class Case:
    def __init__(self, T, H, xt, bt, gate, post=True, gains=True, seed=0):
        rng = np.random.default_rng(seed + T * 7 + H)

        def rand(*shape, dtype=F, scale=1.0, shift=0.0):
            return torch.from_numpy((shift + scale * rng.standard_normal(shape)).astype(np.float32)).cuda().to(dtype)
        self.T, self.H, self.xt, self.bt, self.kind, self.post = T, H, xt, bt, gate, post
        self.x, self.o = rand(T, H, dtype=xt), rand(T, H, dtype=bt, scale=0.5)
        self.gp = rand(H, scale=0.3, shift=1.0) if gains else None
        self.gx = rand(H, scale=0.3, shift=1.0) if gains else None
        shape = {"none": None, "channel": (H,), "token": (T,), "full": (T, H)}[gate]
        self.gate = None if shape is None else rand(*shape)
        self.dxo, self.dn = rand(T, H, dtype=xt), rand(T, H, dtype=bt)
        self.desc = cm.NormDesc(H, CODE[xt], CODE[bt], int(post), KIND[gate], ALPHA, EPS,
                                self.gp.data_ptr() if gains else None, self.gx.data_ptr() if gains else None)

    def gate64(self, gate=None):
        g = self.gate if gate is None else gate
        if g is None:
            return torch.ones((), dtype=torch.float64, device="cuda")
        return g.double()[:, None] if self.kind == "token" else g.double()

    def buffers(self):
        T, H = self.T, self.H
        return (torch.full((T, H), 9.0, dtype=self.xt, device="cuda"), torch.full((T, H), 9.0, dtype=self.bt, device="cuda"),
                torch.full((T,), 9.0, device="cuda"), torch.full((T,), 9.0, device="cuda"))

    def forward(self):
        xo, n, rp, rx = self.buffers()
        cm.coli_moe_block_norm(self.desc, self.x, self.o, self.T, xo, n, gate=self.gate, rstd_post=rp, rstd_pre=rx)
        return xo, n, rp, rx


def one(g):
    return 1.0 if g is None else g.double()


def rstd(v):
    return 1.0 / torch.sqrt(v.square().mean(1) + EPS)


SHAPES = [(1, 6144), (1, 1), (3, 2), (5, 127), (17, 1024), (9, 6144), (3, 8192), (2, 8196), (2, 16384), (2, 9001), (300, 260),
          (9, 6143), (9, 4098), (3000, 33)]
TYPES = [(F, F), (F, B), (B, B)]


@pytest.mark.parametrize("xt,bt", TYPES)
@pytest.mark.parametrize("gate", list(KIND))
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(T, H, gate, xt, bt):
    for post, gains in ((True, True), (True, False), (False, True)):
        c = Case(T, H, xt, bt, gate, post, gains)
        xo, n, rp, rx = c.forward()
        o = c.o.double()
        C = chain(H)
        r = rstd(o)
        if post:
            assert ((rp.double() - r).abs() <= C * U24 * r).all()
            u = o * r[:, None] * one(c.gp)
        else:
            assert (rp == 9.0).all()  # not written
            u = o
        add = c.desc.alpha * c.gate64() * u
        want = c.x.double() + add
        bound = C * U24 * add.abs() + (2 * U24 + HALF[xt]) * want.abs() + 1e-30
        assert ((xo.double() - want).abs() <= bound).all()
        stored = xo.double()  # the second norm reads the stored sum
        r = rstd(stored)
        assert ((rx.double() - r).abs() <= C * U24 * r).all()
        want = stored * r[:, None] * one(c.gx)
        assert ((n.double() - want).abs() <= (C * U24 + HALF[bt] * 1.01) * want.abs() + 1e-30).all()


@pytest.mark.parametrize("xt,bt", TYPES)
@pytest.mark.parametrize("T,H", [(1, 6144), (7, 33)])
def test_first_and_last_block(T, H, xt, bt):
    c = Case(T, H, xt, bt, "channel")
    xo, n, rp, rx = c.forward()
    # before the first block: only the norm of x
    n1, r1 = torch.empty_like(n), torch.empty_like(rx)
    cm.coli_moe_block_norm(c.desc, xo, None, T, None, n1, rstd_pre=r1)
    assert torch.equal(n1, n) and torch.equal(r1, rx)
    # after the last block: only the sum; in place
    x2 = c.x.clone()
    cm.coli_moe_block_norm(c.desc, x2, c.o, T, x2, None, gate=c.gate)
    assert torch.equal(x2, xo)
    x3, n3 = c.x.clone(), torch.empty_like(n)
    cm.coli_moe_block_norm(c.desc, x3, c.o, T, x3, n3, gate=c.gate)
    assert torch.equal(x3, xo) and torch.equal(n3, n)


def formula(c, x, o, gp, gx, gate):
    u = o / torch.sqrt(o.square().mean(1, keepdim=True) + EPS) * gp if c.post else o
    g = gate[:, None] if c.kind == "token" else gate
    x1 = x + ALPHA * g * u
    return x1, x1 / torch.sqrt(x1.square().mean(1, keepdim=True) + EPS) * gx


@pytest.mark.parametrize("gate", list(KIND))
@pytest.mark.parametrize("post", [True, False])
def test_gradient_formula_against_differences(gate, post):
    """The 64-bit gradient that the kernel is held to (autograd of the formula) agrees with
    central differences."""
    c = Case(3, 10, F, F, gate, post)
    ins = [c.x.double(), c.o.double(), c.gp.double(), c.gx.double(),
           torch.ones(c.H, dtype=torch.float64, device="cuda") if c.gate is None else c.gate.double()]
    for t in ins:
        t.requires_grad_(True)
    assert torch.autograd.gradcheck(lambda *a: formula(c, *a), ins, eps=1e-6, atol=1e-6, rtol=1e-5)


def backward(c, xo, rp, rx, dxo=True, dn=True, gate_grad=True):
    T, H = c.T, c.H
    dx, do = torch.full((T, H), 9.0, dtype=c.xt, device="cuda"), torch.full((T, H), 9.0, dtype=c.bt, device="cuda")
    dpost, dpre = torch.full((H,), 9.0, device="cuda"), torch.full((H,), 9.0, device="cuda")
    dgate = None if c.gate is None else torch.full_like(c.gate, 9.0)
    ws = torch.full((cm.coli_moe_block_norm_backward_workspace_size(c.desc, T),), 255, dtype=torch.uint8, device="cuda")
    cm.coli_moe_block_norm_backward(c.desc, xo, c.o, T, c.dxo if dxo else None, c.dn if dn else None, dx, do, ws,
                                    gate=c.gate, rstd_post=rp if c.post else None, rstd_pre=rx if dn else None,
                                    dpost_gain=dpost if c.post else None, dgate=dgate, dpre_gain=dpre if dn else None)
    return dx, do, dpost, dgate, dpre


def check_backward(c, dxo=True, dn=True):
    """Against the formula's gradient, term by term: every result is a sum of terms whose
    sizes are known, and each f32 rounding on the way is at most half a step of one of them."""
    T, H = c.T, c.H
    xo, _, rp, rx = c.forward()
    dx, do, dpost, dgate, dpre = backward(c, xo, rp, rx, dxo, dn)
    C = (2 * chain(H) + 20) * U24
    zero = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    x1, o = xo.double(), c.o.double()
    g, gx, gp = c.gate64(), one(c.gx), one(c.gp)
    # with the saved statistics, which the forward test holds to their formula
    rx, rp = rx.double()[:, None], rp.double()[:, None]
    xh, v = x1 * rx, c.dn.double() * gx if dn else zero
    d0 = c.dxo.double() if dxo else zero
    mean = (v * xh).mean(1, keepdim=True)
    d = d0 + (rx * (v - xh * mean) if dn else 0)
    size = d0.abs() + (rx * (v.abs() + xh.abs() * (v * xh).abs().mean(1, keepdim=True)) if dn else 0)
    assert ((dx.double() - d).abs() <= C * size + HALF[c.xt] * d.abs()).all()
    # the sums over tokens: rows of a CTA one after the other (148 CTAs at least), two CTAs of a
    # cluster, then partial rows of at most 16 x 148 / 2 / 32 in a run and the sums of 32 runs
    S = C + (-(-T // 148) + 2 + 37 + 32) * U24
    if dn:
        t = c.dn.double() * xh
        assert ((dpre.double() - t.sum(0)).abs() <= S * t.abs().sum(0) + 1e-30).all()
    oh = o * rp if c.post else o
    u = oh * gp if c.post else oh
    usize = u.abs()
    if dgate is not None:
        t, ts = ALPHA * u * d, ALPHA * usize * size
        dim = {"channel": 0, "token": 1}.get(c.kind)
        want, bound = (t, ts) if dim is None else (t.sum(dim), ts.sum(dim))
        assert ((dgate.double() - want).abs() <= S * bound + 1e-30).all()
    e, es = ALPHA * g * d, (ALPHA * g).abs() * size
    if c.post:
        t, ts = e * oh, es * oh.abs()
        assert ((dpost.double() - t.sum(0)).abs() <= S * ts.sum(0) + 1e-30).all()
        q, qs = e * gp, es * abs(gp)
        m, ms = (q * oh).mean(1, keepdim=True), (qs * oh.abs()).mean(1, keepdim=True)
        e, es = rp * (q - oh * m), rp * (qs + oh.abs() * ms)
    assert ((do.double() - e).abs() <= 2 * C * es + HALF[c.bt] * e.abs() + 1e-30).all()
    return dx, do, dpost, dgate, dpre


@pytest.mark.parametrize("xt,bt", TYPES)
@pytest.mark.parametrize("gate", list(KIND))
@pytest.mark.parametrize("T,H", SHAPES + [(1000, 64), (296, 8), (301, 2048), (2000, 1024), (450, 6144), (297, 8192)])
def test_backward(T, H, gate, xt, bt):
    for post, gains in ((True, True), (False, False)):
        check_backward(Case(T, H, xt, bt, gate, post, gains))


@pytest.mark.parametrize("T,H", [(5, 96), (2, 6144), (400, 1024)])
def test_backward_with_one_gradient(T, H):
    for gate, (dxo, dn) in itertools.product(("none", "token"), ((True, False), (False, True))):
        check_backward(Case(T, H, F, B, gate), dxo, dn)


def test_backward_against_autograd():
    """The whole gradient at once, from the forward call's own outputs (f32, so that the
    formula's statistics are the saved ones up to rounding)."""
    c = Case(6, 200, F, F, "channel")
    ins = [t.double().requires_grad_(True) for t in (c.x, c.o, c.gp, c.gx, c.gate)]
    x1, n = formula(c, *ins)
    want = torch.autograd.grad([x1, n], ins, [c.dxo.double(), c.dn.double()])
    xo, _, rp, rx = c.forward()
    dx, do, dpost, dgate, dpre = backward(c, xo, rp, rx)
    for got, w in zip((dx, do, dpost, dpre, dgate), want):
        assert (got.double() - w).norm() <= 200 * U24 * w.norm()


def test_backward_is_the_same_every_time_and_without_a_block():
    c = Case(700, 512, F, B, "channel")
    xo, _, rp, rx = c.forward()
    a, b = backward(c, xo, rp, rx), backward(c, xo, rp, rx)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    # before the first block there is no o: the gradient of x alone
    dx, dpre = torch.empty_like(c.x), torch.empty(c.H, device="cuda")
    ws = torch.empty(cm.coli_moe_block_norm_backward_workspace_size(c.desc, c.T), dtype=torch.uint8, device="cuda")
    cm.coli_moe_block_norm_backward(c.desc, xo, None, c.T, c.dxo, c.dn, dx, None, ws, rstd_pre=rx, dpre_gain=dpre)
    assert torch.equal(dx, a[0]) and torch.equal(dpre, a[4])
    # dx in place of dx_out
    dxo = c.dxo.clone()
    cm.coli_moe_block_norm_backward(c.desc, xo, None, c.T, dxo, c.dn, dxo, None, ws, rstd_pre=rx, dpre_gain=dpre)
    assert torch.equal(dxo, dx)


def test_no_tokens():
    c = Case(1, 64, F, F, "channel")
    e = torch.empty(0, 64, device="cuda")
    dgate, dpost, dpre = (torch.full((64,), 9.0, device="cuda") for _ in range(3))
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    r = torch.empty(0, device="cuda")
    cm.coli_moe_block_norm(c.desc, e, e, 0, e, e, gate=c.gate)
    one_row = torch.empty(1, 64, device="cuda")  # empty tensors have no address to pass
    cm.coli_moe_block_norm_backward(c.desc, one_row, one_row, 0, one_row, one_row, one_row, one_row.clone(), ws,
                                    gate=c.gate, rstd_post=one_row[0], rstd_pre=one_row[0], dpost_gain=dpost,
                                    dgate=dgate, dpre_gain=dpre)
    assert float(dgate.abs().sum() + dpost.abs().sum() + dpre.abs().sum()) == 0.0  # sums over no tokens


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_an_empty_batch_forward_and_backward(gate):
    """Empty tensors and no workspace, as a rank without tokens has them."""
    c = Case(1, 64, F, F, gate)
    e, r = torch.empty(0, 64, device="cuda"), torch.empty(0, device="cuda")
    g = {"none": None, "channel": c.gate, "token": r, "full": e}[gate]
    assert cm.coli_moe_block_norm_backward_workspace_size(c.desc, 0) == 0
    dpost, dpre = (torch.full((64,), 9.0, device="cuda") for _ in range(2))
    dgate = None if g is None else torch.full_like(g, 9.0)
    cm.coli_moe_block_norm(c.desc, e, e, 0, e, e, gate=g, rstd_post=r, rstd_pre=r)
    cm.coli_moe_block_norm_backward(c.desc, e, e, 0, e, e, e, e, None, gate=g, rstd_post=r, rstd_pre=r,
                                    dpost_gain=dpost, dgate=dgate, dpre_gain=dpre)
    for d in (dpost, dpre, dgate):
        assert d is None or (d == 0).all()                   # sums over no tokens
    cm.coli_moe_block_norm_backward(c.desc, e, e, 0, e, e, e, e, None, gate=g, rstd_post=r, rstd_pre=r)
    cm.coli_moe_block_norm_backward(c.desc, e, None, 0, e, None, e, None, None)


def test_unusual_rows():
    """A row of zeros, one of infinities and one with a NaN stay apart from their neighbours."""
    c = Case(5, 256, F, F, "none")
    c.x[1], c.o[1] = 0.0, 0.0
    c.o[2, 7] = float("inf")
    c.x[3, 9] = float("nan")
    xo, n, rp, rx = c.forward()
    assert (xo[1] == 0).all() and (n[1] == 0).all()
    assert torch.isnan(n[3]).all() and torch.isnan(xo[2, 7])
    assert torch.isfinite(n[0]).all() and torch.isfinite(n[4]).all()


def test_unaligned_tensors_take_single_elements():
    c = Case(4, 128, B, B, "full")

    def off(a):
        return torch.empty(a.numel() + 1, dtype=a.dtype, device="cuda")[1:].view(a.shape).copy_(a)
    want = c.forward()
    xo, n, rp, rx = (off(t) for t in c.buffers())
    cm.coli_moe_block_norm(c.desc, off(c.x), off(c.o), c.T, xo, n, gate=off(c.gate), rstd_post=rp, rstd_pre=rx)
    assert (xo.double() - want[0].double()).abs().max() <= 2.0 ** -7 * want[0].double().abs().max()
    check_backward(c)


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("T,H", [(3, 40), (2, 33), (700, 1024)])
def test_infinities_of_a_block_without_its_norm_stay_where_they_are(T, H, gate):
    # without post_norm the gradient of o does not depend on o: alpha gate dx, two or three
    # products of f32 and one rounding, whatever o holds
    c = Case(T, H, F, B, gate, post=False, gains=False)
    c.o[:, 1::7] = float("inf")
    c.o[:, 2::7] = float("nan")
    dx, do = torch.empty_like(c.x), torch.empty_like(c.o)
    cm.coli_moe_block_norm_backward(c.desc, None, c.o, T, c.dxo, None, dx, do, None, gate=c.gate)
    assert torch.equal(dx, c.dxo)
    want = c.desc.alpha * c.gate64() * c.dxo.double()
    assert ((do.double() - want).abs() <= (3 * U24 + HALF[B] * 1.01) * want.abs() + 1e-30).all()
    if gate == "channel":  # a channel's gate alone sees its own values
        ws = torch.empty(cm.coli_moe_block_norm_backward_workspace_size(c.desc, T), dtype=torch.uint8, device="cuda")
        dgate = torch.empty_like(c.gate)
        cm.coli_moe_block_norm_backward(c.desc, None, c.o, T, c.dxo, None, dx, do, ws, gate=c.gate, dgate=dgate)
        terms = c.desc.alpha * c.o.double() * c.dxo.double()
        finite = torch.isfinite(c.o.float()).all(0)
        assert torch.equal(torch.isfinite(dgate), finite)
        err = (dgate.double() - terms.sum(0)).abs()[finite]
        assert (err <= (T + 10) * U24 * terms.abs().sum(0)[finite]).all()
