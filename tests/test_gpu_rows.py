"""Sort, dispatch and combine with their gradients against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import int4_routed_expert_top_b200 as cm

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24  # half a step of f32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def picks(T, k, E, drop, seed):
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((T, max(E, k))), 1)[:, :k].astype(np.int32) % E
    idx[rng.random((T, k)) < drop] = -1
    return idx


def plain_sort(idx, E, w=None):
    flat = idx.reshape(-1)
    live = (flat >= 0) & (flat < E)
    if w is not None:
        live &= w.reshape(-1) != 0
    order = np.array([i for e in range(E) for i in np.nonzero(live & (flat == e))[0]], np.int64)
    inv = np.full(flat.size, -1, np.int64)
    inv[order] = np.arange(order.size)
    counts = np.bincount(flat[live], minlength=E)
    return np.concatenate([[0], np.cumsum(counts)]), order, inv.reshape(idx.shape)


def run_sort(idx, E, w=None):
    T, k = idx.shape
    dev = dict(dtype=torch.int32, device="cuda")
    off, inv = torch.full((E + 1,), -7, **dev), torch.full((T, k), -7, **dev)
    tok, slot = torch.full((T * k,), -7, **dev), torch.full((T * k,), -7, **dev)
    ws = torch.empty(cm.coli_moe_sort_workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    cm.coli_moe_sort(torch.from_numpy(idx).cuda(), T, k, E, off, tok, slot, inv, ws if ws.numel() else None,
                     w=None if w is None else torch.from_numpy(w).cuda())
    return off, tok, slot, inv


@pytest.mark.parametrize("T,k,E,drop", [
    (1, 1, 1, 0.0), (1, 8, 256, 0.0), (1, 8, 256, 1.0), (3, 8, 256, 0.2), (33, 2, 5, 0.3), (100, 32, 64, 0.1),
    (127, 8, 1024, 0.5), (128, 8, 3, 0.0),        # 1016 and 1024 picks: one launch
    (1025, 1, 7, 0.1), (511, 8, 1024, 0.5), (700, 9, 1024, 0.2),   # two launches
    (8192, 8, 256, 0.0), (16411, 8, 32, 0.9), (40000, 7, 1, 0.5)])
def test_sort(T, k, E, drop):
    idx = picks(T, k, E, drop, T + k)
    off, tok, slot, inv = (a.cpu().numpy() for a in run_sort(idx, E))
    off0, order, inv0 = plain_sort(idx, E)
    n = order.size
    np.testing.assert_array_equal(off, off0)
    np.testing.assert_array_equal(inv, inv0)
    np.testing.assert_array_equal(tok[:n], order // k)
    np.testing.assert_array_equal(slot[:n], order % k)
    assert (tok[n:] == -7).all() and (slot[n:] == -7).all()


@pytest.mark.parametrize("T", [9, 3000])
def test_sort_drops_zero_weights_and_foreign_experts(T):
    idx = picks(T, 4, 16, 0.0, 3)
    w = np.random.default_rng(4).random((T, 4)).astype(np.float32)
    w[::3, 1] = 0.0
    idx[1::5, 2] = 16
    idx[2::5, 3] = -2147483648
    off, tok, _, inv = (a.cpu().numpy() for a in run_sort(idx, 16, w))
    off0, order, inv0 = plain_sort(idx, 16, w)
    np.testing.assert_array_equal(off, off0)
    np.testing.assert_array_equal(inv, inv0)
    np.testing.assert_array_equal(tok[:order.size], order // 4)


def test_sort_all_to_one_expert_and_no_outputs_but_inv():
    idx = np.full((6000, 1), 11, np.int32)
    off, tok, _, inv = run_sort(idx, 12)
    assert inv.view(-1).tolist() == list(range(6000)) and tok.tolist() == list(range(6000))
    assert off.tolist() == [0] * 12 + [6000]
    off2, inv2 = torch.empty_like(off), torch.empty_like(inv)
    ws = torch.empty(cm.coli_moe_sort_workspace_size(6000, 1, 12), dtype=torch.uint8, device="cuda")
    cm.coli_moe_sort(torch.from_numpy(idx).cuda(), 6000, 1, 12, off2, None, None, inv2, ws)
    assert torch.equal(off, off2) and torch.equal(inv, inv2)


def test_sort_workspace_made_once_for_the_largest_batch():
    """4097 tokens x 8 picks are cut into 33 chunks, 4096 into 64: one workspace for both."""
    k, E = 8, 64
    ws = torch.empty(cm.coli_moe_sort_workspace_size(4097, k, E), dtype=torch.uint8, device="cuda")
    for T in (4097, 4096, 2113, 129, 128):
        idx = picks(T, k, E, 0.1, T)
        off, inv = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
        cm.coli_moe_sort(torch.from_numpy(idx).cuda(), T, k, E, off, None, None, inv, ws)
        off0, _, inv0 = plain_sort(idx, E)
        np.testing.assert_array_equal(off.cpu().numpy(), off0)
        np.testing.assert_array_equal(inv.cpu().numpy(), inv0)


def test_sort_of_no_tokens():
    off = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    cm.coli_moe_sort(z, 0, 2, 4, off, None, None, z, None)
    assert off.tolist() == [0] * 5


SHAPES = [(1, 6144, 8), (1, 1, 1), (3, 7, 2), (5, 256, 32), (65, 1000, 9), (40, 6144, 8), (257, 129, 3), (2, 8200, 10),
          (30, 6143, 8), (9, 6142, 4), (700, 34, 5)]
TYPES = [torch.float32, torch.bfloat16]


def case(T, H, k, dt, seed=0, drop=0.3):
    idx = picks(T, k, max(k, 16), drop, seed + T)
    _, order, inv = plain_sort(idx, max(k, 16))
    return torch.from_numpy(inv.astype(np.int32)).cuda(), order, np.random.default_rng(seed + H)


def rand(rng, *shape, dtype=torch.float32):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda().to(dtype)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,H,k", SHAPES)
def test_dispatch(T, H, k, dt):
    inv, order, rng = case(T, H, k, dt)
    x = rand(rng, T, H, dtype=dt)
    xs = torch.full((T * k, H), 9.0, dtype=dt, device="cuda")
    cm.coli_moe_dispatch(x, T, H, k, inv, xs)
    want = torch.full_like(xs, 9.0)
    if order.size:
        want[:order.size] = x[torch.from_numpy(order // k).cuda()]
    assert torch.equal(xs, want)


def gathered(a, inv):
    got = a.double()[inv.long().clamp(min=0)]
    return torch.where((inv >= 0)[..., None], got, torch.zeros_like(got))


@pytest.mark.parametrize("ot,yt", [(a, b) for a in TYPES for b in TYPES])
@pytest.mark.parametrize("T,H,k", SHAPES)
def test_combine(T, H, k, ot, yt):
    inv, _, rng = case(T, H, k, ot)
    o, w = rand(rng, T * k, H, dtype=ot), rand(rng, T, k)
    res = rand(rng, T, H, dtype=yt)
    for weights, residual in ((w, res), (None, None), (w, None)):
        y = torch.full((T, H), 9.0, dtype=yt, device="cuda")
        cm.coli_moe_combine(o, T, H, k, inv, weights, y, residual=residual)
        terms = gathered(o, inv) * (1.0 if weights is None else weights.double()[..., None])
        want, size = terms.sum(1), terms.abs().sum(1)
        if residual is not None:
            want, size = want + residual.double(), size + residual.double().abs()
        # k fused steps and one sum, half a step each of at most `size`, then the rounding to yt
        bound = (k + 1) * U24 * size * 1.01 + HALF[yt] * want.abs() + 1e-30
        assert ((y.double() - want).abs() <= bound).all()


def test_combine_residual_may_alias_y():
    inv, _, rng = case(40, 128, 4, torch.float32)
    o, w, res = rand(rng, 160, 128), rand(rng, 40, 4), rand(rng, 40, 128)
    y = torch.empty_like(res)
    cm.coli_moe_combine(o, 40, 128, 4, inv, w, y, residual=res)
    cm.coli_moe_combine(o, 40, 128, 4, inv, w, res, residual=res)
    assert torch.equal(y, res)


def dot_bound(H, dt):
    # the longest chain of one lane's fused steps (16 bytes of columns at a time, with a sum per
    # element), then at most 8 of its own sums and 5 in the warp
    return (-(-H // (32 * (16 // dt.itemsize))) + 13) * U24 * 1.01


@pytest.mark.parametrize("ot,yt", [(a, b) for a in TYPES for b in TYPES])
@pytest.mark.parametrize("T,H,k", SHAPES)
def test_combine_backward(T, H, k, ot, yt):
    inv, order, rng = case(T, H, k, ot)
    o, w, dy = rand(rng, T * k, H, dtype=ot), rand(rng, T, k), rand(rng, T, H, dtype=yt)
    for weights in (w, None):
        do, dw = torch.full_like(o, 9.0), torch.full_like(w, 9.0)
        cm.coli_moe_combine_backward(dy, o, T, H, k, inv, weights, do, dw)
        terms = gathered(o, inv) * dy.double()[:, None]
        assert ((dw.double() - terms.sum(2)).abs() <= dot_bound(H, ot) * terms.abs().sum(2) + 1e-30).all()
        assert (dw[inv < 0] == 0).all()
        want = torch.full((T * k, H), 9.0, dtype=torch.float64, device="cuda")
        if order.size:
            t, j = torch.from_numpy(order // k).cuda(), torch.from_numpy(order % k).cuda()
            want[:order.size] = dy.double()[t] * (1.0 if weights is None else weights.double()[t, j][:, None])
        assert ((do.double() - want).abs() <= (U24 + HALF[ot]) * 1.01 * want.abs()).all()
        only_do, only_dw = torch.full_like(o, 9.0), torch.full_like(w, 9.0)
        cm.coli_moe_combine_backward(dy, None, T, H, k, inv, weights, only_do, None)
        cm.coli_moe_combine_backward(dy, o, T, H, k, inv, weights, None, only_dw)
        assert torch.equal(only_do, do) and torch.equal(only_dw, dw)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,H,k", SHAPES)
def test_dispatch_backward(T, H, k, dt):
    inv, _, rng = case(T, H, k, dt)
    dxs = rand(rng, T * k, H, dtype=dt)
    dx = torch.full((T, H), 9.0, dtype=dt, device="cuda")
    cm.coli_moe_dispatch_backward(dxs, T, H, k, inv, dx)
    terms = gathered(dxs, inv)
    assert ((dx.double() - terms.sum(1)).abs()
            <= k * U24 * 1.01 * terms.abs().sum(1) + HALF[dt] * terms.sum(1).abs()).all()


def test_gradients_against_differences():
    """L = sum(c * combine(dispatch(x) * s, w)): dx and dw from the calls against central
    differences of the 64-bit form."""
    T, H, k = 4, 24, 3
    inv, order, rng = case(T, H, k, torch.float32, drop=0.2)
    x, w, c, s = rand(rng, T, H), rand(rng, T, k), rand(rng, T, H), rand(rng, T * k, H)

    def loss(xx, ww):
        rows = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        rows[:order.size] = xx[torch.from_numpy(order // k).cuda()]
        return ((gathered(rows * s.double(), inv) * ww[..., None]).sum(1) * c.double()).sum()

    xs, y = torch.zeros(T * k, H, device="cuda"), torch.empty(T, H, device="cuda")
    cm.coli_moe_dispatch(x, T, H, k, inv, xs)
    o = xs * s
    cm.coli_moe_combine(o, T, H, k, inv, w, y)
    do, dw, dx = torch.zeros_like(o), torch.empty_like(w), torch.empty_like(x)
    cm.coli_moe_combine_backward(c, o, T, H, k, inv, w, do, dw)
    cm.coli_moe_dispatch_backward(do * s, T, H, k, inv, dx)
    h = 1e-4
    for a, da, which in ((x, dx, 0), (w, dw, 1)):
        for i in range(0, a.numel(), 5):
            e = torch.zeros(a.numel(), dtype=torch.float64, device="cuda")
            e[i] = h
            e = e.view(a.shape)
            args = [x.double(), w.double()]
            up, down = list(args), list(args)
            up[which], down[which] = args[which] + e, args[which] - e
            d = (loss(*up) - loss(*down)) / (2 * h)  # the loss is linear in each: exact but for rounding
            assert abs(float(d) - float(da.view(-1)[i])) <= 1e-4 * max(1.0, abs(float(d)))


@pytest.mark.parametrize("H", [64, 65])
def test_unaligned_rows(H):
    """Tensors that begin one element into their storage take the single-element kernels."""
    T, k = 6, 4
    inv, order, rng = case(T, H, k, torch.bfloat16)

    def off(a):
        b = torch.empty(a.numel() + 1, dtype=a.dtype, device="cuda")[1:].view(a.shape)
        return b.copy_(a)
    x = off(rand(rng, T, H, dtype=torch.bfloat16))
    xs, xs0 = off(torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")), torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
    cm.coli_moe_dispatch(x, T, H, k, inv, xs)
    cm.coli_moe_dispatch(x.clone(), T, H, k, inv, xs0)
    assert torch.equal(xs, xs0)
    w = rand(rng, T, k)
    y, y0 = off(torch.zeros(T, H, device="cuda")), torch.zeros(T, H, device="cuda")
    cm.coli_moe_combine(xs, T, H, k, inv, w, y)
    cm.coli_moe_combine(xs0, T, H, k, inv, w, y0)
    assert torch.equal(y, y0)
    do, do0, dw, dw0 = off(torch.zeros_like(xs0)), torch.zeros_like(xs0), torch.empty_like(w), torch.empty_like(w)
    cm.coli_moe_combine_backward(y, xs, T, H, k, inv, w, do, dw)
    cm.coli_moe_combine_backward(y0, xs0, T, H, k, inv, w, do0, dw0)
    assert torch.equal(do, do0)
    # the two kernels add the products in different orders
    size = gathered(xs0, inv).abs().mul(y0.double().abs()[:, None]).sum(2)
    assert ((dw - dw0).double().abs() <= 2 * dot_bound(H, torch.bfloat16) * size).all()


def test_rows_outside_the_buffer_are_not_computed():
    T, H, k = 4, 32, 2
    x, o = torch.ones(T, H, device="cuda"), torch.ones(T * k, H, device="cuda")
    inv = torch.tensor([[0, 8], [-1, 1 << 30], [3, 2], [-5, 7]], dtype=torch.int32, device="cuda")
    xs, y = torch.zeros(T * k, H, device="cuda"), torch.empty(T, H, device="cuda")
    cm.coli_moe_dispatch(x, T, H, k, inv, xs)
    assert xs[:, 0].tolist() == [1, 0, 1, 1, 0, 0, 0, 1]
    cm.coli_moe_combine(o, T, H, k, inv, None, y)
    assert y[:, 0].tolist() == [1, 0, 2, 1]


def test_binding_refuses_wrong_tensors():
    x = torch.ones(4, 32, device="cuda")
    inv = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    xs = torch.zeros(8, 32, device="cuda")
    with pytest.raises(ValueError):
        cm.coli_moe_dispatch(x, 5, 32, 2, inv, xs)               # x is too short
    with pytest.raises(ValueError):
        cm.coli_moe_dispatch(x.t(), 4, 32, 2, inv, xs)           # not contiguous
    with pytest.raises(ValueError):
        cm.coli_moe_dispatch(x.cpu(), 4, 32, 2, inv, xs)
    with pytest.raises(TypeError):
        cm.coli_moe_dispatch(x, 4, 32, 2, inv.long(), xs)
    with pytest.raises(TypeError):
        cm.coli_moe_dispatch(x.half(), 4, 32, 2, inv, xs)
    with pytest.raises(TypeError):
        cm.coli_moe_dispatch(x, 4, 32, 2, inv, xs.bfloat16())
