"""The fused kernel's bounded waits run out without hanging the GPU: with the
test option of coli_moe_layer_set_wait_test, CTA 0's producer never issues one
ring stage, the consumer warps' wait on it gives up after a short limit, the
kernel and the combine return, coli_moe_status reports COLI_E_TIMEOUT, and the
next call on the same workspace (option cleared) is correct and bit-identical
to a call that never saw the option.  The same of the 4-bit floating point product's
waits (coli_moe_fp4_set_wait_test) and of those in the block norm's gradient
(coli_moe_block_norm_set_wait_test), which makes its rows NaN."""
import dataclasses

import numpy as np
import pytest
import torch

import synth
import int4_routed_expert_top_b200 as cm
from tests.workloads import (OracleExperts, build_layer, gap_resampled_tokens, oracle_tokens,
                             rel_err)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,group", [(1, 0), (4, 64), (12, 64)])
def test_wait_gives_up_and_the_next_call_is_correct(T, group):
    wl = dataclasses.replace(synth.TINY, T=T, group=group)
    wr, b = synth.router(wl)
    x, idx_ref, w_ref, _ = gap_resampled_tokens(wl, T, wr, b)
    y_ref = oracle_tokens(wl, OracleExperts(wl), x.numpy(), idx_ref, w_ref)
    L = build_layer(wl, router=(wr, b))
    ws = L.workspace(T)
    xd = x.cuda()
    y = torch.empty((T, wl.H), dtype=torch.float32, device="cuda")
    cm.coli_moe_forward_ex(L.handle, xd, T, y, ws, path=cm.COLI_PATH_FUSED)
    torch.cuda.synchronize()
    y_clean = y.cpu().numpy().copy()
    assert cm.coli_moe_status(L.handle, T, ws) == 0

    cm.coli_moe_layer_set_wait_test(L.handle, 0)
    cm.coli_moe_forward_ex(L.handle, xd, T, y, ws, path=cm.COLI_PATH_FUSED)
    with pytest.raises(cm.ColiError) as e:
        cm.coli_moe_status(L.handle, T, ws)
    assert e.value.code == -6                                  # COLI_E_TIMEOUT

    cm.coli_moe_layer_set_wait_test(L.handle, -1)
    y.fill_(float("nan"))
    cm.coli_moe_forward_ex(L.handle, xd, T, y, ws, path=cm.COLI_PATH_FUSED)
    torch.cuda.synchronize()
    assert cm.coli_moe_status(L.handle, T, ws) == 0
    out = y.cpu().numpy()
    np.testing.assert_array_equal(out.view(np.uint32), y_clean.view(np.uint32))
    assert rel_err(out, y_ref) <= 2e-3
    L.close()


def fp4_call(E, R, K, sizes):
    """Random operands of a grouped MXFP4 product, the call as a function of y and ws, and ws's size."""
    g = torch.Generator(device="cuda").manual_seed(R + K)
    P = sum(sizes)
    off = torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int32, device="cuda")

    def side(n):
        nc, ns = cm.coli_moe_fp4_bytes(cm.COLI_MXFP4, n, K)
        return (torch.randint(0, 256, (nc,), generator=g, device="cuda", dtype=torch.uint8),
                torch.randint(120, 130, (ns,), generator=g, device="cuda", dtype=torch.uint8))
    x, w = side(P), side(E * R)
    return (lambda y, ws: cm.coli_moe_fp4_product(cm.COLI_MXFP4, *x, P, K, *w, E, R, y, ws, offsets=off),
            cm.coli_moe_fp4_product_workspace_size(cm.COLI_MXFP4, P, K, E, R))


# one CTA by itself with tiles cut in several, whole waves of tiles and more, pairs of CTAs likewise
@pytest.mark.parametrize("E,R,K,sizes", [(4, 1024, 6144, [1, 0, 3, 2]), (1, 128 * 150, 4096, [3]), (1, 10240, 6144, [97]),
                                         (2, 5120, 6144, [300, 200])])
@pytest.mark.parametrize("withhold", [0, 1])
def test_product_wait_gives_up_is_reported_and_stays_until_cleared(E, R, K, sizes, withhold):
    """A stage that is never copied, or pieces of cut tiles that are never announced: the call
    returns, what lacks its sums is NaN, the rest is right; the status stays through the
    next calls, which give only NaN, until the workspace is cleared."""
    call, size = fp4_call(E, R, K, sizes)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    good, y = (torch.full((sum(sizes), R), 9.0, device="cuda") for _ in range(2))
    call(good, ws)
    assert cm.coli_moe_fp4_product_status(ws) == 0 and torch.isfinite(good).all()
    cm.coli_moe_fp4_set_wait_test(withhold)
    try:
        call(y, ws)
    finally:
        cm.coli_moe_fp4_set_wait_test(-1)
    for _ in range(2):
        with pytest.raises(cm.ColiError) as e:
            cm.coli_moe_fp4_product_status(ws)
        assert e.value.code == -6                              # COLI_E_TIMEOUT
    gone = torch.isnan(y)
    assert gone.any() and torch.equal(y[~gone], good[~gone])
    y.fill_(9.0)
    call(y, ws)                                                # marked: nothing to trust in ws
    assert torch.isnan(y).all()
    with pytest.raises(cm.ColiError):
        cm.coli_moe_fp4_product_status(ws)
    ws.zero_()
    call(y, ws)
    assert cm.coli_moe_fp4_product_status(ws) == 0 and torch.equal(y, good)


def test_product_status_of_two_calls_is_read_once():
    """Two products on one workspace, as gate/up and down of a block have them: the first one's
    give-up is seen after the second."""
    call, size = fp4_call(4, 1024, 6144, [1, 0, 3, 2])
    ws, y = torch.zeros(size, dtype=torch.uint8, device="cuda"), torch.empty(6, 1024, device="cuda")
    cm.coli_moe_fp4_set_wait_test(0)
    try:
        call(y, ws)
    finally:
        cm.coli_moe_fp4_set_wait_test(-1)
    call(y, ws)
    with pytest.raises(cm.ColiError):
        cm.coli_moe_fp4_product_status(ws)


@pytest.mark.parametrize("H,gate", [(6144, "channel"), (1024, "token"), (512, "full"), (1024, "none")])
@pytest.mark.parametrize("post,dn", [(True, True), (False, False)])
@pytest.mark.parametrize("withhold", [0, 1])
def test_norm_gradient_wait_gives_up_in_nan(H, gate, post, dn, withhold):
    """Rows of CTA 0 from the withheld one on are NaN in every gradient, the sums over tokens with
    them; the others are right, and so is the next call."""
    T = 2000
    g = torch.Generator(device="cuda").manual_seed(H)

    def rand(*shape, dt=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)
    kind = {"none": 0, "channel": 1, "token": 2, "full": 3}[gate]
    shape = {"none": None, "channel": (H,), "token": (T,), "full": (T, H)}[gate]
    gv = None if shape is None else rand(*shape)
    gains = rand(H), rand(H)
    desc = cm.NormDesc(H, cm.COLI_F32, cm.COLI_BF16, int(post), kind, 0.7, 1e-5, gains[0].data_ptr(), gains[1].data_ptr())
    x, o, dxo, dnv = rand(T, H), rand(T, H, dt=torch.bfloat16), rand(T, H), rand(T, H, dt=torch.bfloat16)
    r = rand(T).abs(), rand(T).abs()
    ws = torch.empty(cm.coli_moe_block_norm_backward_workspace_size(desc, T), dtype=torch.uint8, device="cuda")

    def run():
        out = dict(dx=torch.full_like(x, 9.0), d_o=torch.full_like(o, 9.0),
                   dpost_gain=torch.full((H,), 9.0, device="cuda") if post else None,
                   dpre_gain=torch.full((H,), 9.0, device="cuda") if dn else None,
                   dgate=None if gv is None else torch.full_like(gv, 9.0))
        cm.coli_moe_block_norm_backward(desc, x, o, T, dxo, dnv if dn else None, out["dx"], out["d_o"], ws, gate=gv,
                                        rstd_post=r[0] if post else None, rstd_pre=r[1] if dn else None,
                                        dpost_gain=out["dpost_gain"], dgate=out["dgate"], dpre_gain=out["dpre_gain"])
        return {n: a for n, a in out.items() if a is not None}
    good = run()
    cm.coli_moe_block_norm_set_wait_test(withhold)
    try:
        bad = run()
    finally:
        cm.coli_moe_block_norm_set_wait_test(-1)
    rows = torch.isnan(bad["dx"]).all(1)
    assert torch.equal(torch.isnan(bad["dx"]).any(1), rows)                 # whole rows
    at = torch.nonzero(rows)[:, 0].tolist()
    step = at[1] - at[0]
    assert at == list(range(withhold * step, T, step)) and step % 148 == 0   # one CTA's
    for n, a in bad.items():
        if n in ("dx", "d_o") or (n == "dgate" and gate in ("token", "full")):
            assert torch.isnan(a[rows]).all() and torch.equal(a[~rows], good[n][~rows]), n
        else:
            assert torch.isnan(a).all(), n
    again = run()
    for n in good:
        assert torch.equal(again[n], good[n]), n
