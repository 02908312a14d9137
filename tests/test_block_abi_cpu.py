"""Refusals of the operators around the experts (status codes before any launch),
their sizes, and the plain 4-bit formats that the GPU tests use.  No GPU."""
import ctypes
import math

import numpy as np
import pytest

import int4_routed_expert_top_b200 as cm
from tests import fp4_format as ff

INVAL, UNSUPPORTED, WORKSPACE = -1, -4, -5
A = 1 << 20  # an aligned address that no refused call touches


def code(name, *args):
    return getattr(cm.lib, name)(*args)


SORT = dict(idx=A, w=None, T=4, k=2, E=8, off=A, tok=A, slot=A, inv=A, ws=None, n=0, s=None)
DISPATCH = dict(x=A, xt=0, T=4, H=64, k=2, inv=A, xs=A, s=None)
COMBINE = dict(o=A, ot=0, T=4, H=64, k=2, inv=A, w=A, res=None, y=A, yt=0, s=None)
COMBINE_B = dict(dy=A, yt=0, o=A, ot=0, T=4, H=64, k=2, inv=A, w=A, do=A, dw=A, s=None)
QUANT = dict(fmt=0, x=A, xt=0, n=8, rows=8, K=64, act=0, src=None, count=None, g=None, c=A, sc=A, v=None, s=None)
PRODUCT = dict(fmt=0, xc=A, xs=A, P=8, K=64, wc=A, ws=A, E=2, R=128, off=A, al=None, y=A, yt=0, w=A,
               n=1 << 40, s=None)


@pytest.mark.parametrize("name,good,change,want", [
    ("coli_moe_sort", SORT, dict(idx=None), INVAL),
    ("coli_moe_sort", SORT, dict(off=None), INVAL),
    ("coli_moe_sort", SORT, dict(inv=None), INVAL),
    ("coli_moe_sort", SORT, dict(k=0), INVAL),
    ("coli_moe_sort", SORT, dict(k=33), INVAL),
    ("coli_moe_sort", SORT, dict(E=0), INVAL),
    ("coli_moe_sort", SORT, dict(E=1025), INVAL),
    ("coli_moe_sort", SORT, dict(T=-1), INVAL),
    ("coli_moe_sort", SORT, dict(T=1 << 30), INVAL),
    ("coli_moe_sort", SORT, dict(T=8192, k=8), WORKSPACE),
    ("coli_moe_sort", SORT, dict(T=8192, k=8, ws=A, n=4), WORKSPACE),
    ("coli_moe_dispatch", DISPATCH, dict(x=None), INVAL),
    ("coli_moe_dispatch", DISPATCH, dict(xs=None), INVAL),
    ("coli_moe_dispatch", DISPATCH, dict(xt=2), INVAL),
    ("coli_moe_dispatch", DISPATCH, dict(H=0), INVAL),
    ("coli_moe_dispatch", DISPATCH, dict(T=1, H=(1 << 24) + 1), INVAL),
    ("coli_moe_dispatch", DISPATCH, dict(T=1 << 24, k=32, H=1 << 17), INVAL),
    ("coli_moe_dispatch_backward", DISPATCH, dict(inv=None), INVAL),
    ("coli_moe_combine", COMBINE, dict(o=None), INVAL),
    ("coli_moe_combine", COMBINE, dict(y=None), INVAL),
    ("coli_moe_combine", COMBINE, dict(yt=7), INVAL),
    ("coli_moe_combine_backward", COMBINE_B, dict(dy=None), INVAL),
    ("coli_moe_combine_backward", COMBINE_B, dict(do=None, dw=None), INVAL),
    ("coli_moe_combine_backward", COMBINE_B, dict(o=None), INVAL),
    ("coli_moe_fp4_quantize", QUANT, dict(fmt=2), INVAL),
    ("coli_moe_fp4_quantize", QUANT, dict(K=48), INVAL),
    ("coli_moe_fp4_quantize", QUANT, dict(K=0), INVAL),
    ("coli_moe_fp4_quantize", QUANT, dict(rows=-1), INVAL),
    ("coli_moe_fp4_quantize", QUANT, dict(n=7), INVAL),
    ("coli_moe_fp4_quantize", QUANT, dict(act=2), INVAL),
    ("coli_moe_fp4_quantize", QUANT, dict(g=A), INVAL),
    ("coli_moe_fp4_quantize", QUANT, dict(x=A + 8), INVAL),
    ("coli_moe_fp4_quantize", QUANT, dict(v=A + 4), INVAL),
    ("coli_moe_fp4_quantize", QUANT, dict(c=None), INVAL),
    ("coli_moe_fp4_product", PRODUCT, dict(R=100), INVAL),
    ("coli_moe_fp4_product", PRODUCT, dict(E=1025), INVAL),
    ("coli_moe_fp4_product", PRODUCT, dict(off=None), INVAL),
    ("coli_moe_fp4_product", PRODUCT, dict(K=100), INVAL),
    ("coli_moe_fp4_product", PRODUCT, dict(yt=3), INVAL),
    ("coli_moe_fp4_product", PRODUCT, dict(E=1 << 9, R=1 << 23), INVAL),
    ("coli_moe_fp4_product", PRODUCT, dict(xc=A + 4), INVAL),
    ("coli_moe_fp4_product", PRODUCT, dict(y=None), INVAL),
    ("coli_moe_fp4_product", PRODUCT, dict(w=None), WORKSPACE),
    ("coli_moe_fp4_product", PRODUCT, dict(n=1000), WORKSPACE),
])
def test_refusals(name, good, change, want):
    assert code(name, *{**good, **change}.values()) == want
    assert cm.coli_moe_last_error()


def norm(**kw):
    d = dict(H=64, xt=0, bt=1, post_norm=1, gate_kind=1, alpha=1.0, eps=1e-5, post_gain=A, pre_gain=A)
    d.update(kw)
    return ctypes.byref(cm.NormDesc(*d.values()))


NORM = dict(desc=norm(), x=A, o=A, gate=A, T=4, xo=A, no=A, rp=None, rx=None, s=None)
NORM_B = dict(desc=norm(), xo=A, o=A, gate=A, T=4, rp=A, rx=A, dxo=A, dn=A, dx=A, do=A, dpost=A, dgate=A, dpre=A,
              ws=A, n=1 << 40, s=None)


@pytest.mark.parametrize("name,good,change,want", [
    ("coli_moe_block_norm", NORM, dict(desc=None), INVAL),
    ("coli_moe_block_norm", NORM, dict(desc=norm(H=0)), INVAL),
    ("coli_moe_block_norm", NORM, dict(desc=norm(H=16385)), INVAL),
    ("coli_moe_block_norm", NORM, dict(desc=norm(xt=1, bt=0)), UNSUPPORTED),
    ("coli_moe_block_norm", NORM, dict(desc=norm(gate_kind=4)), INVAL),
    ("coli_moe_block_norm", NORM, dict(desc=norm(eps=0.0)), INVAL),
    ("coli_moe_block_norm", NORM, dict(desc=norm(eps=math.nan)), INVAL),
    ("coli_moe_block_norm", NORM, dict(desc=norm(alpha=math.inf)), INVAL),
    ("coli_moe_block_norm", NORM, dict(gate=None), INVAL),
    ("coli_moe_block_norm", NORM, dict(desc=norm(gate_kind=0)), INVAL),
    ("coli_moe_block_norm", NORM, dict(x=None), INVAL),
    ("coli_moe_block_norm", NORM, dict(xo=None), INVAL),
    ("coli_moe_block_norm", NORM, dict(o=None, no=None), INVAL),
    ("coli_moe_block_norm", NORM, dict(T=-1), INVAL),
    ("coli_moe_block_norm_backward", NORM_B, dict(dx=None), INVAL),
    ("coli_moe_block_norm_backward", NORM_B, dict(dxo=None, dn=None), INVAL),
    ("coli_moe_block_norm_backward", NORM_B, dict(do=None), INVAL),
    ("coli_moe_block_norm_backward", NORM_B, dict(o=None), INVAL),
    ("coli_moe_block_norm_backward", NORM_B, dict(rx=None), INVAL),
    ("coli_moe_block_norm_backward", NORM_B, dict(rp=None), INVAL),
    ("coli_moe_block_norm_backward", NORM_B, dict(desc=norm(post_norm=0)), INVAL),   # dpost_gain asked for
    ("coli_moe_block_norm_backward", NORM_B, dict(desc=norm(gate_kind=0), gate=None), INVAL),
    ("coli_moe_block_norm_backward", NORM_B, dict(ws=None), WORKSPACE),
    ("coli_moe_block_norm_backward", NORM_B, dict(n=16), WORKSPACE),
])
def test_norm_refusals(name, good, change, want):
    assert code(name, *{**good, **change}.values()) == want
    assert cm.coli_moe_last_error()


@pytest.mark.parametrize("name,good,buffers", [
    ("coli_moe_sort", {**SORT, "w": A}, "idx w off tok slot inv"),
    ("coli_moe_dispatch", DISPATCH, "x inv xs"),
    ("coli_moe_dispatch_backward", DISPATCH, "x inv xs"),
    ("coli_moe_combine", {**COMBINE, "res": A}, "o inv w res y"),
    ("coli_moe_combine_backward", COMBINE_B, "dy o inv w do dw"),
    ("coli_moe_fp4_quantize", {**QUANT, "fmt": 1, "src": A, "count": A, "g": A, "v": A}, "x src count g c sc v"),
    ("coli_moe_fp4_product", {**PRODUCT, "al": A}, "xc xs wc ws off al y"),
    ("coli_moe_block_norm", {**NORM, "rp": A, "rx": A}, "x o gate xo no rp rx"),
    ("coli_moe_block_norm_backward", NORM_B, "xo o gate rp rx dxo dn dx do dpost dgate dpre"),
])
def test_addresses_between_elements_are_refused(name, good, buffers):
    for b in buffers.split():
        assert code(name, *{**good, b: A + 1}.values()) == INVAL, b
        assert cm.coli_moe_last_error()


def test_nothing_to_do_succeeds():
    assert code("coli_moe_dispatch", *{**DISPATCH, "T": 0, "x": None}.values()) == 0
    assert code("coli_moe_combine", *{**COMBINE, "T": 0}.values()) == 0
    assert code("coli_moe_combine_backward", *{**COMBINE_B, "T": 0}.values()) == 0
    assert code("coli_moe_block_norm", *{**NORM, "T": 0}.values()) == 0
    assert code("coli_moe_fp4_quantize", *{**QUANT, "rows": 0}.values()) == 0
    assert code("coli_moe_fp4_product", *{**PRODUCT, "P": 0}.values()) == 0


def test_sizes():
    assert cm.coli_moe_sort_workspace_size(1, 8, 256) == 0
    assert cm.coli_moe_sort_workspace_size(8192, 8, 256) >= 256 * 4
    assert cm.coli_moe_fp4_bytes(cm.COLI_MXFP4, 130, 160) == (130 * 80, 2 * 2 * 512)
    assert cm.coli_moe_fp4_bytes(cm.COLI_NVFP4, 130, 160) == (130 * 80, 2 * 3 * 512)
    small = cm.coli_moe_fp4_product_workspace_size(cm.COLI_MXFP4, 8, 64, 256, 128)
    assert small < cm.coli_moe_fp4_product_workspace_size(cm.COLI_MXFP4, 1 << 16, 64, 32, 256)


def test_plain_format_hand_values():
    # one block of each kind by hand: max 6.5 = 1.625 * 2^2 -> scale 2^0, 6.5 saturates to 6;
    # 2.5, 0.25, 5 tie to even (2, 0, 4); 3.5 -> 4; -0.75 -> -1
    x = np.zeros((1, 32), np.float32)
    x[0, :8] = [6.5, 2.5, 0.25, 5.0, 3.5, -0.75, 1.25, -1.75]
    codes, byte, val = ff.quantize(x, "mx")
    assert byte.tolist() == [[127]]
    assert val[0, :8].tolist() == [6, 2, 0, 4, 4, -1, 1, -2]
    assert codes[0, :4].tolist() == [7 | 4 << 4, 0 | 6 << 4, 6 | 10 << 4, 2 | 12 << 4]
    # max 12 with g = 1: s = 2, exactly representable
    x = np.zeros((1, 16), np.float32)
    x[0, :4] = [12, 5, -1, 0.5]
    codes, byte, val = ff.quantize(x, "nv")
    assert ff.E4M3[byte[0, 0]] == 2 and val[0, :4].tolist() == [12, 4, -1, 0]  # 2.5 and 0.25 tie to even


def test_plain_format_round_trip_and_layout():
    rng = np.random.default_rng(5)
    for fmt in ("mx", "nv"):
        x = rng.standard_normal((133, 160)).astype(np.float32)
        codes, byte, val = ff.quantize(x, fmt)
        again = ff.quantize(val, fmt)  # the values are representable: blocks keep their largest magnitude
        np.testing.assert_array_equal(ff.values(codes, byte, fmt).astype(np.float32), val)
        np.testing.assert_array_equal(ff.untile_scales(ff.tile_scales(byte), 133, byte.shape[1])[:, :byte.shape[1]], byte)
        if fmt == "nv":
            np.testing.assert_array_equal(again[2], val)
        # a magnitude is within half of the widest step (2) below 6, or saturated
        err = np.abs(val - x)
        d = np.repeat(np.abs(x).reshape(133, -1, ff.BLOCK[fmt]).max(2), ff.BLOCK[fmt], 1)
        assert (err <= 0.26 * d).all()


def never_smaller(sizes):
    return all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("k,E", [(1, 8), (8, 256), (10, 512), (32, 1024)])
def test_sort_workspace_of_more_tokens_serves_fewer(k, E):
    """A workspace made once for the largest batch takes every smaller one."""
    around = sorted({max(0, n // k + d) for n in (0, 512, 1024, 2048, 32768, 65536, 98304, 1 << 20) for d in range(-3, 4)}
                    | set(range(2000, 8300)))
    assert never_smaller([cm.coli_moe_sort_workspace_size(T, k, E) for T in around])


def test_product_workspace_of_more_rows_serves_fewer():
    for E, R, K in ((1, 1, 32), (1, 4096, 6144), (1, 10240, 256), (1, 10240, 2048), (1, 2560, 6144), (8, 2560, 1024),
                    (32, 256, 64), (32, 4096, 6144), (256, 128, 64), (1024, 128, 32)):
        rows = sorted({n + d for n in (1, 32, 224, 448, 1000, 7168, 32 * E, 224 * E, 30000, 1 << 24) for d in range(0, 3)}
                      | set(range(0, 3000, 7)))
        assert never_smaller([cm.coli_moe_fp4_product_workspace_size(cm.COLI_NVFP4, P, K, E, R) for P in rows])


@pytest.mark.parametrize("H", [1, 8, 64, 130, 1024, 6143, 6144, 8192, 8200, 16384])
@pytest.mark.parametrize("xt,bt", [(0, 0), (0, 1), (1, 1)])
def test_norm_gradient_workspace_of_more_tokens_serves_fewer(H, xt, bt):
    desc = cm.NormDesc(H, xt, bt, 1, cm.COLI_GATE_CHANNEL, 1.0, 1e-5, None, None)
    assert never_smaller([cm.coli_moe_block_norm_backward_workspace_size(desc, T) for T in range(0, 2000)])


def test_norm_gradient_of_no_tokens_needs_no_addresses():
    """Empty tensors have no address: nothing but the sums over tokens is asked of the call."""
    none = {**NORM_B, "T": 0, **{b: None for b in "xo o gate rp rx dxo dn dx do dpost dgate dpre ws".split()}, "n": 0}
    for desc in (norm(gate_kind=0), norm(), norm(gate_kind=2), norm(gate_kind=3, post_norm=0)):
        assert code("coli_moe_block_norm_backward", *{**none, "desc": desc}.values()) == 0
    # what no tensor of any length could be is refused still
    assert code("coli_moe_block_norm_backward", *{**none, "desc": norm(gate_kind=0), "dgate": A}.values()) == INVAL
    assert code("coli_moe_block_norm_backward", *{**none, "desc": norm(post_norm=0), "dpost": A}.values()) == INVAL
    assert code("coli_moe_block_norm_backward", *{**none, "dpre": A + 2}.values()) == INVAL


def test_product_sizes_up_to_31_bits():
    """The number of row tiles of the largest matrices, in 64 bits: a pair of CTAs for each either way."""
    most = 2 ** 31 - 1
    pairs = cm.coli_moe_fp4_product_workspace_size(cm.COLI_MXFP4, 40, 32, 1, 1 << 30)
    assert pairs > cm.coli_moe_fp4_product_workspace_size(cm.COLI_MXFP4, 32, 32, 1, 1 << 30)
    assert cm.coli_moe_fp4_product_workspace_size(cm.COLI_MXFP4, 40, 32, 1, most) == pairs
    assert cm.coli_moe_fp4_product_workspace_size(cm.COLI_MXFP4, most, 32, 1, 1) >= pairs


def test_wait_test_takes_only_what_it_knows():
    assert code("coli_moe_fp4_set_wait_test", 2) == INVAL
    try:
        for withhold in (0, 1):
            assert code("coli_moe_fp4_set_wait_test", withhold) == 0
            for change in (dict(yt=1), dict(fmt=1)):   # refused before any launch
                assert code("coli_moe_fp4_product", *{**PRODUCT, **change}.values()) == UNSUPPORTED
    finally:
        assert code("coli_moe_fp4_set_wait_test", -1) == 0


def test_norm_wait_test_takes_only_what_it_knows():
    try:
        assert code("coli_moe_block_norm_set_wait_test", 0) == 0
        for change in (dict(), dict(T=4000, desc=norm(H=63)), dict(T=4000, desc=norm(bt=0)), dict(T=4000, desc=norm(H=8192))):
            assert code("coli_moe_block_norm_backward", *{**NORM_B, **change}.values()) == UNSUPPORTED
    finally:
        assert code("coli_moe_block_norm_set_wait_test", -1) == 0
