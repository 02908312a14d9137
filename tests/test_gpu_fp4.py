"""The 4-bit floating point quantiser (bit for bit) and the grouped product against
their plain forms."""
import numpy as np
import pytest
import torch

import int4_routed_expert_top_b200 as cm
from tests import fp4_format as ff

pytestmark = pytest.mark.gpu

FMT = {"mx": cm.COLI_MXFP4, "nv": cm.COLI_NVFP4}
F, B = torch.float32, torch.bfloat16
HALF = {F: 2.0 ** -24, B: 2.0 ** -8}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def quantize(fmt, x, rows, K, fill=0xAA, **kw):
    nc, ns = cm.coli_moe_fp4_bytes(FMT[fmt], rows, K)
    codes = torch.full((nc,), fill, dtype=torch.uint8, device="cuda")
    scales = torch.full((ns,), fill, dtype=torch.uint8, device="cuda")
    cm.coli_moe_fp4_quantize(FMT[fmt], x, rows, K, codes, scales, **kw)
    return codes, scales


def check_codes(fmt, codes, scales, want, rows, K):
    c0, b0, _ = want
    np.testing.assert_array_equal(codes.cpu().numpy().reshape(rows, K // 2), c0)
    nb = K // ff.BLOCK[fmt]
    got = ff.untile_scales(scales.cpu().numpy(), rows, nb)
    np.testing.assert_array_equal(got[:, :nb], b0)
    assert (got[:, nb:] == 0).all()   # blocks past the row's end


def hard_rows(K, seed=1):
    """Rows of every sort: ordinary, ties, powers of two, tiny, huge, zero, outliers."""
    rng = np.random.default_rng(seed)
    rows = [rng.standard_normal(K), rng.standard_normal(K) * 2.0 ** rng.integers(-12, 12, K), np.zeros(K),
            rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 8.0, -0.25, -5.0], K),
            2.0 ** rng.integers(-6, 7, K).astype(float), np.full(K, 1e-38), np.full(K, -3e38),
            rng.standard_normal(K) * 1e-40, np.where(np.arange(K) % 37 == 0, 300.0, 1e-3), -np.zeros(K),
            rng.standard_normal(K) * 1e-30, np.full(K, 6.0 * 448)]
    return np.stack(rows).astype(np.float32)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("dt", [F, B])
@pytest.mark.parametrize("K", [32, 64, 96, 160, 256, 288, 1024, 6144])
def test_quantize_bits(fmt, dt, K):
    x = dev(hard_rows(K)).to(dt)
    rows = x.shape[0]
    for g in ([None] if fmt == "mx" else [None, 0.0125, 2.0 ** -20, 3.7]):
        want = ff.quantize(x.float().cpu().numpy(), fmt, g)
        gs = None if g is None else torch.tensor([g], device="cuda")
        vals = torch.full((rows, K), 9.0, dtype=dt, device="cuda")
        codes, scales = quantize(fmt, x, rows, K, gscale=gs, values=vals)
        check_codes(fmt, codes, scales, want, rows, K)
        assert torch.equal(vals, dev(want[2]).to(dt))
        c2, s2 = quantize(fmt, x, rows, K, gscale=gs)
        assert torch.equal(c2, codes)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("rows", [1, 127, 128, 129, 300])
@pytest.mark.parametrize("K", [32, 96, 128, 160, 224, 256, 544])
def test_quantize_many_rows(fmt, rows, K):
    x = np.random.default_rng(rows).standard_normal((rows, K)).astype(np.float32)
    codes, scales = quantize(fmt, dev(x), rows, K)
    check_codes(fmt, codes, scales, ff.quantize(x, fmt), rows, K)


@pytest.mark.parametrize("fmt", list(FMT))
def test_quantize_blocks_without_a_number(fmt):
    x = np.random.default_rng(2).standard_normal((4, 128)).astype(np.float32)
    x[0, 5], x[1, 40], x[2, 100] = np.inf, -np.inf, np.nan
    vals = torch.empty(4, 128, device="cuda")
    codes, scales = quantize(fmt, dev(x), 4, 128, values=vals)
    want = ff.quantize(x, fmt)
    check_codes(fmt, codes, scales, want, 4, 128)
    assert np.array_equal(vals.cpu().numpy(), want[2], equal_nan=True) and np.isnan(want[2]).any()


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("act", [cm.COLI_ACT_NONE, cm.COLI_ACT_SWIGLU])
def test_quantize_picked_rows_and_count(fmt, act):
    K, n, rows = 96, 5, 9
    x = np.random.default_rng(3).integers(-8, 9, (n, K * (1 + act))).astype(np.float32)
    src = np.array([4, 0, 0, 2, -1, 5, 3, 1, 2], np.int32)
    count = torch.tensor([7], dtype=torch.int32, device="cuda")
    nc, ns = cm.coli_moe_fp4_bytes(FMT[fmt], rows, K)
    codes, scales = (torch.full((m,), 0xAA, dtype=torch.uint8, device="cuda") for m in (nc, ns))
    vals = torch.full((rows, K), 9.0, device="cuda")
    cm.coli_moe_fp4_quantize(FMT[fmt], dev(x), rows, K, codes, scales, act=act, src=dev(src), count=count, values=vals)
    if act:
        # the same SwiGLU in f32 through the library's plain rows: any rounding of silu is its own
        t = dev(x)
        a = t[:, :K]
        x = ((a / (1 + torch.exp(-a))) * t[:, K:]).cpu().numpy()
    rowsx = np.where(((src >= 0) & (src < n))[:, None], x[np.clip(src, 0, n - 1)], 0)
    _, _, v = ff.quantize(rowsx, fmt)
    got = vals.cpu().numpy()
    assert (got[7:] == 9.0).all() and (codes.cpu().numpy().reshape(rows, -1)[7:] == 0xAA).all()
    assert (got[4:6] == 0).all()
    if not act:
        np.testing.assert_array_equal(got[:7], v[:7])
    else:
        # silu to a few roundings: a value may land one code further where it is next to a
        # tie: half the widest step (2 of 6) more than the rounding itself, on few values
        amax = np.repeat(np.abs(rowsx).reshape(rows, -1, ff.BLOCK[fmt]).max(2), ff.BLOCK[fmt], 1)
        assert (np.abs(got[:7] - v[:7]) <= 0.5 * amax[:7]).all()
        assert (got[:7] != v[:7]).mean() <= 0.01


def weights(fmt, n, K, rng, wide=False):
    """Random codes and scale bytes (as values up to 2^4)."""
    codes = rng.integers(0, 256, (n, K // 2)).astype(np.uint8)
    nb = K // ff.BLOCK[fmt]
    if fmt == "mx":
        byte = rng.integers(100 if wide else 123, 150 if wide else 130, (n, nb))
    else:
        byte = rng.integers(1 if wide else 0x30, 0x7F if wide else 0x48, (n, nb))
    return codes, byte.astype(np.uint8)


def product(fmt, xc, xb, wc, wb, E, R, offsets, alpha, yt, P, K, fill=9.0):
    y = torch.full((P, R), fill, dtype=yt, device="cuda")
    ws = torch.full((cm.coli_moe_fp4_product_workspace_size(FMT[fmt], P, K, E, R),), 255, dtype=torch.uint8, device="cuda")
    off = None if offsets is None else dev(np.asarray(offsets, np.int32))
    args = (FMT[fmt], dev(xc.reshape(-1)), dev(ff.tile_scales(xb)), P, K, dev(wc.reshape(-1)), dev(ff.tile_scales(wb)), E, R)
    cm.coli_moe_fp4_product(*args, y, ws, offsets=off, alpha=None if alpha is None else dev(alpha))
    assert cm.coli_moe_fp4_product_status(ws) == 0
    return y


def check_product(fmt, E, R, K, sizes, yt=F, seed=0, wide=False, alpha=True):
    rng = np.random.default_rng(seed)
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    P = int(offsets[-1]) + (3 if E > 1 else 0)   # rows behind the last expert's
    xc, xb = weights(fmt, P, K, rng, wide)
    wc, wb = weights(fmt, E * R, K, rng, wide)
    al = (0.5 + rng.random(E)).astype(np.float32) if alpha else None
    y = product(fmt, xc, xb, wc, wb, E, R, offsets if E > 1 else None, al, yt, P, K)
    X, W = dev(ff.values(xc, xb, fmt)), dev(ff.values(wc, wb, fmt))
    off2 = 0.0
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        a = 1.0 if al is None else float(al[e])
        w = W[e * R:(e + 1) * R]
        want, size = a * (X[lo:hi] @ w.T), a * (X[lo:hi].abs() @ w.abs().T)
        err = (y[lo:hi].double() - want).abs()
        # products are exact; one addition into the f32 accumulator per 64 columns, each off by
        # at most two units of the last place of a partial sum (2^-22 of the terms' size), the
        # joined pieces, the factor and the output's rounding
        bound = (-(-K // 64) + 24) * 2.0 ** -22 * size + HALF[yt] * want.abs()
        assert (err <= bound + 1e-30).all(), (e, float((err - bound).max()))
        off2 += float(err.square().sum() / want.square().sum().clamp(min=1e-30)) / E if hi > lo else 0.0
    assert (y[int(offsets[-1]):] == 9.0).all()
    return off2 ** 0.5


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("R,K,n", [(128, 256, 1), (128, 32, 3), (128, 64, 16), (1, 256, 1), (5, 96, 2), (130, 160, 17),
                                   (256, 512, 33), (384, 288, 48), (200, 1056, 31), (6144, 2048, 1)])
def test_product_one_group(fmt, R, K, n):
    for yt in (F, B):
        check_product(fmt, 1, R, K, [n], yt)


@pytest.mark.parametrize("fmt", list(FMT))
# 40 tiles of 256 x 224 or more: pairs of CTAs; the others one CTA by itself with several row tiles
@pytest.mark.parametrize("R,K,n", [(128, 256, 49), (100, 1024, 192), (384, 2048, 193), (1000, 96, 500), (256, 6144, 400),
                                   (10240, 256, 49), (10240, 512, 128), (10112, 288, 129), (10100, 1024, 192),
                                   (10240, 2048, 193), (10496, 512, 224), (5248, 768, 225), (5120, 96, 440),
                                   (10240, 6144, 40), (20000, 128, 449)])
def test_product_one_group_many_rows(fmt, R, K, n):
    for yt in (F, B):
        check_product(fmt, 1, R, K, [n], yt)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("R,K,sizes", [
    (128, 256, [0, 1, 0, 5, 2, 0]), (256, 512, [0] * 30 + [1] + [0] * 33), (128, 96, [31, 32, 33, 64, 65]),
    (256, 1024, [7] * 9), (128, 512, [0, 300, 0, 1, 200, 17]), (384, 2048, [130, 259, 5, 0]),
    (128, 64, [1] * 1024), (4096, 256, [1, 0, 0, 1, 1, 0, 2, 0] * 4),
    (1792, 256, [0, 300, 0, 1, 200, 17]), (1920, 512, [0, 300, 0, 1, 200, 17]),     # pairs
    (2688, 2048, [130, 259, 5, 0]), (256, 160, [33] * 45), (128, 320, [40, 0, 225, 3] * 12)])
def test_product_groups(fmt, R, K, sizes):
    for yt in (F, B):
        check_product(fmt, len(sizes), R, K, sizes, yt, seed=len(sizes))


@pytest.mark.parametrize("tiles,K,n", [(149, 512, 1), (149, 768, 2), (150, 1024, 1), (297, 512, 1), (75, 512, 60),
                                       (75, 768, 50), (76, 1280, 49), (151, 512, 100), (222, 768, 64)])
def test_product_few_tiles_left_over(tiles, K, n):
    """A little more than whole waves of tiles (148 CTAs, or 74 pairs of them): the rest has
    fewer stages than there are CTAs, so that some get none."""
    rows = 128 if n <= 48 else 256
    check_product("mx", 1, rows * tiles, K, [n])


@pytest.mark.parametrize("fmt", list(FMT))
def test_product_wide_scales_and_no_alpha(fmt):
    check_product(fmt, 3, 256, 512, [4, 70, 9], wide=True, alpha=False)


@pytest.mark.parametrize("fmt", list(FMT))
def test_product_accuracy(fmt):
    """The sum over 6144 columns in f32: near the rounding of one f32 sum, for few and many rows."""
    assert check_product(fmt, 1, 256, 6144, [5]) <= 5e-6
    assert check_product(fmt, 1, 256, 6144, [300]) <= 5e-6
    assert check_product(fmt, 1, 10240, 6144, [60]) <= 5e-6


def test_product_nan_scale_stays_in_its_row():
    rng = np.random.default_rng(8)
    xc, xb = weights("mx", 40, 256, rng)
    wc, wb = weights("mx", 256, 256, rng)
    xb[7, 3], wb[100, 0] = 255, 255
    y = product("mx", xc, xb, wc, wb, 1, 256, None, None, F, 40, 256).cpu().numpy()
    want = np.zeros((40, 256), bool)
    want[7], want[:, 100] = True, True
    np.testing.assert_array_equal(np.isnan(y), want)


def test_product_offsets_out_of_range_stay_in_bounds():
    rng = np.random.default_rng(9)
    xc, xb = weights("nv", 10, 128, rng)
    wc, wb = weights("nv", 4 * 128, 128, rng)
    good = product("nv", xc, xb, wc, wb, 4, 128, [0, 2, 5, 10, 10], None, F, 10, 128)
    same = product("nv", xc, xb, wc, wb, 4, 128, [-3, 2, 5, 99, 50], None, F, 10, 128)
    assert torch.equal(good, same)


@pytest.mark.parametrize("R", [256, 1408])
def test_product_is_the_same_every_time(R):
    rng = np.random.default_rng(10)
    xc, xb = weights("mx", 700, 1024, rng)
    wc, wb = weights("mx", 8 * R, 1024, rng)
    off = [0, 100, 100, 350, 360, 400, 650, 651, 700]
    a = product("mx", xc, xb, wc, wb, 8, R, off, None, F, 700, 1024)
    for _ in range(3):
        assert torch.equal(a, product("mx", xc, xb, wc, wb, 8, R, off, None, F, 700, 1024))
    assert float((a[400:650] - product("mx", xc[400:650], xb[400:650], wc[5 * R:6 * R], wb[5 * R:6 * R], 1, R,
                                       None, None, F, 250, 1024)).abs().max()) <= 1e-5 * float(a.abs().max())


def test_product_one_expert_with_offsets():
    """E = 1 with offsets: only the rows they name."""
    rng = np.random.default_rng(11)
    for P, R in ((20, 128), (90, 128), (90, 10240)):
        xc, xb = weights("mx", P, 256, rng)
        wc, wb = weights("mx", R, 256, rng)
        all_rows = product("mx", xc, xb, wc, wb, 1, R, None, None, F, P, 256)
        some = product("mx", xc, xb, wc, wb, 1, R, [3, P - 5], None, F, P, 256)
        assert (some[:3] == 9.0).all() and (some[P - 5:] == 9.0).all()
        X, W = dev(ff.values(xc, xb, "mx")), dev(ff.values(wc, wb, "mx"))
        want, size = X @ W.T, X.abs() @ W.abs().T
        for y, lo, hi in ((all_rows, 0, P), (some, 3, P - 5)):
            assert ((y[lo:hi].double() - want[lo:hi]).abs() <= 28 * 2.0 ** -22 * size[lo:hi]).all()


def test_product_two_streams_at_once():
    """Two calls with their own workspaces, their CTAs taking turns on the SMs."""
    rng = np.random.default_rng(12)
    calls = []
    for n, R in ((40, 19200), (700, 9728), (3, 38400)):
        xc, xb = weights("mx", n, 512, rng)
        wc, wb = weights("mx", R, 512, rng)
        args = [dev(xc.reshape(-1)), dev(ff.tile_scales(xb)), n, 512, dev(wc.reshape(-1)), dev(ff.tile_scales(wb)), 1, R]
        size = cm.coli_moe_fp4_product_workspace_size(FMT["mx"], n, 512, 1, R)
        want, ws = torch.empty(n, R, device="cuda"), torch.zeros(size, dtype=torch.uint8, device="cuda")
        cm.coli_moe_fp4_product(FMT["mx"], *args, want, ws)
        calls.append((args, want, torch.empty_like(want), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for args, _, y, ws, stream in calls:
            cm.coli_moe_fp4_product(FMT["mx"], *args, y, ws, stream=stream)
    torch.cuda.synchronize()
    for _, want, y, ws, _ in calls:
        assert cm.coli_moe_fp4_product_status(ws) == 0 and torch.equal(y, want)


@pytest.mark.parametrize("P,R", [(2 ** 31 - 1, 1), (1, 2 ** 31 - 1), (33, 2 ** 26 + 1)])
def test_product_of_the_most_rows(P, R):
    """As many rows of either side as their 31 bits allow, a K of one block: zeros but for
    the last rows (and one a third of the way), whose products are whole numbers."""
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        pytest.skip("needs 70 GB")
    K = 32

    def side(n, seed):
        nc, ns = cm.coli_moe_fp4_bytes(cm.COLI_MXFP4, n, K)
        codes, scales = (torch.zeros(m, dtype=torch.uint8, device="cuda") for m in (nc, ns))
        scales.view(-1, 4)[:, 0] = 127
        at = sorted({n // 3, *range(max(0, n - 300), n)})
        small = np.random.default_rng(seed).integers(0, 256, (len(at), K // 2)).astype(np.uint8)
        codes.view(n, K // 2)[torch.tensor(at, device="cuda")] = dev(small)
        return codes, scales, at, ff.values(small, np.full((len(at), 1), 127, np.uint8), "mx")
    xc, xs, xat, X = side(P, 1)
    wc, ws_, wat, W = side(R, 2)
    y = torch.full((P, R), 9.0, dtype=B, device="cuda")
    ws = torch.zeros(cm.coli_moe_fp4_product_workspace_size(cm.COLI_MXFP4, P, K, 1, R), dtype=torch.uint8, device="cuda")
    cm.coli_moe_fp4_product(cm.COLI_MXFP4, xc, xs, P, K, wc, ws_, 1, R, y, ws)
    assert cm.coli_moe_fp4_product_status(ws) == 0
    i, j = torch.tensor(xat, device="cuda"), torch.tensor(wat, device="cuda")
    # sums of 32 multiples of 0.25 up to 36: exact in f32, so one rounding to bf16 and nothing else
    assert torch.equal(y[i][:, j], dev((X @ W.T).astype(np.float32)).to(B))
    y[i[:, None], j] = 0
    assert int(torch.count_nonzero(y)) == 0


def pair_inputs(fmt, sizes, R, K, seed):
    """Inputs of a grouped product whose scales differ from stage to stage by many powers of two."""
    rng = np.random.default_rng(seed)
    P, E = sum(sizes), len(sizes)
    lo, hi, block = (100, 150, 32) if fmt == "mx" else (0x08, 0x78, 16)
    sides = []
    for n in (P, E * R):
        codes = rng.integers(0, 256, (n, K // 2)).astype(np.uint8)
        stage = rng.integers(lo, hi, (n, -(-K // 256)))     # a base for each 256 columns, and a little about it
        byte = np.repeat(stage, 256 // block, 1)[:, :K // block] + rng.integers(0, 4, (n, K // block))
        sides.append((codes, byte.astype(np.uint8)))
    return sides, np.concatenate([[0], np.cumsum(sizes)])


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("sizes,R,K", [([1, 32, 94, 225, 0, 127, 449, 33], 2560, 2080), ([700], 5120, 2208)])
def test_product_of_pairs_reads_no_stale_scales(fmt, sizes, R, K):
    """Two sets of inputs in turn through the same buffers and workspace, many times: the same
    bits every time, those of a first call, which are right."""
    P, E = sum(sizes), len(sizes)
    assert in_pairs(fmt, E, R, K, P)
    sets, want = [], []
    for seed in (1, 2):
        ((xc, xb), (wc, wb)), off = pair_inputs(fmt, sizes, R, K, seed)
        y = product(fmt, xc, xb, wc, wb, E, R, off if E > 1 else None, None, F, P, K)
        X, W = dev(ff.values(xc, xb, fmt)), dev(ff.values(wc, wb, fmt))
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            w = W[e * R:(e + 1) * R]
            size = X[lo:hi].abs() @ w.abs().T   # the bound of check_product
            assert ((y[lo:hi].double() - X[lo:hi] @ w.T).abs() <= (-(-K // 64) + 24) * 2.0 ** -22 * size).all()
        want.append(y)
        sets.append([dev(a) for a in (xc.reshape(-1), ff.tile_scales(xb), wc.reshape(-1), ff.tile_scales(wb))])
    offsets = dev(off.astype(np.int32))
    ws = torch.zeros(cm.coli_moe_fp4_product_workspace_size(FMT[fmt], P, K, E, R), dtype=torch.uint8, device="cuda")
    xc, xs, wc, wsc = (torch.empty_like(a) for a in sets[0])
    y, wrong = torch.empty_like(want[0]), torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(60):
        for to, a in zip((xc, xs, wc, wsc), sets[i & 1]):
            to.copy_(a)
        cm.coli_moe_fp4_product(FMT[fmt], xc, xs, P, K, wc, wsc, E, R, y, ws, offsets=offsets if E > 1 else None)
        wrong += (y != want[i & 1]).sum()
    assert int(wrong) == 0 and cm.coli_moe_fp4_product_status(ws) == 0


def test_product_of_pairs_with_offsets_that_overlap_stays_in_bounds():
    """Offsets that are not ascending name more row tiles than P rows have."""
    P, R, K, E = 900, 2560, 2048, 8
    rng = np.random.default_rng(3)
    xc, xb = weights("mx", P, K, rng)
    wc, wb = weights("mx", E * R, K, rng)
    size = cm.coli_moe_fp4_product_workspace_size(cm.COLI_MXFP4, P, K, E, R)
    assert in_pairs("mx", E, R, K, P)
    y, ws = torch.full((P + 300, R), 9.0, device="cuda"), torch.full((size + 65536,), 7, dtype=torch.uint8, device="cuda")
    off = dev(np.array([0, P, 0, P, 0, P, 0, P, 0], np.int32))
    cm.coli_moe_fp4_product(cm.COLI_MXFP4, dev(xc.reshape(-1)), dev(ff.tile_scales(xb)), P, K, dev(wc.reshape(-1)),
                            dev(ff.tile_scales(wb)), E, R, y[:P], ws[:size], offsets=off)
    assert cm.coli_moe_fp4_product_status(ws) == 0
    assert (y[P:] == 9.0).all() and (ws[size:] == 7).all()


def in_pairs(fmt, E, R, K, n):
    """Whether a product takes pairs of CTAs, by the workspace that these need."""
    size = cm.coli_moe_fp4_product_workspace_size
    return size(FMT[fmt], n, K, E, R) > size(FMT[fmt], 1, K, E, R)


@pytest.mark.parametrize("fmt", list(FMT))
# row counts about the ends of half tiles and tiles, last weight rows and columns of every sort
@pytest.mark.parametrize("R,K,n", [(35300, 96, 440), (70300, 32, 225), (14100, 1056, 224), (10240, 2048, 193), (6000, 2208, 449),
                                   (33920, 1024, 129), (33000, 1184, 128), (10300, 6144, 97), (70400, 256, 250)])
def test_product_in_pairs_one_group(fmt, R, K, n):
    assert in_pairs(fmt, 1, R, K, n)
    for yt in (F, B):
        check_product(fmt, 1, R, K, [n], yt)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("R,K,sizes", [(3456, 1024, [0, 300, 0, 1, 200, 817]), (2688, 2080, [130, 859, 5, 0]),
                                       (640, 800, [129, 0, 225, 3, 400] * 9), (128, 2560, [33, 70, 224, 225, 500] * 12)])
def test_product_in_pairs_groups(fmt, R, K, sizes):
    assert in_pairs(fmt, len(sizes), R, K, sum(sizes))
    for yt in (F, B):
        check_product(fmt, len(sizes), R, K, sizes, yt, seed=len(sizes))


@pytest.mark.parametrize("tiles,K,n", [(75, 1024, 193), (76, 1280, 200), (151, 512, 193), (222, 768, 97), (75, 512, 449)])
def test_product_in_pairs_few_tiles_left_over(tiles, K, n):
    assert in_pairs("mx", 1, 256 * tiles, K, n)
    check_product("mx", 1, 256 * tiles, K, [n])


@pytest.mark.parametrize("fmt", list(FMT))
def test_product_in_pairs_accuracy_and_wide_scales(fmt):
    assert check_product(fmt, 1, 10240, 6144, [97]) <= 5e-6
    check_product(fmt, 3, 5120, 2048, [90, 370, 200], wide=True, alpha=False)


def test_product_in_pairs_nan_scale_stays_in_its_row():
    rng = np.random.default_rng(8)
    xc, xb = weights("mx", 440, 96, rng)
    wc, wb = weights("mx", 35300, 96, rng)
    xb[7, 2], xb[300, 0], wb[100, 0], wb[35299, 1] = 255, 255, 255, 255
    y = torch.isnan(product("mx", xc, xb, wc, wb, 1, 35300, None, None, F, 440, 96))
    want = torch.zeros_like(y)
    for r in (7, 300):
        want[r] = True
    for c in (100, 35299):
        want[:, c] = True
    assert torch.equal(y, want)


def test_product_in_pairs_one_expert_with_offsets():
    rng = np.random.default_rng(11)
    P, R, K = 440, 35300, 256
    xc, xb = weights("mx", P, K, rng)
    wc, wb = weights("mx", R, K, rng)
    y = product("mx", xc, xb, wc, wb, 1, R, [3, P - 5], None, F, P, K)
    assert (y[:3] == 9.0).all() and (y[P - 5:] == 9.0).all()
    X, W = dev(ff.values(xc, xb, "mx")), dev(ff.values(wc, wb, "mx"))
    assert ((y[3:P - 5].double() - (X @ W.T)[3:P - 5]).abs() <= 28 * 2.0 ** -22 * (X.abs() @ W.abs().T)[3:P - 5]).all()


def test_product_in_pairs_on_two_streams_at_once():
    """Pairs of two calls and CTAs by themselves of a third taking turns on the SMs."""
    rng = np.random.default_rng(12)
    calls = []
    for n, R in ((200, 38400), (700, 12800), (3, 38400)):
        xc, xb = weights("mx", n, 512, rng)
        wc, wb = weights("mx", R, 512, rng)
        args = [dev(xc.reshape(-1)), dev(ff.tile_scales(xb)), n, 512, dev(wc.reshape(-1)), dev(ff.tile_scales(wb)), 1, R]
        assert in_pairs("mx", 1, R, 512, n) == (n > 3)
        size = cm.coli_moe_fp4_product_workspace_size(FMT["mx"], n, 512, 1, R)
        want, ws = torch.empty(n, R, device="cuda"), torch.zeros(size, dtype=torch.uint8, device="cuda")
        cm.coli_moe_fp4_product(FMT["mx"], *args, want, ws)
        calls.append((args, want, torch.empty_like(want), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for args, _, y, ws, stream in calls:
            cm.coli_moe_fp4_product(FMT["mx"], *args, y, ws, stream=stream)
    torch.cuda.synchronize()
    for _, want, y, ws, _ in calls:
        assert cm.coli_moe_fp4_product_status(ws) == 0 and torch.equal(y, want)
