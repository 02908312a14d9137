"""The operators around the experts of a routed MoE block, as measured work.

Five operators, each with its plain form (elementary torch operations in 32 bits),
the library's calls, and its definition in 64 bits:

  dispatch       the picks (token, slot) sorted by expert and the tokens copied
                 into that order (coli_moe_sort, coli_moe_dispatch)
  combine        the experts' rows back to their tokens with the routing weights
                 (coli_moe_combine), and the gradients of both directions
  norm           RMSNorm after a block, its gate and residual scale, the residual
                 sum and the RMSNorm before the next block (coli_moe_block_norm),
                 and the gradient of all of it
  quantize       rows to 4-bit floating point in blocks with a shared scale
                 (coli_moe_fp4_quantize): "mx" = 32 values and a power of two,
                 "nv" = 16 values and an E4M3 scale under one f32 scale
  product        rows of activations, quantised, times the 4-bit weights of the
                 expert that each row belongs to (coli_moe_fp4_quantize,
                 coli_moe_fp4_product)
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token of the GLM-5.2-shaped layer (hidden 6144, 256 experts, top-8)
        dict(name="dispatch_decode", op="dispatch", T=1, H=6144, E=256, k=8, xt="bf16", drop=0.0),
        # a prefill batch at the library's largest T, some picks dropped (top-p, other ranks' experts)
        dict(name="dispatch_prefill", op="dispatch", T=8192, H=6144, E=256, k=8, xt="bf16", drop=0.2),
        # three verified positions of speculative decoding
        dict(name="combine_verify", op="combine", T=3, H=6144, E=256, k=8, ot="bf16", yt="f32", drop=0.0,
             grad=False),
        # a training step's micro-batch: output, and the gradients of rows, weights and tokens
        dict(name="combine_train", op="combine", T=4096, H=6144, E=256, k=8, ot="bf16", yt="f32", drop=0.1,
             grad=True),
        # between two blocks of a decoded token
        dict(name="norm_decode", op="norm", T=1, H=6144, xt="f32", bt="bf16", post=True, gate="channel",
             grad=False),
        # between two blocks of a prefill batch, one gate value per token
        dict(name="norm_prefill", op="norm", T=8192, H=6144, xt="bf16", bt="bf16", post=True, gate="token",
             grad=False),
        # the gradient at a block boundary of a training micro-batch
        dict(name="norm_train", op="norm", T=4096, H=6144, xt="f32", bt="bf16", post=True, gate="channel",
             grad=True),
        # activations of a small verify batch
        dict(name="quantize_verify", op="quantize", fmt="mx", rows=24, K=6144, xt="bf16"),
        # one expert's gate and up masters times eight: weights quantised at load time
        dict(name="quantize_weights", op="quantize", fmt="nv", rows=32768, K=6144, xt="f32"),
        # gate/up projection of one decoded token: 8 of 256 experts, bound by their weights
        dict(name="product_decode", op="product", fmt="mx", T=1, k=8, E=256, R=4096, K=6144, act="none"),
        # down projection of a 64-token batch over a quarter of the experts, SwiGLU before it
        dict(name="product_batch", op="product", fmt="nv", T=64, k=8, E=64, R=6144, K=2048, act="swiglu"),
        # gate/up projection of a prefill batch on one rank of eight (32 experts)
        dict(name="product_prefill", op="product", fmt="mx", T=4096, k=8, E=32, R=4096, K=6144, act="none"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "norm", "quantize", "product"])
    if op in ("dispatch", "combine"):
        E = _log(rng, 1, 512)
        c = dict(op=op, T=_log(rng, 1, 8000), H=_log(rng, 8, 6144), E=E, k=rng.randint(1, min(E, 10)),
                 drop=rng.choice([0.0, 0.0, 0.3, 0.9]))
        if op == "dispatch":
            return dict(c, xt=rng.choice(["f32", "bf16"]))
        return dict(c, T=min(c["T"], 4000), k=min(c["k"], 8), ot=rng.choice(["f32", "bf16"]), yt="f32",
                    grad=rng.random() < 0.5)
    if op == "norm":
        xt, bt = rng.choice([("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
        return dict(op=op, T=_log(rng, 1, 4000), H=_log(rng, 1, 6144), xt=xt, bt=bt, post=rng.random() < 0.8,
                    gate=rng.choice(["none", "channel", "token", "full"]), grad=rng.random() < 0.5)
    fmt = rng.choice(["mx", "nv"])
    if op == "quantize":
        return dict(op=op, fmt=fmt, rows=_log(rng, 1, 30000), K=32 * _log(rng, 1, 190),
                    xt=rng.choice(["f32", "bf16"]))
    E = rng.choice([1, 1, _log(rng, 2, 48)])
    K = 32 * _log(rng, 1, 190)
    R = _log(rng, 1, 4096) if E == 1 else 128 * _log(rng, 1, 32)
    return dict(op=op, fmt=fmt, T=_log(rng, 1, 4000), k=rng.randint(1, min(E, 8)), E=E, R=R, K=K,
                act=rng.choice(["none", "swiglu"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _acts(g, rows, cols, dt):
    """Activations: N(0, 1) with a few channels 8 times larger, as hidden states have them."""
    x = _randn(g, rows, cols)
    big = torch.randint(0, cols, (max(1, cols // 512),), generator=g, device="cuda")
    x[:, big] *= 8.0
    return x.to(DT[dt])


def _route(g, T, k, E, drop):
    """Picks of a skewed router: k different experts per token, some dropped (-1), and weights."""
    z = _randn(g, T, E) + 0.5 * _randn(g, E)
    s, idx = torch.topk(torch.sigmoid(z), k, dim=1)
    w = s / s.sum(1, keepdim=True)
    if drop:
        gone = torch.rand(T, k, generator=g, device="cuda") < drop
        idx, w = idx.masked_fill(gone, -1), w.masked_fill(gone, 0.0)
    return idx.to(torch.int32).contiguous(), w.contiguous()


def _tiled(s):
    """Scale bytes [rows, blocks] in the layout of 128 rows by 4 blocks (see the library's header)."""
    rows, nb = s.shape
    pr, pb = -(-rows // 128) * 128, -(-nb // 4) * 4
    full = torch.zeros(pr, pb, dtype=torch.uint8, device=s.device)
    full[:rows, :nb] = s
    return full.view(pr // 128, 4, 32, pb // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _stable_inverse(idx, E):
    """The picks in the order of their experts: (offsets [E+1], pick of each row, inv [T, k])."""
    flat = idx.view(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True)[1]
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rank = torch.empty_like(order)
    rank[order] = torch.arange(order.numel(), device=order.device)
    inv = torch.where(key < E, rank, -1).view_as(idx)
    return offsets, order, inv


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    op = c["op"]
    if op == "dispatch":
        P = c["T"] * c["k"]
        s["idx"], _ = _route(g, c["T"], c["k"], c["E"], c["drop"])
        s["x"] = _acts(g, c["T"], c["H"], c["xt"])
        s["offsets"] = torch.zeros(c["E"] + 1, dtype=torch.int32, device="cuda")
        s["tok"] = torch.zeros(P, dtype=torch.int32, device="cuda")
        s["slot"] = torch.zeros(P, dtype=torch.int32, device="cuda")
        s["inv"] = torch.zeros(c["T"], c["k"], dtype=torch.int32, device="cuda")
        s["xs"] = torch.zeros(P, c["H"], dtype=DT[c["xt"]], device="cuda")
    elif op == "combine":
        P = c["T"] * c["k"]
        idx, s["w"] = _route(g, c["T"], c["k"], c["E"], c["drop"])
        s["inv"] = _stable_inverse(idx, c["E"])[2].to(torch.int32).contiguous()
        s["o"] = _randn(g, P, c["H"]).to(DT[c["ot"]])
        s["y"] = torch.zeros(c["T"], c["H"], dtype=DT[c["yt"]], device="cuda")
        s["residual"] = _randn(g, c["T"], c["H"]).to(DT[c["yt"]])
        if c["grad"]:
            s["dy"] = _randn(g, c["T"], c["H"]).to(DT[c["yt"]])
            s["dxs"] = _randn(g, P, c["H"]).to(DT[c["ot"]])
            s["do"] = torch.zeros(P, c["H"], dtype=DT[c["ot"]], device="cuda")
            s["dw"] = torch.zeros(c["T"], c["k"], device="cuda")
            s["dx"] = torch.zeros(c["T"], c["H"], dtype=DT[c["ot"]], device="cuda")
    elif op == "norm":
        T, H = c["T"], c["H"]
        s["x"] = _acts(g, T, H, c["xt"])
        s["o"] = (0.3 * _randn(g, T, H)).to(DT[c["bt"]])
        s["post"] = 1.0 + 0.2 * _randn(g, H)
        s["pre"] = 1.0 + 0.2 * _randn(g, H)
        shape = {"none": None, "channel": (H,), "token": (T,), "full": (T, H)}[c["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(_randn(g, *shape))
        s["alpha"], s["eps"] = 0.5, 1e-5
        s["x_out"] = torch.zeros(T, H, dtype=DT[c["xt"]], device="cuda")
        s["n"] = torch.zeros(T, H, dtype=DT[c["bt"]], device="cuda")
        s["r_post"] = torch.zeros(T, device="cuda")
        s["r_pre"] = torch.zeros(T, device="cuda")
        if c["grad"]:  # what the forward pass of this step has kept
            x1, _, ro, rx = _norm_plain(s, c)
            s["x_out"], s["r_post"], s["r_pre"] = x1, ro, rx
            s["dx_out"] = _randn(g, T, H).to(DT[c["xt"]])
            s["dn"] = _randn(g, T, H).to(DT[c["bt"]])
            s["dx"], s["do"] = torch.zeros_like(s["x"]), torch.zeros_like(s["o"])
            s["dpost"], s["dpre"] = torch.zeros(H, device="cuda"), torch.zeros(H, device="cuda")
            s["dgate"] = None if shape is None else torch.zeros(shape, device="cuda")
    elif op == "quantize":
        s["x"] = _acts(g, c["rows"], c["K"], c["xt"])
        s["g"] = (s["x"].abs().amax().float() / (448.0 * 6.0)).reshape(1)
        s["values"] = torch.zeros_like(s["x"])
    else:
        T, k, E, R, K = c["T"], c["k"], c["E"], c["R"], c["K"]
        blk = 32 if c["fmt"] == "mx" else 16
        s["P"] = P = T * k
        idx, _ = _route(g, T, k, E, 0.0)
        off, _, _ = _stable_inverse(idx, E)
        s["offsets"], s["nmax"] = off.to(torch.int32).contiguous(), int((off[1:] - off[:-1]).max())
        s["x"] = _acts(g, P, K * (2 if c["act"] == "swiglu" else 1), "bf16")
        s["codes"] = torch.randint(0, 256, (E * R * (K // 2),), generator=g, device="cuda", dtype=torch.uint8)
        nb = K // blk
        lo, hi = (117, 123) if c["fmt"] == "mx" else (0x30, 0x58)  # 2^-10 .. 2^-5, or 0.5 .. 16
        s["scales"] = _tiled(torch.randint(lo, hi, (E * R, nb), generator=g, device="cuda", dtype=torch.uint8))
        s["g"] = torch.full((1,), 0.0125, device="cuda")
        s["alpha"] = (0.0125 * (1e-3 + 0.004 * torch.rand(E, generator=g, device="cuda"))
                      if c["fmt"] == "nv" else torch.ones(E, device="cuda"))
        s["y"] = torch.zeros(P, R, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _dispatch_plain(s, c):
    offsets, order, inv = _stable_inverse(s["idx"], c["E"])
    n = offsets[-1]
    live = torch.arange(order.numel(), device="cuda") < n
    tok = order // c["k"]
    s["tok"].copy_(torch.where(live, tok, s["tok"].long()))
    s["slot"].copy_(torch.where(live, order % c["k"], s["slot"].long()))
    torch.where(live[:, None], s["x"][tok], s["xs"], out=s["xs"])
    return {"offsets": offsets.to(torch.int32), "tok": s["tok"], "slot": s["slot"],
            "inv": inv.to(torch.int32), "xs": s["xs"]}


def _rows_of(a, inv):
    """Rows [T, k, H] of every pick in f32, zero where the pick has none."""
    got = a[inv.long().clamp(min=0)].float()
    return got * (inv >= 0)[..., None]


def _combine_plain(s, c):
    inv, w = s["inv"], s["w"]
    o = _rows_of(s["o"], inv)
    out = {"y": ((w[..., None] * o).sum(1) + s["residual"].float()).to(DT[c["yt"]])}
    if c["grad"]:
        dy = s["dy"].float()
        out["dw"] = (o * dy[:, None, :]).sum(2)
        live = inv.reshape(-1) >= 0
        rows = (w[..., None] * dy[:, None, :]).reshape(-1, c["H"]).to(DT[c["ot"]])
        s["do"][inv.reshape(-1).long()[live]] = rows[live]
        out["do"] = s["do"]
        out["dx"] = _rows_of(s["dxs"], inv).sum(1).to(DT[c["ot"]])
    return out


def _gate_of(gate, kind):
    if kind == "none":
        return 1.0
    return gate[:, None] if kind == "token" else gate


def _norm_plain(s, c):
    o = s["o"].float()
    ro = torch.rsqrt(o.square().mean(1) + s["eps"]) if c["post"] else torch.ones(c["T"], device="cuda")
    u = o * ro[:, None] * s["post"] if c["post"] else o
    x1 = (s["x"].float() + s["alpha"] * _gate_of(s["gate"], c["gate"]) * u).to(DT[c["xt"]])
    xf = x1.float()
    rx = torch.rsqrt(xf.square().mean(1) + s["eps"])
    n = (xf * rx[:, None] * s["pre"]).to(DT[c["bt"]])
    return x1, n, ro, rx


def _norm_grad_plain(s, c):
    o, x1 = s["o"].float(), s["x_out"].float()
    ro, rx = s["r_post"][:, None], s["r_pre"][:, None]
    dn = s["dn"].float()
    xh = x1 * rx
    dpre = (dn * xh).sum(0)
    v = dn * s["pre"]
    d = s["dx_out"].float() + rx * (v - xh * (v * xh).mean(1, keepdim=True))
    gate = _gate_of(s["gate"], c["gate"])
    oh = o * ro if c["post"] else o
    u = oh * s["post"] if c["post"] else oh
    du = s["alpha"] * gate * d
    out = {"dx": d.to(DT[c["xt"]]), "dpre": dpre}
    if c["gate"] != "none":
        dg = s["alpha"] * u * d
        out["dgate"] = dg.sum(0) if c["gate"] == "channel" else dg.sum(1) if c["gate"] == "token" else dg
    if c["post"]:
        out["dpost"] = (du * oh).sum(0)
        v = du * s["post"]
        du = ro * (v - oh * (v * oh).mean(1, keepdim=True))
    out["do"] = du.to(DT[c["bt"]])
    return out


def _round_e2m1(a):
    """The index of the E2M1 magnitude nearest to a >= 0 (ties to the even one)."""
    n = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return n.long()


def _pow2(e):
    """2^e in f32 for whole e in [-127, 127]: its bits, since powers by exp or pow may be an ulp off."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _quantized_values(x, fmt, g):
    """Quantise rows and return the f32 values that codes and scales stand for."""
    lut = torch.tensor(E2M1, device=x.device)
    rows, K = x.shape
    if fmt == "mx":
        b = x.float().view(rows, K // 32, 32)
        m = b.abs().amax(2)
        e = torch.where(m > 0, torch.frexp(m)[1] - 3, torch.full_like(m, -127, dtype=torch.int32)).clamp(-127, 127)
        q = b * _pow2(-e)[..., None]
        return (lut[_round_e2m1(q.abs())] * _pow2(e)[..., None] * torch.sign(q)).view(rows, K)
    b = x.float().view(rows, K // 16, 16)
    m = b.abs().amax(2)
    sc = (m / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    d = sc * g
    r = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    q = b * r[..., None]
    return (lut[_round_e2m1(q.abs())] * torch.sign(q) * d[..., None]).view(rows, K)


def _weights_plain(s, c, which):
    """f32 values [n, R, K] of the weights of the experts `which` (without the f32 scale)."""
    E, R, K = c["E"], c["R"], c["K"]
    blk = 32 if c["fmt"] == "mx" else 16
    nb = K // blk
    pr, pb = -(-E * R // 128) * 128, -(-nb // 4) * 4
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    codes = s["codes"].view(E, R, K // 2)
    sc = s["scales"].view(pr // 128, pb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(pr, pb)[:E * R, :nb]
    sc = sc.view(E, R, nb)
    if which is not None:
        codes, sc = codes[which], sc[which]
    pairs = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], 1)  # byte -> its even and odd column
    v = pairs[codes.int()].view(codes.shape[0], R, nb, blk)
    scale = _pow2(sc.int() - 127) if c["fmt"] == "mx" else sc.contiguous().view(torch.float8_e4m3fn).float()
    return v.mul_(scale[..., None]).view(codes.shape[0], R, K)


def _product_plain(s, c):
    x, E, P, R, K = s["x"], c["E"], s["P"], c["R"], c["K"]
    if c["act"] == "swiglu":
        a, b = x[:, :K].float(), x[:, K:].float()
        x = a / (1.0 + torch.exp(-a)) * b
    xq = _quantized_values(x, c["fmt"], s["g"])
    if c["fmt"] == "nv":
        xq = xq / s["g"]
    p = torch.arange(P, device="cuda")
    e = torch.searchsorted(s["offsets"][1:].contiguous(), p.to(torch.int32), right=True)
    if P < E:  # fewer rows than experts: their own weights alone
        y = torch.bmm(_weights_plain(s, c, e), xq[:, :, None])[:, :, 0]
    else:      # every expert's rows padded to the longest
        pad = torch.zeros(E, s["nmax"], K, device="cuda")
        pos = p - s["offsets"].long()[e]
        pad[e, pos] = xq
        y = torch.bmm(pad, _weights_plain(s, c, None).transpose(1, 2))[e, pos]
    return {"y": (y * s["alpha"][e][:, None]).to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _workspace(s, size):
    """The scratch space that a program keeps beside its buffers: made at the first pass."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(size(), 1), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_own(s, c):
    import int4_routed_expert_top_b200 as cm
    op = c["op"]
    if op == "dispatch":
        ws = _workspace(s, lambda: cm.coli_moe_sort_workspace_size(c["T"], c["k"], c["E"]))
        cm.coli_moe_sort(s["idx"], c["T"], c["k"], c["E"], s["offsets"], s["tok"], s["slot"], s["inv"], ws)
        cm.coli_moe_dispatch(s["x"], c["T"], c["H"], c["k"], s["inv"], s["xs"])
        return {n: s[n] for n in ("offsets", "tok", "slot", "inv", "xs")}
    if op == "combine":
        cm.coli_moe_combine(s["o"], c["T"], c["H"], c["k"], s["inv"], s["w"], s["y"], residual=s["residual"])
        out = {"y": s["y"]}
        if c["grad"]:
            cm.coli_moe_combine_backward(s["dy"], s["o"], c["T"], c["H"], c["k"], s["inv"], s["w"], s["do"],
                                         s["dw"])
            cm.coli_moe_dispatch_backward(s["dxs"], c["T"], c["H"], c["k"], s["inv"], s["dx"])
            out.update(do=s["do"], dw=s["dw"], dx=s["dx"])
        return out
    if op == "norm":
        if "desc" not in s:
            kinds = {"none": cm.COLI_GATE_NONE, "channel": cm.COLI_GATE_CHANNEL, "token": cm.COLI_GATE_TOKEN,
                     "full": cm.COLI_GATE_FULL}
            s["desc"] = cm.NormDesc(c["H"], cm.COLI_F32 if c["xt"] == "f32" else cm.COLI_BF16,
                                    cm.COLI_F32 if c["bt"] == "f32" else cm.COLI_BF16, int(c["post"]),
                                    kinds[c["gate"]], s["alpha"], s["eps"],
                                    s["post"].data_ptr() if c["post"] else None, s["pre"].data_ptr())
        if not c["grad"]:
            cm.coli_moe_block_norm(s["desc"], s["x"], s["o"], c["T"], s["x_out"], s["n"], gate=s["gate"],
                                   rstd_post=s["r_post"] if c["post"] else None, rstd_pre=s["r_pre"])
            out = {"x": s["x_out"], "n": s["n"], "r_pre": s["r_pre"]}
            if c["post"]:
                out["r_post"] = s["r_post"]
            return out
        ws = _workspace(s, lambda: cm.coli_moe_block_norm_backward_workspace_size(s["desc"], c["T"]))
        cm.coli_moe_block_norm_backward(s["desc"], s["x_out"], s["o"], c["T"], s["dx_out"], s["dn"], s["dx"],
                                        s["do"], ws, gate=s["gate"],
                                        rstd_post=s["r_post"] if c["post"] else None, rstd_pre=s["r_pre"],
                                        dpost_gain=s["dpost"] if c["post"] else None, dgate=s["dgate"],
                                        dpre_gain=s["dpre"])
        out = {"dx": s["dx"], "do": s["do"], "dpre": s["dpre"]}
        if c["post"]:
            out["dpost"] = s["dpost"]
        if c["gate"] != "none":
            out["dgate"] = s["dgate"]
        return out
    fmt = cm.COLI_MXFP4 if c["fmt"] == "mx" else cm.COLI_NVFP4
    g = s["g"] if c["fmt"] == "nv" else None
    rows, K = (c["rows"], c["K"]) if op == "quantize" else (s["P"], c["K"])
    if "xc" not in s:
        nc, ns = cm.coli_moe_fp4_bytes(fmt, rows, K)
        s["xc"] = torch.empty(nc, dtype=torch.uint8, device="cuda")
        s["xsc"] = torch.empty(ns, dtype=torch.uint8, device="cuda")
    if op == "quantize":
        cm.coli_moe_fp4_quantize(fmt, s["x"], rows, K, s["xc"], s["xsc"], gscale=g, values=s["values"])
        return {"values": s["values"]}
    act = cm.COLI_ACT_SWIGLU if c["act"] == "swiglu" else cm.COLI_ACT_NONE
    ws = _workspace(s, lambda: cm.coli_moe_fp4_product_workspace_size(fmt, rows, K, c["E"], c["R"]))
    cm.coli_moe_fp4_quantize(fmt, s["x"], rows, K, s["xc"], s["xsc"], act=act, gscale=g)
    cm.coli_moe_fp4_product(fmt, s["xc"], s["xsc"], rows, K, s["codes"], s["scales"], c["E"], c["R"], s["y"], ws,
                            offsets=s["offsets"], alpha=s["alpha"])
    return {"y": s["y"]}


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    op = c["op"]
    if op == "dispatch":
        return _dispatch_plain(state, c)
    if op == "combine":
        return _combine_plain(state, c)
    if op == "norm":
        if c["grad"]:
            return _norm_grad_plain(state, c)
        x1, n, ro, rx = _norm_plain(state, c)
        out = {"x": x1, "n": n, "r_pre": rx}
        if c["post"]:
            out["r_post"] = ro
        return out
    if op == "quantize":
        return {"values": _quantized_values(state["x"], c["fmt"], state["g"]).to(DT[c["xt"]])}
    return _product_plain(state, c)


# ---------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------
def work(case):
    c = case
    size = {"f32": 4, "bf16": 2}
    op = c["op"]
    if op == "dispatch":
        live = c["T"] * c["k"] * (1 - c["drop"])
        return {"bytes": 12 * c["T"] * c["k"] + 8 * live + (c["T"] + live) * c["H"] * size[c["xt"]], "flops": 0}
    if op == "combine":
        live = c["T"] * c["k"] * (1 - c["drop"])
        rows, toks = live * c["H"] * size[c["ot"]], c["T"] * c["H"] * size[c["yt"]]
        b, f = rows + 2 * toks + 8 * c["T"] * c["k"], 2 * live * c["H"]
        if c["grad"]:
            # dy, o (read once for y and dw), do, dxs, dx
            b += toks + 2 * rows + c["T"] * c["H"] * size[c["ot"]] + 4 * c["T"] * c["k"]
            f += 4 * live * c["H"]
        return {"bytes": b, "flops": f}
    if op == "norm":
        n = c["T"] * c["H"]
        gate = {"none": 0, "channel": 4 * c["H"], "token": 4 * c["T"], "full": 4 * n}[c["gate"]]
        if c["grad"]:
            return {"bytes": n * (3 * size[c["xt"]] + 3 * size[c["bt"]]) + 2 * gate + 16 * c["H"] + 8 * c["T"],
                    "flops": 25 * n}
        return {"bytes": n * (2 * size[c["xt"]] + 2 * size[c["bt"]]) + gate + 8 * c["H"] + 8 * c["T"],
                "flops": 10 * n}
    blk = 32 if c["fmt"] == "mx" else 16
    if op == "quantize":
        n = c["rows"] * c["K"]
        return {"bytes": n * 2 * size[c["xt"]] + n / 2 + n / blk, "flops": 4 * n}
    P, E, R, K = c["T"] * c["k"], c["E"], c["R"], c["K"]
    live = c["k"] if c["T"] == 1 else E * (1 - (1 - c["k"] / E) ** c["T"])
    per = K / 2 + K / blk
    return {"bytes": live * R * per + P * K * (4 if c["act"] == "swiglu" else 2) + P * R * 2,
            "flops": 2.0 * P * R * K}


# ---------------------------------------------------------------------------
# definitions in 64 bits
# ---------------------------------------------------------------------------
def _np(t):
    return t.detach().double().cpu().numpy() if t.is_floating_point() else t.detach().cpu().numpy()


def _exact_dispatch(s, c):
    idx = s["idx"].cpu().numpy().astype(np.int64).reshape(-1)
    xs = torch.zeros_like(s["xs"], dtype=torch.float64)
    inv = np.full(idx.size, -1, np.int64)
    picks = [np.nonzero(idx == e)[0] for e in range(c["E"])]
    order = np.concatenate(picks).astype(np.int64)
    offsets = np.concatenate([[0], np.cumsum([len(p) for p in picks])])
    inv[order] = np.arange(order.size)
    tok, slot = np.zeros(idx.size, np.int64), np.zeros(idx.size, np.int64)
    tok[:order.size], slot[:order.size] = order // c["k"], order % c["k"]
    xs[:order.size] = s["x"].double()[torch.from_numpy(order // c["k"]).cuda()]
    return {"offsets": offsets.astype(np.int32), "tok": tok.astype(np.int32), "slot": slot.astype(np.int32),
            "inv": inv.astype(np.int32).reshape(c["T"], c["k"]), "xs": xs}


def _exact_combine(s, c):
    inv, w, o = s["inv"].long(), s["w"].double(), s["o"]
    y = s["residual"].double().clone()
    out = {}
    if c["grad"]:
        dy = s["dy"].double()
        dw = torch.zeros_like(w)
        do = torch.zeros(o.shape, dtype=torch.float64, device="cuda")
        dx = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        has = torch.nonzero(inv[:, j] >= 0)[:, 0]
        rows = inv[has, j]
        y[has] += w[has, j, None] * o[rows].double()
        if c["grad"]:
            dw[has, j] = torch.einsum("th,th->t", o[rows].double(), dy[has])
            do[rows] = w[has, j, None] * dy[has]
            dx[has] += s["dxs"][rows].double()
    out["y"] = y
    if c["grad"]:
        out.update(dw=dw, do=do, dx=dx)
    return out


def _exact_norm(s, c):
    T, H = c["T"], c["H"]
    o, post, pre = s["o"].double(), s["post"].double(), s["pre"].double()
    gate = torch.ones((), dtype=torch.float64, device="cuda") if s["gate"] is None else s["gate"].double()
    if c["gate"] == "token":
        gate = gate.reshape(T, 1)
    a, eps = s["alpha"], s["eps"]
    if not c["grad"]:
        r = 1.0 / torch.sqrt(torch.einsum("th,th->t", o, o) / H + eps)
        u = torch.einsum("th,t,h->th", o, r, post) if c["post"] else o
        x1 = s["x"].double() + a * (gate * u)
        stored = x1.to(DT[c["xt"]]).double()  # the next norm reads the stored sum
        rx = 1.0 / torch.sqrt(torch.einsum("th,th->t", stored, stored) / H + eps)
        out = {"x": x1, "n": torch.einsum("th,t,h->th", stored, rx, pre), "r_pre": rx}
        if c["post"]:
            out["r_post"] = r
        return out
    x1, dn = s["x_out"].double(), s["dn"].double()
    rx = s["r_pre"].double()
    dpre = torch.einsum("th,th,t->h", dn, x1, rx)
    dot = torch.einsum("th,h,th->t", dn, pre, x1) / H
    dx = s["dx_out"].double() + torch.einsum("th,h,t->th", dn, pre, rx) - x1 * (rx ** 3 * dot)[:, None]
    out = {"dx": dx, "dpre": dpre}
    ro = s["r_post"].double()
    u = torch.einsum("th,t,h->th", o, ro, post) if c["post"] else o
    if c["gate"] != "none":
        full = a * dx * u
        out["dgate"] = {"channel": lambda: full.sum(0), "token": lambda: full.sum(1), "full": lambda: full}[c["gate"]]()
    du = a * dx * gate
    if c["post"]:
        out["dpost"] = torch.einsum("th,th,t->h", du, o, ro)
        dot = torch.einsum("th,h,th->t", du, post, o) / H
        du = torch.einsum("th,h,t->th", du, post, ro) - o * (ro ** 3 * dot)[:, None]
    out["do"] = du
    return out


def _powers(device):
    return torch.from_numpy(np.ldexp(1.0, np.arange(255) - 127)).to(device)  # the values of E8M0 bytes


def _exact_fp4(x, fmt, g):
    """Values of quantised rows (f64 in, f64 out; the f32 roundings of the definition included)."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    mids = (grid[1:] + grid[:-1]) / 2
    blk = 32 if fmt == "mx" else 16
    b = x.reshape(-1, blk)
    m = b.abs().max(1, keepdim=True)[0]
    if fmt == "mx":
        scale = _powers(x.device)[torch.where(m > 0, torch.frexp(m)[1] - 3 + 127, 0).long()]
        q = b / scale
    else:
        g32 = torch.tensor(float(g), dtype=torch.float32)
        six = float(torch.tensor(6.0, dtype=torch.float32) * g32)
        t = (m / six).float().clamp(max=448.0).to(torch.float8_e4m3fn).double()
        scale = (t * float(g32)).float().double()
        r = torch.where(scale > 0, (1.0 / scale).float().double(), torch.zeros_like(scale))
        q = (b * r).float().double()
    a = q.abs()
    lo = torch.bucketize(a, mids)                       # mids[lo-1] < a <= mids[lo]
    at = mids[lo.clamp(max=6)]
    up = (lo < 7) & (a == at) & (lo % 2 == 1)           # a tie goes to the even index
    v = grid[lo + up.long()] * torch.where(q < 0, -1.0, 1.0)
    return (v * scale).reshape(x.shape)


def _exact_product(s, c):
    E, R, K = c["E"], c["R"], c["K"]
    if 2.0 * s["P"] * R * K > 4e12:
        return None
    blk = 32 if c["fmt"] == "mx" else 16
    nb = K // blk
    off = s["offsets"].cpu().tolist()
    y = torch.zeros(s["P"], R, dtype=torch.float64, device="cuda")
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    r = torch.arange(E * R, device="cuda")
    b = torch.arange(nb, device="cuda")
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        by = s["codes"].view(E, R, K // 2)[e]
        nib = torch.empty(R, K, dtype=torch.int64, device="cuda")
        nib[:, 0::2], nib[:, 1::2] = (by & 15).long(), (by >> 4).long()
        v = grid[nib & 7] * torch.where(nib >= 8, -1.0, 1.0)
        re = r[e * R:(e + 1) * R, None]
        at = ((re // 128 * -(-nb // 4) + b // 4) * 32 + re % 32) * 16 + (re % 128) // 32 * 4 + b % 4
        sc = s["scales"][at]
        scale = _powers("cuda")[sc.long()] if c["fmt"] == "mx" else sc.view(torch.float8_e4m3fn).double()
        v = (v.view(R, nb, blk) * scale[..., None]).view(R, K)
        x = s["x"][lo:hi].double()
        if c["act"] == "swiglu":
            x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
            x = x.float().double()
        xq = _exact_fp4(x, c["fmt"], float(s["g"]))
        if c["fmt"] == "nv":
            xq = xq / float(s["g"])
        y[lo:hi] = (xq @ v.T) * s["alpha"][e].double()
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], case["op"]
    if op == "dispatch":
        return _exact_dispatch(s, c)
    if op == "combine":
        return _exact_combine(s, c)
    if op == "norm":
        return _exact_norm(s, c)
    if op == "quantize":
        return {"values": _exact_fp4(s["x"].double(), c["fmt"], float(s["g"]))}
    return _exact_product(s, c)
