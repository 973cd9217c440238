"""Cases of the operators around the MoE expert layer: what is measured, on which inputs.

  norm_quantize        RMSNorm before a block, its result rounded to BF16 and quantized (MXFP8,
                       MXFP4, NVFP4 per token), or kept in BF16 only
  norm_backward        gradients of that norm, with the residual branch's gradient added
  gate_residual        RMSNorm after a block, times its gate and scale, added to the residual
  gate_residual_backward
  route                top-k routing: combine weights, per-expert counts, expert-major slots, and
                       the balance loss of the counts and the mean probabilities
  route_backward       gradient of the weights and of the balance loss to the router's logits
  combine_backward     gradients of the weighted top-k combine to the expert outputs and weights

`run` computes the plain form (elementary torch operations) or, where `own` is true, calls the
package. Sizes: hidden 7168 with 256 experts and 16384 tokens, hidden 2048 with 128 experts and
4096 tokens, top-8, as in the package's MoE workloads.
"""

import math

import torch

own = False

FLT_MAX = 3.40282346638528859812e38
EPS = 1e-6
COEF = 0.015625          # balance-loss coefficient
RES, BRANCH = 0.5, 0.75  # scales of the residual stream and of the block's branch (all three exact in binary32)


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch's hidden states normed and quantized for the MXFP8 projections
        dict(name="norm mxfp8 decode", op="norm_quantize", rows=8, cols=7168, fmt="mxfp8", keep_n=True, x32=False),
        # tokens entering the NVFP4 experts; the BF16 copy feeds the router
        dict(name="norm nvfp4 4096x2048", op="norm_quantize", rows=4096, cols=2048, fmt="nvfp4", keep_n=True,
             x32=False),
        # a training batch ahead of an MXFP8 layer
        dict(name="norm mxfp8 16384x7168", op="norm_quantize", rows=16384, cols=7168, fmt="mxfp8", keep_n=True,
             x32=False),
        # the same batch on the way back: gradients from the experts and from the router, residual added
        dict(name="norm backward 16381x7168", op="norm_backward", rows=16381, cols=7168, x32=False, dn16=False,
             two=True, res=True),
        # a few sequences' tokens after a block, one gate per token
        dict(name="gate residual decode", op="gate_residual", rows=5, cols=2048, mode="token", x32=False, y16=False),
        # a training batch after the experts' FP32 combine, one learned scale per channel
        dict(name="gate residual 16384x7168", op="gate_residual", rows=16384, cols=7168, mode="channel", x32=False,
             y16=False),
        dict(name="gate residual bwd 8191x7168", op="gate_residual_backward", rows=8191, cols=7168, mode="channel",
             x32=False, y16=False),
        # routing of a decode batch
        dict(name="route decode", op="route", tokens=8, experts=256, topk=8, pad=1, masked=False, dead=0, loss=False),
        # routing of a padded training batch with the balance loss, slots padded for the weight gradients
        dict(name="route 16384x256", op="route", tokens=16384, experts=256, topk=8, pad=32, masked=True, dead=0,
             loss=True),
        dict(name="route backward 16384x256", op="route_backward", tokens=16384, experts=256, topk=8, masked=True,
             dead=0, loss=True),
        # gradients through the combine: a small ragged batch, and a training batch
        dict(name="combine backward 1021x2048", op="combine_backward", tokens=1021, experts=128, topk=8, pad=8,
             cols=2048, dy16=False),
        dict(name="combine backward 8192x7168", op="combine_backward", tokens=8192, experts=256, topk=8, pad=32,
             cols=7168, dy16=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_quantize", "norm_quantize", "norm_backward", "gate_residual", "gate_residual_backward",
                     "route", "route", "route_backward", "combine_backward"])
    if op in ("route", "route_backward"):
        topk = rng.randint(1, 12)
        case = dict(op=op, tokens=_log(rng, 1, 16384), experts=_log(rng, 16, 512), topk=topk,
                    masked=rng.random() < 0.5, dead=rng.choice([0, 0, 3]), loss=rng.random() < 0.7)
        if op == "route":
            case["pad"] = rng.choice([1, 8, 32])
        return case
    cols = 32 * _log(rng, 8, 256)
    if op == "combine_backward":
        topk = rng.randint(1, 10)
        most = 8192 * 7168 * 8 // (cols * topk)
        return dict(op=op, tokens=_log(rng, 16, min(16384, most)), experts=_log(rng, 16, 256), topk=topk,
                    pad=rng.choice([1, 8, 32]), cols=cols, dy16=rng.random() < 0.3)
    case = dict(op=op, rows=_log(rng, 1, min(16384, 16384 * 7168 // cols)), cols=cols, x32=rng.random() < 0.3)
    if op == "norm_quantize":
        case.update(fmt=rng.choice(["mxfp8", "nvfp4", "mxfp4", "bf16"]))
        case.update(keep_n=case["fmt"] == "bf16" or rng.random() < 0.6)
    elif op == "norm_backward":
        case.update(dn16=rng.random() < 0.4, two=rng.random() < 0.5, res=rng.random() < 0.7)
    else:
        case.update(mode=rng.choice(["none", "token", "channel", "full"]), y16=rng.random() < 0.4)
    return case


# --------------------------------------------------------------------------- inputs

def _gen(seed, n):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + n) & 0x7FFFFFFF)
    return g


def _randn(seed, n, *shape):
    return torch.randn(shape, generator=_gen(seed, n), device="cuda", dtype=torch.float32)


def _f32(*shape):
    return torch.empty(shape, device="cuda", dtype=torch.float32)


def _hidden(seed, n, rows, cols, dtype):
    """Hidden states: tokens of different magnitude, a few channels that run large."""
    x = _randn(seed, n, rows, cols) * torch.exp(_randn(seed, n + 1, rows, 1))
    return (x * (1.0 + 9.0 * (_randn(seed, n + 2, cols) > 2.3))).to(dtype)


def _rstd(x):
    return torch.rsqrt(x.double().square().mean(1) + EPS).float()


def _route_inputs(case, seed):
    T, G = case["tokens"], case["experts"]
    logits = 1.5 * _randn(seed, 0, T, G) + 0.5 * _randn(seed, 1, G)        # experts differ in popularity
    logits[1::7] = torch.round(logits[1::7] * 4) / 4                       # rows with ties
    if case["dead"]:
        logits[:, torch.randperm(G, generator=_gen(seed, 2), device="cuda")[:case["dead"]]] = -math.inf
    valid = None
    if case["masked"]:                                                     # the padding tokens of a batch
        valid = torch.rand(T, generator=_gen(seed, 3), device="cuda") < 0.9
    return logits, valid


def prepare(case, seed):
    st, op = dict(case), case["op"]
    xt = torch.float32 if case.get("x32") else torch.bfloat16
    if op in ("norm_quantize", "norm_backward", "gate_residual", "gate_residual_backward"):
        T, H = case["rows"], case["cols"]
        st["weight"] = 1.0 + 0.2 * _randn(seed, 10, H)
    if op == "norm_quantize":
        st["x"] = _hidden(seed, 0, T, H, xt)
    elif op == "norm_backward":
        st["x"] = _hidden(seed, 0, T, H, xt)
        st["rstd"] = _rstd(st["x"])
        gt = torch.bfloat16 if case["dn16"] else torch.float32
        st["dn"] = (1e-3 * _randn(seed, 3, T, H)).to(gt)
        st["dn2"] = (1e-3 * _randn(seed, 4, T, H)).to(gt) if case["two"] else None
        st["d_res"] = (1e-3 * _randn(seed, 5, T, H)).to(xt) if case["res"] else None
    elif op in ("gate_residual", "gate_residual_backward"):
        st["y"] = _hidden(seed, 0, T, H, torch.bfloat16 if case["y16"] else torch.float32)
        shape = {"none": None, "token": (T,), "channel": (H,), "full": (T, H)}[case["mode"]]
        st["gate"] = None if shape is None else torch.sigmoid(_randn(seed, 3, *shape))
        if op == "gate_residual":
            st["x"] = _hidden(seed, 4, T, H, xt)
        else:
            st["rstd"] = _rstd(st["y"])
            st["d_out"] = (1e-3 * _randn(seed, 4, T, H)).to(xt)
    elif op in ("route", "route_backward"):
        st["logits"], st["valid"] = _route_inputs(case, seed)
        if op == "route_backward":
            idx, w, counts = _choose(st["logits"], st["valid"], case["topk"])[:3]
            st.update(topk_idx=idx, weights=w, counts=counts, d_weights=1e-2 * _randn(seed, 4, *w.shape),
                      d_loss=1.0 + 0.1 * _randn(seed, 5, 1) if case["loss"] else None)
    else:
        T, G, k, H = case["tokens"], case["experts"], case["topk"], case["cols"]
        plan = _plan(_route_inputs(dict(case, dead=0, masked=False), seed)[0], None, k, case["pad"])
        st.update({n: plan[n] for n in ("slot_of", "weights", "row_index")})
        st["o"] = _randn(seed, 6, plan["row_index"].numel(), H)
        st["dy"] = (1e-3 * _randn(seed, 7, T, H)).to(torch.bfloat16 if case["dy16"] else torch.float32)
    return st


# --------------------------------------------------------------------------- plain form

def _round_bf16(v):
    """A float64 tensor rounded once, to nearest even, to BF16."""
    m, e = torch.frexp(v)
    return torch.ldexp(torch.round(m * 256.0), e - 8).to(torch.bfloat16)


def _e2m1(v):
    """v rounded to the nearest E2M1 value, ties to even, saturating at 6."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.clamp(torch.round(a / step) * step, max=6.0), v)


def _div32(a, b):
    """a / b of binary32 tensors, correctly rounded to binary32."""
    return (a.double() / b.double()).float()


def _mx_exponent(amax, top, frac):
    """Code of the smallest 2^e with amax <= frac * 2^top * 2^e (0 for a block of zeros)."""
    m, e = torch.frexp(amax)
    code = torch.clamp(e - 1 - top + (2.0 * m > frac) + 127, 0, 254)
    return torch.where(amax == 0, 0, code)


def _quantize(n, fmt):
    """The quantized copy of BF16 n: for MXFP8 its elements and scales, for the 4-bit formats the
    BF16 values that elements and scales stand for."""
    T, H = n.shape
    v = n.float()
    if fmt == "nvfp4":
        b = v.view(T, H // 16, 16)
        a = b.abs().amax(2)
        A = a.amax(1, keepdim=True)
        s_enc = torch.where(A == 0, 1.0, torch.clamp(_div32(torch.full_like(A, 2688.0), A), max=FLT_MAX))
        t = _div32(torch.ones_like(A), s_enc)
        S = torch.clamp(_div32(a, torch.full_like(a, 6.0)) * s_enc, max=448.0).to(torch.float8_e4m3fn).float()
        r = torch.where(S == 0, 0.0, torch.clamp(_div32(s_enc.expand_as(S), S), max=FLT_MAX))
        q = _e2m1(b * r.unsqueeze(2))
        return {"values": ((q * S.unsqueeze(2)) * t.unsqueeze(2)).view(T, H).to(torch.bfloat16)}
    b = v.view(T, H // 32, 32)
    code = _mx_exponent(b.abs().amax(2), *((8, 1.75) if fmt == "mxfp8" else (2, 1.5)))
    scaled = torch.ldexp(b, (127 - code).unsqueeze(2))
    if fmt == "mxfp8":
        return {"q": scaled.to(torch.float8_e4m3fn).view(T, H), "s": code.to(torch.uint8).view(torch.float8_e8m0fnu)}
    return {"values": torch.ldexp(_e2m1(scaled), (code - 127).unsqueeze(2)).view(T, H).to(torch.bfloat16)}


def _plain_norm_quantize(st):
    x = st["x"].double()
    r = 1.0 / torch.sqrt(x.square().mean(1, keepdim=True) + EPS)
    n = _round_bf16(x * r * st["weight"].double())
    out = {"rstd": r[:, 0].float()}
    if st["keep_n"]:
        out["n"] = n
    if st["fmt"] != "bf16":
        out.update(_quantize(n, st["fmt"]))
    return out


def _plain_norm_backward(st):
    x, r, dn = st["x"].float(), st["rstd"].unsqueeze(1), st["dn"].float()
    if st["dn2"] is not None:
        dn = dn + st["dn2"].float()
    xh = x * r
    g = dn * st["weight"]
    dx = r * (g - xh * (g * xh).mean(1, keepdim=True))
    if st["d_res"] is not None:
        dx = dx + RES * st["d_res"].float()
    return {"dx": dx.to(st["x"].dtype), "dw": (dn * xh).sum(0)}


def _gate(st):
    """The gate, laid out to multiply (rows, cols)."""
    g = st["gate"]
    return 1.0 if g is None else g.unsqueeze(1) if st["mode"] == "token" else g


def _plain_gate_residual(st):
    y = st["y"].float()
    r = 1.0 / torch.sqrt(y.square().mean(1, keepdim=True) + EPS)
    branch = _gate(st) * (y * r * st["weight"])
    return {"out": (RES * st["x"].float() + BRANCH * branch).to(st["x"].dtype), "rstd": r[:, 0]}


def _plain_gate_residual_backward(st):
    y, r, d = st["y"].float(), st["rstd"].unsqueeze(1), BRANCH * st["d_out"].float()
    yh = y * r
    dn = d * _gate(st)
    g = dn * st["weight"]
    out = {"dy": (r * (g - yh * (g * yh).mean(1, keepdim=True))).to(st["y"].dtype), "dw": (dn * yh).sum(0)}
    if st["gate"] is not None:
        dg = d * (yh * st["weight"])
        out["dgate"] = dg if st["mode"] == "full" else dg.sum(1 if st["mode"] == "token" else 0)
    return out


def _choose(logits, valid, topk):
    """Chosen experts (-1: none), their weights, per-expert counts followed by the number of routed
    tokens, and the routed tokens. The largest logits first, ties to the lower expert; an expert at
    minus infinity is never chosen; weights are the softmax over the chosen ones."""
    T, G = logits.shape
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :topk], idx[:, :topk]
    live = top > -math.inf
    if valid is not None:
        live = live & valid.unsqueeze(1)
    routed = live[:, 0]
    e = torch.where(live, torch.exp(top - torch.where(routed, top[:, 0], 0.0).unsqueeze(1)), 0.0)
    w = e / torch.where(routed, e.sum(1), 1.0).unsqueeze(1)
    counts = torch.zeros(G + 2, dtype=torch.int32, device=logits.device)
    idx = torch.where(live, idx, -1)
    counts.index_add_(0, torch.where(live, idx, G + 1).reshape(-1), torch.ones_like(idx, dtype=torch.int32).reshape(-1))
    counts[G] = routed.sum()
    return idx.to(torch.int32), w, counts[:G + 1], routed


def slots(tokens, experts, topk, pad):
    """Slots that hold any routing of so many tokens, every expert's range a multiple of pad."""
    n = tokens * topk
    return (n + min(experts, n) * (pad - 1)) // pad * pad


def _plan(logits, valid, topk, pad):
    """Expert-major slots, tokens ascending inside an expert; every expert's range is padded to a
    multiple of pad, and what is left of the buffer is dealt out in such units, low experts first."""
    T, G = logits.shape
    idx, w, counts, routed = _choose(logits, valid, topk)
    total = slots(T, G, topk, pad)
    padded = (counts[:G].long() + pad - 1) // pad
    spare = total // pad - padded.sum()
    padded = (padded + spare // G + (torch.arange(G, device=idx.device) < spare % G)) * pad
    offsets = torch.cat([torch.zeros_like(padded[:1]), padded.cumsum(0)])
    flat = idx.reshape(-1).long()
    chosen, order = torch.sort(torch.where(flat < 0, G, flat), stable=True)
    first = torch.cat([torch.zeros_like(padded[:1]), counts[:G].long().cumsum(0)])
    at = torch.arange(T * topk, device=idx.device)
    slot = torch.where(chosen < G, torch.cat([offsets[:G], offsets[:1]])[chosen] + at - first[chosen], -1)
    slot_of = torch.empty_like(slot)
    slot_of[order] = slot
    row_index = torch.full((total + 1,), -1, dtype=torch.int32, device=idx.device)
    row_index[torch.where(slot < 0, total, slot)] = (order // topk).to(torch.int32)
    return {"topk_idx": idx, "weights": w, "counts": counts, "offsets": offsets, "row_index": row_index[:total],
            "slot_of": slot_of.view(T, topk)}


def _softmax(logits, routed):
    m = torch.where(routed, logits.amax(1), 0.0).unsqueeze(1)
    e = torch.where(routed.unsqueeze(1), torch.exp(logits - m), 0.0)
    return e / torch.where(routed, e.sum(1), 1.0).unsqueeze(1)


def _plain_route(st):
    out = _plan(st["logits"], st["valid"], st["topk"], st["pad"])
    if st["loss"]:
        G, counts = st["experts"], out["counts"]
        routed = out["topk_idx"][:, 0] >= 0
        mean_p = _softmax(st["logits"], routed).sum(0) / torch.clamp(counts[G], min=1)
        share = counts[:G].float() / torch.clamp(counts[:G].sum(), min=1)
        out["loss"] = (COEF * G) * (share * mean_p).sum().reshape(1)
    return out


def _plain_route_backward(st):
    idx, w, dw, G = st["topk_idx"].long(), st["weights"], st["d_weights"], st["experts"]
    live = idx >= 0
    d = torch.where(live, w * (dw - (w * dw).sum(1, keepdim=True)), 0.0)
    out = torch.zeros((idx.shape[0], G + 1), dtype=torch.float32, device=idx.device)
    out = out.scatter(1, torch.where(live, idx, G), d)[:, :G].contiguous()
    if st["loss"]:
        counts = st["counts"]
        p = _softmax(st["logits"], live[:, 0])
        c = st["d_loss"] * ((COEF * G) * counts[:G].float() / torch.clamp(counts[:G].sum(), min=1)
                            / torch.clamp(counts[G], min=1))
        out += p * (c - (p * c).sum(1, keepdim=True))
    return {"d_logits": out}


def _plain_combine_backward(st):
    slot, w, dy, o = st["slot_of"], st["weights"], st["dy"].float(), st["o"]
    T, k = slot.shape
    row = st["row_index"].long()
    of_slot = torch.zeros(row.numel(), dtype=torch.float32, device=row.device)
    of_slot[slot.reshape(-1)] = w.reshape(-1)
    d_o = torch.where(row.unsqueeze(1) < 0, 0.0, dy[torch.clamp(row, min=0)] * of_slot.unsqueeze(1)).to(torch.bfloat16)
    dots = (dy[torch.clamp(row, min=0)] * o).sum(1)
    return {"d_o": d_o, "d_weights": dots[slot]}


_plain = {"norm_quantize": _plain_norm_quantize, "norm_backward": _plain_norm_backward,
          "gate_residual": _plain_gate_residual, "gate_residual_backward": _plain_gate_residual_backward,
          "route": _plain_route, "route_backward": _plain_route_backward, "combine_backward": _plain_combine_backward}


# --------------------------------------------------------------------------- the package's calls

def _own_norm_quantize(st):
    from microscaling_precision_quantization_amd import binding as B
    fmt = {"mxfp8": B.MXFP8, "mxfp4": B.MXFP4, "nvfp4": B.NVFP4, "bf16": B.BF16}[st["fmt"]]
    n, q, s, t, rstd = B.rmsnorm_quantize(st["x"], st["weight"], eps=EPS, fmt=fmt, keep_n=st["keep_n"])
    out = {"rstd": rstd}
    if n is not None:
        out["n"] = n
    if st["fmt"] == "mxfp8":
        out.update(q=q.view(torch.float8_e4m3fn), s=s.view(torch.float8_e8m0fnu))
    elif q is not None:
        out["values"] = B.dequantize(fmt, q, s, t)
    return out


def _own_norm_backward(st):
    from microscaling_precision_quantization_amd import binding as B
    dx, dw = B.rmsnorm_backward(st["dn"], st["x"], st["rstd"], st["weight"], dn2=st["dn2"], d_res=st["d_res"],
                                res_scale=RES)
    return {"dx": dx, "dw": dw}


def _own_gate_residual(st):
    from microscaling_precision_quantization_amd import binding as B
    out, rstd = B.rmsnorm_gate_residual(st["x"], st["y"], st["weight"], st["gate"], gate_mode=st["mode"], eps=EPS,
                                        branch_scale=BRANCH, res_scale=RES)
    return {"out": out, "rstd": rstd}


def _own_gate_residual_backward(st):
    from microscaling_precision_quantization_amd import binding as B
    dy, dw, dgate = B.rmsnorm_gate_residual_backward(st["d_out"], st["y"], st["rstd"], st["weight"], st["gate"],
                                                     gate_mode=st["mode"], branch_scale=BRANCH)
    out = {"dy": dy, "dw": dw}
    if dgate is not None:
        out["dgate"] = dgate
    return out


def _own_route(st):
    from microscaling_precision_quantization_amd import binding as B
    plan = B.moe_route(st["logits"], st["topk"], pad=st["pad"], valid=st["valid"],
                       balance_coef=COEF if st["loss"] else None)
    out = {n: getattr(plan, n) for n in ("topk_idx", "weights", "counts", "offsets", "row_index", "slot_of")}
    if st["loss"]:
        out["loss"] = plan.loss
    return out


def _own_route_backward(st):
    from microscaling_precision_quantization_amd import binding as B
    return {"d_logits": B.moe_route_backward(st["logits"], st["topk_idx"], st["weights"], st["counts"],
                                             d_weights=st["d_weights"], d_loss=st["d_loss"], balance_coef=COEF)}


def _own_combine_backward(st):
    from microscaling_precision_quantization_amd import binding as B
    d_o, d_w = B.moe_combine_backward(st["dy"], st["o"], st["slot_of"], st["weights"], st["row_index"])
    return {"d_o": d_o, "d_weights": d_w}


_own = {"norm_quantize": _own_norm_quantize, "norm_backward": _own_norm_backward,
        "gate_residual": _own_gate_residual, "gate_residual_backward": _own_gate_residual_backward,
        "route": _own_route, "route_backward": _own_route_backward, "combine_backward": _own_combine_backward}


def run(st):
    return (_own if own else _plain)[st["op"]](st)


# --------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    size = lambda wide: 4 if wide else 2
    if op in ("route", "route_backward"):
        T, G, k = case["tokens"], case["experts"], case["topk"]
        if op == "route":
            return {"bytes": 4 * T * G + T * bool(case["masked"]) + 16 * T * k + 4 * slots(T, G, k, case["pad"]) + 12 * G,
                    "flops": T * G * (k + (8 if case["loss"] else 0))}
        return {"bytes": (4 + 4 * bool(case["loss"])) * T * G + 12 * T * k + 4 * G, "flops": 8 * T * G}
    if op == "combine_backward":
        T, k, H = case["tokens"], case["topk"], case["cols"]
        return {"bytes": size(not case["dy16"]) * T * H + 4 * T * k * H
                + 2 * slots(T, case["experts"], k, case["pad"]) * H + 16 * T * k, "flops": 3 * T * k * H}
    T, H = case["rows"], case["cols"]
    x = size(case["x32"])
    if op == "norm_quantize":
        q = {"mxfp8": 1 + 1 / 32, "mxfp4": 0.5 + 1 / 32, "nvfp4": 0.5625, "bf16": 0}[case["fmt"]]
        return {"bytes": T * H * (x + q + 2 * case["keep_n"]) + 4 * H + 4 * T, "flops": 8 * T * H}
    if op == "norm_backward":
        g = size(not case["dn16"]) * (2 if case["two"] else 1)
        return {"bytes": T * H * (g + x + x + x * case["res"]) + 8 * H + 4 * T, "flops": 11 * T * H}
    y = size(not case["y16"])
    gate = {"none": 0, "token": 4 * T, "channel": 4 * H, "full": 4 * T * H}[case["mode"]]
    if op == "gate_residual":
        return {"bytes": T * H * (2 * x + y) + gate + 4 * H + 4 * T, "flops": 8 * T * H}
    return {"bytes": T * H * (x + 2 * y) + 2 * gate + 8 * H + 4 * T, "flops": 14 * T * H}


# --------------------------------------------------------------------------- 64 bits

def _nearest(v, mantissa, low, top):
    """float64 v rounded to nearest even on a float grid: `mantissa` bits below the leading one,
    smallest exponent `low`, largest magnitude `top`."""
    a = v.abs()
    e = torch.clamp(torch.floor(torch.log2(torch.where(a > 0, a, 1.0))), min=low)
    e = torch.where(torch.exp2(e) > a, torch.clamp(e - 1, min=low), e)     # log2 next to a power of two
    unit = torch.exp2(e - mantissa)
    return torch.copysign(torch.clamp(torch.round(a / unit) * unit, max=top), v)


def _fl32(v):
    return v.float().double()


def _exact_norm_quantize(st):
    x = st["x"].double()
    H = x.shape[1]
    ms = (x * x).sum(1, keepdim=True) / H + EPS
    n = x / torch.sqrt(ms) * st["weight"].double()
    out = {"rstd": (1.0 / torch.sqrt(ms))[:, 0]}
    if st["keep_n"]:
        out["n"] = n
    if st["fmt"] == "bf16":
        return out
    v = _nearest(n, 7, -126, math.inf)
    if st["fmt"] == "nvfp4":                                # the scale steps are binary32 by definition
        b = v.view(x.shape[0], -1, 16)
        a = b.abs().amax(2, keepdim=True)
        A = a.amax(1, keepdim=True)
        enc = torch.where(A == 0, 1.0, torch.clamp(_fl32(2688.0 / A), max=FLT_MAX))
        S = _nearest(torch.clamp(_fl32(_fl32(a / 6.0) * enc), max=448.0), 3, -6, 448.0)
        r = torch.where(S == 0, 0.0, torch.clamp(_fl32(enc / S), max=FLT_MAX))
        out["values"] = (_nearest(_fl32(b * r), 1, 0, 6.0) * S * _fl32(1.0 / enc)).view_as(x)
        return out
    b = v.view(x.shape[0], -1, 32)
    a = b.abs().amax(2, keepdim=True)
    top = 448.0 if st["fmt"] == "mxfp8" else 6.0
    e = torch.clamp(torch.ceil(torch.log2(torch.where(a > 0, a / top, 2.0 ** -127))), -127, 127)
    e = torch.where((a <= top * torch.exp2(e - 1)) & (e > -127), e - 1, e)  # log2 next to a power of two
    e = torch.where(a > top * torch.exp2(e), e + 1, e)
    if st["fmt"] == "mxfp8":
        out["q"] = _nearest(b / torch.exp2(e), 3, -6, 448.0).view_as(x)
        out["s"] = torch.exp2(e)[:, :, 0]
    else:
        out["values"] = (_nearest(b / torch.exp2(e), 1, 0, 6.0) * torch.exp2(e)).view_as(x)
    return out


def _exact_norm_backward(st):
    x, r, w = st["x"].double(), st["rstd"].double()[:, None], st["weight"].double()
    dn = st["dn"].double() + (0.0 if st["dn2"] is None else st["dn2"].double())
    s = (dn * w * x).sum(1, keepdim=True) / x.shape[1]
    dx = r * dn * w - r ** 3 * s * x
    if st["d_res"] is not None:
        dx += RES * st["d_res"].double()
    return {"dx": dx, "dw": torch.mv((dn * x).t(), r[:, 0])}


def _gate64(st, T, H):
    if st["gate"] is None:
        return torch.ones((1, 1), dtype=torch.float64, device="cuda").expand(T, H)
    g = st["gate"].double()
    return (g[:, None] if st["mode"] == "token" else g).expand(T, H)


def _exact_gate_residual(st):
    y = st["y"].double()
    rstd = ((y * y).sum(1) / y.shape[1] + EPS) ** -0.5
    norm = y * rstd[:, None] * st["weight"].double()
    return {"out": st["x"].double() * RES + norm * _gate64(st, *y.shape) * BRANCH, "rstd": rstd}


def _exact_gate_residual_backward(st):
    y, r, w = st["y"].double(), st["rstd"].double()[:, None], st["weight"].double()
    d = st["d_out"].double() * BRANCH
    g = _gate64(st, *y.shape)
    s = (d * g * w * y).sum(1, keepdim=True) / y.shape[1]
    out = {"dy": r * d * g * w - r ** 3 * s * y, "dw": (d * g * y * r).sum(0)}
    if st["gate"] is not None:
        dg = d * y * r * w
        out["dgate"] = {"token": lambda: dg.sum(1), "channel": lambda: dg.sum(0), "full": lambda: dg}[st["mode"]]()
    return out


def _probabilities(logits, live):
    return torch.nan_to_num(torch.softmax(logits.double(), 1), nan=0.0) * live.double()[:, None]


def _exact_route(st):
    z = st["logits"].double()
    T, G = z.shape
    k = st["topk"]
    ok = torch.isfinite(z).any(1)
    if st["valid"] is not None:
        ok &= st["valid"]
    # rank of every expert in its row: how many are larger, or equal with a lower index
    rank = torch.cat([((z[a:a + 256, None, :] > z[a:a + 256, :, None])
                       | ((z[a:a + 256, None, :] == z[a:a + 256, :, None])
                          & (torch.arange(G, device=z.device)[None, None, :]
                             < torch.arange(G, device=z.device)[None, :, None]))).sum(2) for a in range(0, T, 256)])
    chosen = (rank < k) & torch.isfinite(z) & ok[:, None]
    p = torch.softmax(torch.where(chosen, z, -math.inf), 1)
    w = torch.zeros((T, G + 1), dtype=torch.float64, device=z.device)
    w = w.scatter(1, torch.where(chosen, rank, G), torch.where(chosen, torch.nan_to_num(p), 0.0))
    out = {"topk_idx": None, "weights": w[:, :k], "counts": None, "offsets": None, "row_index": None, "slot_of": None}
    if st["loss"]:
        f = chosen.double().sum(0)
        live = float(ok.sum())
        mean = _probabilities(z, ok).sum(0)
        out["loss"] = (COEF * G / max(live, 1.0) / torch.clamp(f.sum(), min=1.0) * torch.dot(f, mean)).reshape(1)
    return out


def _exact_route_backward(st):
    z, idx, w, dw = st["logits"].double(), st["topk_idx"].long(), st["weights"].double(), st["d_weights"].double()
    T, G = z.shape
    on = (idx >= 0).double()
    d = torch.zeros((T, G), dtype=torch.float64, device=z.device)
    d.scatter_add_(1, idx.clamp(min=0), on * w * (dw - (on * w * dw).sum(1, keepdim=True)))
    if st["loss"]:
        f = st["counts"][:G].double()
        c = st["d_loss"].double() * COEF * G * f / (f.sum().clamp(min=1.0) * st["counts"][G].double().clamp(min=1.0))
        p = _probabilities(z, on[:, 0])
        d += p * c - p * torch.mv(p, c)[:, None]
    return {"d_logits": d}


def _exact_combine_backward(st):
    slot, w, o = st["slot_of"], st["weights"].double(), st["o"]
    d_o = torch.zeros(o.shape, dtype=torch.float64, device="cuda")
    d_w = torch.empty(w.shape, dtype=torch.float64, device="cuda")
    dy = st["dy"].double()
    for j in range(w.shape[1]):
        d_o[slot[:, j]] = w[:, j, None] * dy
        d_w[:, j] = (dy * o[slot[:, j]].double()).sum(1)
    return {"d_o": d_o, "d_weights": d_w}


def exact(case, seed):
    return {"norm_quantize": _exact_norm_quantize, "norm_backward": _exact_norm_backward,
            "gate_residual": _exact_gate_residual, "gate_residual_backward": _exact_gate_residual_backward,
            "route": _exact_route, "route_backward": _exact_route_backward,
            "combine_backward": _exact_combine_backward}[case["op"]](prepare(case, seed))
