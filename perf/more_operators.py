"""Cases of what surrounds the experts in a block of a mixture-of-experts
model: the root-mean-square norm with the residual's addition in front of it
(with an MXFP8 copy of its output), the router, and their gradients, with the
gradient of the routing weights through the combine.

Each case runs in a plain form (elementary torch operations in float32, in
float64 where choices are compared) or, where ``own`` is true, through the
package's entry points.

Definitions
  route     s = softmax(l) or sigmoid(l) per token; c = s + bias;
            with groups, a group's score is the sum of its group_top largest c
            and only the groups_kept best groups stay; experts = the k largest
            c in falling order (ties: lowest index); weights = scale s, divided
            by their sum over the k chosen if renorm
  route_backward   dl from the gradients of the weights (and of all scores)
  dweights  dw[t, i] = sum_n dout[t, n] y[slot_of[t, i], n]
  norm      h = x + residual rounded to the residual's type,
            y = bf16(h / sqrt(mean(h^2) + eps) w);
            MXFP8 of y: per 32 columns the scale byte S = max(floor(log2 amax)
            - 8 + 127, 0) and E4M3 codes of y 2^(127 - S), at most 448
  norm_backward    g = dy + dy2, xh = h rstd, a = g w:
            dh = dh_in + rstd (a - xh mean(a xh)),  dw = sum over rows of g xh
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
SCALE = 2.5  # factor of the routing weights
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    grouped = {"score": "sigmoid", "bias": True, "renorm": True, "groups": 8, "kept": 4, "group_top": 2}
    plain = {"score": "softmax", "bias": False, "renorm": True, "groups": 1, "kept": 1, "group_top": 1}
    return [
        # generation: a few tokens, latency
        {"name": "route_decode", "op": "route", "T": 16, "E": 256, "k": 8, "logits": "bf16", "scores": False, **grouped},
        # a training batch, experts balanced by a bias, choices limited to half of the groups
        {"name": "route_batch", "op": "route", "T": 32768, "E": 256, "k": 8, "logits": "fp32", "scores": False,
         **grouped},
        # an odd number of experts in three groups, all scores kept for a balance loss
        {"name": "route_odd", "op": "route", "T": 8191, "E": 165, "k": 6, "logits": "bf16", "scores": True, **plain,
         "groups": 3, "kept": 2},
        # gradient of the training batch
        {"name": "route_backward_batch", "op": "route_backward", "T": 32768, "E": 256, "k": 8, "logits": "bf16",
         "dscores": False, "score": "sigmoid", "renorm": True},
        # softmax weights as they are, and a balance loss on all scores
        {"name": "route_backward_scores", "op": "route_backward", "T": 4096, "E": 128, "k": 8, "logits": "fp32",
         "dscores": True, "score": "softmax", "renorm": False},
        # 4096 tokens, top 8 of 16 experts: the routed layer of the benchmark
        {"name": "dweights_layer", "op": "dweights", "T": 4096, "k": 8, "N": 7168},
        # a small batch of odd size
        {"name": "dweights_odd", "op": "dweights", "T": 509, "k": 3, "N": 1480},
        # generation: a few tokens, MXFP8 rows for the next product
        {"name": "norm_decode", "op": "norm", "M": 16, "N": 7168, "residual": "bf16", "weight": "bf16", "quant": True,
         "y": False},
        # a training batch: bf16 rows for router and dispatch, MXFP8 rows for a dense product, statistics kept
        {"name": "norm_batch", "op": "norm", "M": 32768, "N": 7168, "residual": "bf16", "weight": "bf16",
         "quant": True, "y": True},
        # short rows without a residual (heads of a projection)
        {"name": "norm_heads", "op": "norm", "M": 250001, "N": 128, "residual": "none", "weight": "fp32",
         "quant": False, "y": True},
        # gradient of the training batch: two readers of the norm's output, a residual stream behind it
        {"name": "norm_backward_batch", "op": "norm_backward", "M": 32768, "N": 7168, "residual": "bf16",
         "weight": "bf16", "dy2": True, "dh_in": True},
        # a small batch with a float32 residual stream
        {"name": "norm_backward_odd", "op": "norm_backward", "M": 1531, "N": 1480, "residual": "fp32",
         "weight": "fp32", "dy2": False, "dh_in": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, unit):
    """An odd multiple of unit from 64 to 16384."""
    return unit * (_log(rng, max(1, 64 // unit), 16384 // unit - 1) | 1)


def draw(rng):
    op = rng.choice(("route", "route", "route_backward", "dweights", "norm", "norm", "norm_backward"))
    if op in ("route", "route_backward"):
        groups = rng.choice((1, 1, 2, 4, 8, 3, 5)) if op == "route" else 1
        E = groups * _log(rng, 4, 512 // groups)
        T = _log(rng, 1, min(65535, (1 << 24) // E)) | 1
        kept = rng.randint(1, groups)
        k = min(_log(rng, 1, 16), E // groups * kept)
        case = {"op": op, "T": T, "E": E, "k": k, "logits": rng.choice(("bf16", "fp32")),
                "score": rng.choice(("softmax", "sigmoid")), "renorm": rng.random() < 0.6}
        if op == "route":
            case.update(scores=rng.random() < 0.3, bias=rng.random() < 0.6, groups=groups, kept=kept,
                        group_top=rng.choice((1, 2)))
        else:
            case["dscores"] = rng.random() < 0.5
        return case
    if op == "dweights":
        N, k = _width(rng, 8), rng.randint(1, 9)
        return {"op": op, "T": _log(rng, 1, max(1, (1 << 28) // (N * k))) | 1, "k": k, "N": N}
    quant = op == "norm" and rng.random() < 0.6
    N = _width(rng, 32 if quant else 8)
    case = {"op": op, "M": _log(rng, 1, 230_000_000 // N) | 1, "N": N, "weight": rng.choice(("bf16", "fp32"))}
    if op == "norm":
        case.update(residual=rng.choice(("none", "bf16", "bf16", "fp32")), quant=quant,
                    y=not quant or rng.random() < 0.5)
        if case["residual"] == "fp32":
            case["M"] = max(1, case["M"] * 2 // 3)
    else:
        case.update(residual=rng.choice(("bf16", "bf16", "fp32")), dy2=rng.random() < 0.5, dh_in=rng.random() < 0.7)
        if case["residual"] == "fp32":
            case["M"] = max(1, case["M"] // 2)
    return case


# -- inputs -------------------------------------------------------------------


def _randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    state = {"case": case}
    if op in ("route", "route_backward"):
        T, E, k = case["T"], case["E"], case["k"]
        popular = _randn(gen, E, scale=0.5, dtype=torch.float32)
        state["logits"] = (_randn(gen, T, E, scale=1.5, dtype=torch.float32) + popular).to(TYPES[case["logits"]])
        if op == "route":
            state["bias"] = _randn(gen, E, scale=0.1, dtype=torch.float32) if case["bias"] else None
        else:
            noise = state["logits"].float() + _randn(gen, T, E, scale=0.1, dtype=torch.float32)
            state["experts"] = noise.topk(k, dim=1).indices.to(torch.int32)
            state["dweights"] = _randn(gen, T, k, dtype=torch.float32)
            state["dscores"] = _randn(gen, T, E, scale=0.01, dtype=torch.float32) if case["dscores"] else None
    elif op == "dweights":
        T, k, N = case["T"], case["k"], case["N"]
        state["dout"], state["y"] = _randn(gen, T, N), _randn(gen, T * k, N)
        slots = torch.randperm(T * k, generator=gen, device="cuda").to(torch.int32).reshape(T, k)
        dropped = torch.rand((T, k), generator=gen, device="cuda") < 0.02  # routed to another GPU's experts
        state["slot_of"] = slots.masked_fill_(dropped, -1)
    else:
        M, N = case["M"], case["N"]
        weight = 1 + _randn(gen, N, scale=0.2, dtype=torch.float32)
        state["weight"] = weight.to(TYPES[case["weight"]])
        kind = TYPES.get(case["residual"], torch.bfloat16)
        if op == "norm":
            state["x"] = _randn(gen, M, N)
            state["residual"] = None if case["residual"] == "none" else _randn(gen, M, N, scale=2.0, dtype=kind)
        else:
            h = state["h"] = _randn(gen, M, N, scale=2.0, dtype=kind)
            state["rstd"] = torch.cat([(p.double().square().mean(1) + EPS).rsqrt().float() for p in h.split(8192)])
            state["dy"] = _randn(gen, M, N)
            state["dy2"] = _randn(gen, M, N, scale=0.1) if case["dy2"] else None
            state["dh_in"] = _randn(gen, M, N, dtype=kind) if case["dh_in"] else None
    return state


# -- plain forms ----------------------------------------------------------------


def _scores(logits, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route(state):
    case, E, k = state["case"], state["case"]["E"], state["case"]["k"]
    s = _scores(state["logits"].double(), case["score"])  # float64: choices lie next to each other
    c = s if state["bias"] is None else s + state["bias"]
    if case["groups"] > 1:
        c = c.reshape(-1, case["groups"], E // case["groups"])
        best = torch.sort(c, dim=2, descending=True).values[:, :, :case["group_top"]].sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices
        dropped = torch.ones_like(best, dtype=torch.bool).scatter_(1, order[:, :case["kept"]], False)
        c = torch.where(dropped[:, :, None], -math.inf, c).reshape(-1, E)
    experts = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, experts)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return experts.to(torch.int32), (SCALE * w).float(), s.float() if case["scores"] else None


def _route_backward(state):
    case = state["case"]
    s = _scores(state["logits"].float(), case["score"])
    experts, g = state["experts"].long(), state["dweights"]
    if case["renorm"]:
        chosen = s.gather(1, experts)
        total = chosen.sum(1, keepdim=True)
        g = (g - (g * chosen).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s) if state["dscores"] is None else state["dscores"].clone()
    ds.scatter_add_(1, experts, SCALE * g)
    dl = s * (1 - s) * ds if case["score"] == "sigmoid" else s * (ds - (s * ds).sum(1, keepdim=True))
    return dl.to(state["logits"].dtype)


def _dweights(state):
    slot = state["slot_of"].long()
    rows = torch.where((slot >= 0)[:, :, None], state["y"][slot.clamp(min=0)].float(), 0.0)
    return (rows * state["dout"].float()[:, None, :]).sum(2)


def _mxfp8(y):
    """E4M3 codes and packed scales of bf16 rows."""
    M, N = y.shape
    blocks = y.float().reshape(M, N // 32, 32)
    _, e = torch.frexp(blocks.abs().amax(2))  # amax in [2^(e-1), 2^e)
    S = torch.where((blocks == 0).all(2), 0, (e - 1 - 8 + 127).clamp(min=0))
    codes = torch.ldexp(blocks, (127 - S)[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    # byte (r, b) at unit (r / 32, b / 8), lane 32 (b % 2) + r % 32, byte (b % 8) / 2
    units = torch.zeros((32 * -(-M // 32), 8 * -(-N // 256)), dtype=torch.uint8, device=y.device)
    units[:M, :N // 32] = S.to(torch.uint8)
    units = units.reshape(-1, 32, units.shape[1] // 8, 4, 2).permute(0, 2, 4, 1, 3).contiguous()
    return codes.reshape(M, N), units.reshape(-1).view(torch.float8_e8m0fnu)


def _norm(state):
    x, residual = state["x"], state["residual"]
    h = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    v = h.float()
    rstd = 1 / torch.sqrt((v * v).mean(1) + EPS)
    y = (v * rstd[:, None] * state["weight"].float()).to(torch.bfloat16)
    out = {"rstd": rstd}
    if residual is not None:
        out["h"] = h
    if state["case"]["y"]:
        out["y"] = y
    if state["case"]["quant"]:
        out["q"], out["s"] = _mxfp8(y)
    return out


def _norm_backward(state):
    h, w = state["h"].float(), state["weight"].float()
    g = state["dy"].float()
    if state["dy2"] is not None:
        g = g + state["dy2"].float()
    rstd = state["rstd"][:, None]
    xh, a = h * rstd, g * w
    dh = rstd * (a - xh * (a * xh).mean(1, keepdim=True))
    if state["dh_in"] is not None:
        dh = dh + state["dh_in"].float()
    return {"dh": dh.to(state["h"].dtype), "dweight": (g * xh).sum(0)}


def _call(state):
    """The same through the package."""
    import mxfp8_block_scaled_04_amd as mx

    case, op = state["case"], state["case"]["op"]
    if op == "route":
        return mx.mx_router(state["logits"], case["k"], bias=state["bias"], groups=case["groups"],
                            groups_kept=case["kept"], group_top=case["group_top"], score=case["score"],
                            renorm=case["renorm"], scale=SCALE, scores=True if case["scores"] else None)
    if op == "route_backward":
        return mx.mx_router_backward(state["logits"], state["experts"], state["dweights"], dscores=state["dscores"],
                                     score=case["score"], renorm=case["renorm"], scale=SCALE)
    if op == "dweights":
        return mx.mx_combine_dweights(state["dout"], state["y"], state["slot_of"])
    if op == "norm":
        y, h, q, s, rstd = mx.mx_rms_norm(state["x"], state["weight"], residual=state["residual"], eps=EPS,
                                          y=True if case["y"] else None, q=True if case["quant"] else None, rstd=True)
        out = {"rstd": rstd}
        if state["residual"] is not None:
            out["h"] = h
        if case["y"]:
            out["y"] = y
        if case["quant"]:
            out["q"], out["s"] = q.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)
        return out
    dh, _, dweight = mx.mx_rms_norm_backward(state["dy"], state["h"], state["weight"], state["rstd"],
                                             dy2=state["dy2"], dh_in=state["dh_in"], dweight=torch.float32)
    return {"dh": dh, "dweight": dweight}


PLAIN = {"route": _route, "route_backward": _route_backward, "dweights": _dweights, "norm": _norm,
         "norm_backward": _norm_backward}


def run(state):
    if own:
        return _call(state)
    return PLAIN[state["case"]["op"]](state)


# -- what a pass cannot do without ----------------------------------------------


def work(case):
    op, wide = case["op"], {"bf16": 2, "fp32": 4, "none": 0}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (wide[case["logits"]] + 4 * case["scores"]) + 8 * T * k + 4 * E * case["bias"],
                "flops": 10 * T * E}
    if op == "route_backward":
        # without a gradient of the scores, softmax weights that are renormalised and sigmoid ones depend on the chosen logits only
        T, E, k, size = case["T"], case["E"], case["k"], wide[case["logits"]]
        some = not case["dscores"] and (case["renorm"] or case["score"] == "sigmoid")
        return {"bytes": T * (k if some else E) * size + T * E * (size + 4 * case["dscores"]) + 8 * T * k,
                "flops": 10 * T * (k if some else E)}
    if op == "dweights":
        T, k, N = case["T"], case["k"], case["N"]
        return {"bytes": 2 * T * N * (1 + k) + 8 * T * k, "flops": 2 * T * k * N}
    M, N, r = case["M"], case["N"], wide[case["residual"]]
    if op == "norm":
        return {"bytes": M * N * (2 + 2 * r + 2 * case["y"] + case["quant"] * 33 / 32) + 4 * M
                + N * wide[case["weight"]], "flops": 6 * M * N}
    return {"bytes": M * N * (2 + 2 * case["dy2"] + r * (2 + case["dh_in"])) + 4 * M + N * (wide[case["weight"]] + 4),
            "flops": 10 * M * N}


# -- in 64 bits, from the definitions ---------------------------------------------


def _exact_route(case, state):
    E, k = case["E"], case["k"]
    l = state["logits"].double().cpu().numpy()
    if case["score"] == "sigmoid":
        s = np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    else:
        s = np.exp(l - (l.max(1) + np.log(np.exp(l - l.max(1, keepdims=True)).sum(1)))[:, None])
    c = s.copy() if state["bias"] is None else s + state["bias"].double().cpu().numpy()
    if case["groups"] > 1:
        part = c.reshape(len(c), case["groups"], -1)
        best = np.partition(part, part.shape[2] - 1, axis=2)[:, :, -1]
        if case["group_top"] == 2 and part.shape[2] > 1:
            best = np.partition(part, part.shape[2] - 2, axis=2)[:, :, -2:].sum(2)
        # a group's rank: how many have more, or as much and a lower index
        g = np.arange(case["groups"])
        ahead = (best[:, None, :] > best[:, :, None]) | ((best[:, None, :] == best[:, :, None]) & (g[None, :] < g[:, None]))
        c[np.repeat(ahead.sum(2) >= case["kept"], E // case["groups"], axis=1)] = -np.inf
    experts = np.argsort(-c, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, experts, 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return experts.astype(np.int32), SCALE * w, s if case["scores"] else None


def _exact_route_backward(case, state):
    """By the chain rule, written with the derivative of each chosen weight by each logit."""
    l, g = state["logits"].double(), state["dweights"].double()
    experts = state["experts"].long()
    p = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
    chosen = p.gather(1, experts)
    ds = torch.zeros_like(l) if state["dscores"] is None else state["dscores"].double()
    if case["score"] == "softmax":
        out = p * ds - p * (p * ds).sum(1, keepdim=True)
    else:
        out = p * torch.sigmoid(-l) * ds
    if case["renorm"]:
        w = chosen / chosen.sum(1, keepdim=True)
        mixed = (g * w).sum(1, keepdim=True)
        # d log s_i / d l_i is 1 (softmax, its common part cancels) or 1 - s_i
        slope = torch.ones_like(w) if case["score"] == "softmax" else torch.sigmoid(-l).gather(1, experts)
        return out.scatter_add_(1, experts, SCALE * w * (g - mixed) * slope)
    if case["score"] == "softmax":
        out -= p * SCALE * (g * chosen).sum(1, keepdim=True)
        return out.scatter_add_(1, experts, SCALE * g * chosen)
    return out.scatter_add_(1, experts, SCALE * g * chosen * torch.sigmoid(-l).gather(1, experts))


def _exact_mxfp8(y):
    M, N = y.shape
    blocks = y.reshape(M, N // 32, 32).double()
    amax = blocks.abs().amax(2)
    S = torch.where(amax > 0, torch.floor(torch.log2(amax)) - 8, -127.0).clamp(min=-127) + 127
    codes = (blocks * torch.exp2(127 - S)[:, :, None]).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    KB = 8 * -(-N // 256)
    r = torch.arange(M, device=y.device)[:, None]
    b = torch.arange(N // 32, device=y.device)[None, :]
    at = (r // 32) * 32 * KB + (b // 8) * 256 + 4 * (32 * (b % 2) + r % 32) + (b % 8) // 2
    s = torch.full((32 * -(-M // 32) * KB,), 2.0 ** -127, dtype=torch.float64, device=y.device)
    s[at.reshape(-1)] = torch.exp2(S - 127).reshape(-1)
    return codes.double().reshape(M, N), s


def _exact_norm(case, state):
    x, residual = state["x"], state["residual"]
    h = x if residual is None else (x.double() + residual.double()).to(residual.dtype)
    ms = (h.double() ** 2).sum(1) / case["N"] + EPS
    y = h.double() / torch.sqrt(ms)[:, None] * state["weight"].double()
    out = {"rstd": 1 / torch.sqrt(ms)}
    if residual is not None:
        out["h"] = x.double() + residual.double()
    if case["y"]:
        out["y"] = y
    if case["quant"]:
        out["q"], out["s"] = _exact_mxfp8(y.to(torch.bfloat16))
    return out


def _exact_norm_backward(case, state):
    """In slices of rows."""
    N, step = case["N"], max(1, (1 << 26) // case["N"])
    dh, dw = [], torch.zeros(N, dtype=torch.float64, device="cuda")
    for at in range(0, case["M"], step):
        g, h, r = (state[n][at:at + step].double() for n in ("dy", "h", "rstd"))
        if state["dy2"] is not None:
            g = g + state["dy2"][at:at + step].double()
        xh = h * r[:, None]
        a = g * state["weight"].double()
        d = r[:, None] * a - xh * (r * (a * xh).sum(1) / N)[:, None]
        dh.append(d if state["dh_in"] is None else d + state["dh_in"][at:at + step].double())
        dw += (g * xh).sum(0)
    return {"dh": torch.cat(dh), "dweight": dw}


def exact(case, seed):
    state, op = prepare(case, seed), case["op"]
    if op == "route":
        return _exact_route(case, state)
    if op == "route_backward":
        return _exact_route_backward(case, state)
    if op == "norm":
        return _exact_norm(case, state)
    if op == "norm_backward":
        return _exact_norm_backward(case, state)
    rows, k = [], case["k"]
    step = max(1, (1 << 26) // (k * case["N"]))
    for at in range(0, case["T"], step):
        slot = state["slot_of"][at:at + step].long()
        y = state["y"][slot.clamp(min=0)].double()
        rows.append((y * state["dout"][at:at + step, None].double()).sum(2).masked_fill_(slot < 0, 0.0))
    return torch.cat(rows)
