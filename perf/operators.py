"""Cases of the training step of unquantized (bf16) experts: the products
grouped by expert with ragged group sizes (forward, input gradient, weight
gradient) and the AdamW step over many tensors at once, with its states in 32
or in 8 bits, optionally after clipping by the gradients' global norm.

Each case runs in a plain form (elementary torch operations in float32) or,
where ``own`` is true, through the package's entry points.

Definitions
  forward   out[r, :] = x[r, :] w[e]^T     for the rows r of expert e
  dgrad     dx[r, :]  = dy[r, :] w[e]
  wgrad     dw[e]     = (dw[e] +) sum over the rows r of e of dy[r, :]^T x[r, :]
  AdamW     g' = c g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2,
            w = (1 - lr d) w - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
            with c = 1, or min(1, max_norm / |all gradients|_2)
  8-bit states: per block of 256 consecutive elements of a tensor one float32
            scale s = max(amax, 2^-100) / 448 and E4M3 codes of m / s, and the
            same for sqrt(v), whose codes are at least 2^-9 where v > 0
"""
import math

import numpy as np
import torch

own = False

BLOCK = 256        # elements per scale of an 8-bit state
TINY = 2.0 ** -100  # smallest block maximum that a scale is made for
BETA1, BETA2, EPS, LR, DECAY, MAX_NORM = 0.9, 0.95, 1e-8, 3e-4, 0.1, 1.0
STEPS_DONE = 200   # the step count of the states that prepare() makes


def listed():
    return [
        # one token routed to 8 of 16 experts: generation, bound by reading their weights
        {"name": "forward_one_token", "op": "forward", "M": 8, "N": 4096, "K": 7168, "G": 16, "spread": "distinct"},
        # the smallest layer of the tests, with an empty expert: latency
        {"name": "forward_tiny", "op": "forward", "M": 512, "N": 128, "K": 256, "G": 4, "spread": "dirichlet"},
        # many experts with a long tail of short groups
        {"name": "forward_ragged", "op": "forward", "M": 65536, "N": 2048, "K": 7168, "G": 128, "spread": "zipf"},
        # the gate+up projection of a training batch
        {"name": "forward_gate_up", "op": "forward", "M": 32768, "N": 4096, "K": 7168, "G": 16, "spread": "dirichlet"},
        # input gradient of the down projection
        {"name": "dgrad_down", "op": "dgrad", "M": 32768, "N": 7168, "K": 2048, "G": 16, "spread": "dirichlet"},
        # a small batch with sizes that are no multiple of a tile
        {"name": "dgrad_odd", "op": "dgrad", "M": 1531, "N": 1480, "K": 1032, "G": 8, "spread": "dirichlet"},
        # weight gradient of the down projection, added to the float32 gradient of earlier micro-batches
        {"name": "wgrad_down", "op": "wgrad", "M": 32768, "N": 7168, "K": 2048, "G": 16, "spread": "dirichlet",
         "out": "fp32_add"},
        # a small batch with odd sizes, gradient in bf16
        {"name": "wgrad_odd", "op": "wgrad", "M": 1531, "N": 1480, "K": 1032, "G": 8, "spread": "dirichlet",
         "out": "bf16"},
        # norms, biases and a router: many short float32 tensors, latency
        {"name": "adamw_short", "op": "adamw", "tensors": 96, "smallest": 16, "largest": 7168, "state": 32,
         "weights": "fp32", "grad": "fp32", "clip": False},
        # a layer's experts in bf16 with float32 masters, after clipping
        {"name": "adamw_experts", "op": "adamw", "tensors": 48, "smallest": 7168, "largest": 58720256, "state": 32,
         "weights": "master", "grad": "bf16", "clip": True},
        # the short tensors with 8-bit states, after clipping
        {"name": "adamw8_short", "op": "adamw", "tensors": 96, "smallest": 16, "largest": 7168, "state": 8,
         "weights": "master", "grad": "bf16", "clip": True},
        # the layer's experts with 8-bit states, gradients accumulated in float32
        {"name": "adamw8_experts", "op": "adamw", "tensors": 48, "smallest": 7168, "largest": 58720256, "state": 8,
         "weights": "master", "grad": "fp32", "clip": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    """An odd multiple of 8, 64 or 256 from 128 to 7168."""
    unit = rng.choice((8, 64, 256))
    return min(unit * (_log(rng, max(1, 128 // unit), 7168 // unit) | 1), 7168)


def draw(rng):
    op = rng.choice(("forward", "dgrad", "wgrad", "adamw", "adamw"))
    if op == "adamw":
        tensors = _log(rng, 1, 256)
        smallest = _log(rng, 1, 20000)
        largest = max(smallest, _log(rng, 1000, 58720256 // max(1, tensors // 12)))
        return {"op": op, "tensors": tensors, "smallest": smallest, "largest": largest,
                "state": rng.choice((32, 8)), "weights": rng.choice(("fp32", "master", "bf16")),
                "grad": rng.choice(("fp32", "bf16")), "clip": rng.random() < 0.5}
    while True:
        G = _log(rng, 1, 128)
        M = _log(rng, 1 if op == "forward" else 64, 65534) | 1
        N, K = _width(rng), _width(rng)
        if M * N * K <= 32768 * 4096 * 7168 and G * N * K <= 128 * 2048 * 7168:
            break
    case = {"op": op, "M": M, "N": N, "K": K, "G": G, "spread": rng.choice(("dirichlet", "zipf", "even"))}
    if op == "wgrad":
        case["out"] = rng.choice(("bf16", "fp32", "fp32_add"))
    return case


# -- inputs -------------------------------------------------------------------


def _group_sizes(case, seed):
    r = np.random.Generator(np.random.PCG64(seed))
    M, G, spread = case["M"], case["G"], case["spread"]
    if spread == "distinct":  # each row has an expert of its own
        n = np.zeros(G, np.int64)
        n[r.permutation(G)[:M]] = 1
        return n
    if spread == "even":
        p = np.full(G, 1.0 / G)
    elif spread == "dirichlet":
        p = r.dirichlet(np.full(G, 0.5))
    else:
        p = (1.0 + np.arange(G)) ** -1.2
        p = r.permutation(p / p.sum())
    return r.multinomial(M, p)


def _randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)


def _sizes(case):
    T, a, b = case["tensors"], case["smallest"], case["largest"]
    return [int(a * (b / a) ** (i / max(1, T - 1))) if T > 1 else b for i in range(T)]


def _encode(x):
    """E4M3 codes (as float8) and scales of a flat float32 tensor of whole blocks."""
    amax = x.view(-1, BLOCK).abs().amax(1).clamp_min(TINY)
    return (x.view(-1, BLOCK) * (448.0 / amax)[:, None]).to(torch.float8_e4m3fn).view(-1), amax / 448.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] != "adamw":
        M, N, K, G = (case[k] for k in "MNKG")
        sizes = _group_sizes(case, seed)
        ends = np.concatenate([[0], np.cumsum(sizes)])
        s = {"op": case["op"], "ends": [int(e) for e in ends],
             "offsets": torch.from_numpy(ends.astype(np.int32)).cuda()}
        if case["op"] != "wgrad":
            s["w"] = _randn(gen, G, N, K, scale=K ** -0.5 if case["op"] == "forward" else N ** -0.5)
        if case["op"] != "dgrad":
            s["x"] = _randn(gen, M, K)
        if case["op"] != "forward":
            s["dy"] = _randn(gen, M, N)
        if case["op"] == "wgrad":
            kind = torch.bfloat16 if case["out"] == "bf16" else torch.float32
            s["add"] = case["out"] == "fp32_add"
            s["out"] = (_randn(gen, G, N, K, dtype=kind) if s["add"] else
                        torch.zeros((G, N, K), dtype=kind, device="cuda"))
        else:
            s["out"] = torch.zeros((M, N if case["op"] == "forward" else K), dtype=torch.bfloat16, device="cuda")
        return s
    # the tensors are slices of flat buffers, each beginning at a whole block
    sizes = _sizes(case)
    starts = np.concatenate([[0], np.cumsum([-(-n // BLOCK) * BLOCK for n in sizes])]).tolist()
    total = starts[-1]
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, n in zip(starts, sizes):
        inside[a:a + n] = True

    def flat(scale, dtype=torch.float32):
        return _randn(gen, total, scale=scale, dtype=dtype).mul_(inside)

    s = {"op": "adamw", "state": case["state"], "clip": case["clip"], "sizes": sizes, "starts": starts,
         "decay": [DECAY if n > 7168 else 0.0 for n in sizes]}
    master = flat(0.02)
    if case["weights"] == "fp32":
        s["w"], s["master"] = master, None
    else:
        s["w"], s["master"] = master.bfloat16(), master if case["weights"] == "master" else None
    s["g"] = flat(1e-3, torch.bfloat16 if case["grad"] == "bf16" else torch.float32)
    m, r = flat(3e-4), flat(1e-3).abs_()
    if case["state"] == 32:
        s["m"], s["v"] = m, r.square_()
    else:
        (s["m"], s["m_scale"]), (s["v"], s["v_scale"]) = _encode(m), _encode(r)
    s["steps"] = torch.tensor([STEPS_DONE, 0], dtype=torch.int64, device="cuda")
    s["done"] = STEPS_DONE
    if own:
        import mxfp8_block_scaled_04_amd as mx

        def parts(name, per=1):
            t = s.get(name)
            return None if t is None else [t[a // per:(a + n + per - 1) // per] for a, n in zip(starts, sizes)]

        s["plan"] = mx.mx_adamw_plan(parts("w"), parts("g"), parts("m"), parts("v"), masters=parts("master"),
                                     m_scales=parts("m_scale", BLOCK), v_scales=parts("v_scale", BLOCK),
                                     weight_decay=s["decay"])
        s["norm"] = torch.zeros(2, dtype=torch.float32, device="cuda")
    return s


# -- the plain forms ----------------------------------------------------------


def _plain_products(s):
    groups = [(e, a, b) for e, (a, b) in enumerate(zip(s["ends"], s["ends"][1:])) if b > a]
    if s["op"] == "forward":
        done = [s["out"][a:b].copy_(s["x"][a:b].float() @ s["w"][e].float().t()) for e, a, b in groups]
    elif s["op"] == "dgrad":
        done = [s["out"][a:b].copy_(s["dy"][a:b].float() @ s["w"][e].float()) for e, a, b in groups]
    else:
        if not s["add"]:
            s["out"].zero_()
        done = [s["out"][e].add_(s["dy"][a:b].float().t() @ s["x"][a:b].float()) if s["add"] else
                s["out"][e].copy_(s["dy"][a:b].float().t() @ s["x"][a:b].float()) for e, a, b in groups]
    del done
    return s["out"]


def _blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def _plain_decode(codes, scale):
    return (_blocks(codes.float()) * scale[:, None]).view(-1)[:codes.numel()]


def _plain_encode(x, codes, scale):
    b = _blocks(x)
    amax = b.abs().amax(1).clamp_min(TINY)
    scaled = b * (448.0 / amax)[:, None]
    codes.copy_(scaled.view(-1)[:x.numel()].to(torch.float8_e4m3fn))
    scale.copy_(amax / 448.0)


def _plain_tensor(s, i, c, step_size, root):
    """One tensor's step; c: the factor of the gradients."""
    a, n = s["starts"][i], s["sizes"][i]
    part, blocks = slice(a, a + n), slice(a // BLOCK, (a + n + BLOCK - 1) // BLOCK)
    g = s["g"][part].float() * c
    w = s["w"] if s["master"] is None else s["master"]
    if s["state"] == 32:
        m, v = s["m"][part], s["v"][part]
    else:
        m = _plain_decode(s["m"][part], s["m_scale"][blocks])
        v = _plain_decode(s["v"][part], s["v_scale"][blocks]).square()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    new = w[part].float() * (1 - LR * s["decay"][i]) - step_size * (m / (v.sqrt() * root + EPS))
    w[part].copy_(new)
    if s["master"] is not None:
        s["w"][part].copy_(new)
    if s["state"] == 32:
        s["m"][part].copy_(m)
        s["v"][part].copy_(v)
    else:
        _plain_encode(m, s["m"][part], s["m_scale"][blocks])
        r = v.sqrt()
        amax = _blocks(r).amax(1).clamp_min(TINY)
        least = (amax * (2.0 ** -9 / 448.0)).repeat_interleave(BLOCK)[:n]
        _plain_encode(torch.where(v > 0, torch.maximum(r, least), r), s["v"][part], s["v_scale"][blocks])


def _plain_adamw(s):
    s["done"] += 1
    c = 1.0
    if s["clip"]:
        parts = [s["g"][a:a + n].float().square().sum() for a, n in zip(s["starts"], s["sizes"])]
        s["norm_value"] = torch.stack(parts).sum().sqrt()
        c = (MAX_NORM / s["norm_value"]).clamp_max(1.0)
    step_size = LR / (1 - BETA1 ** s["done"])
    root = 1 / math.sqrt(1 - BETA2 ** s["done"])
    done = [_plain_tensor(s, i, c, step_size, root) for i in range(len(s["sizes"]))]
    del done
    return _adamw_outputs(s, s.get("norm_value"))


def _adamw_outputs(s, norm):
    return {k: s[k] for k in ("w", "master", "m", "v", "m_scale", "v_scale") if s.get(k) is not None} | (
        {"norm": norm} if s["clip"] else {})


# -- the package's entry points -----------------------------------------------


def _own(s):
    import mxfp8_block_scaled_04_amd as mx

    if s["op"] == "forward":
        return mx.mx_grouped_gemm_bf16(s["x"], s["w"], s["offsets"], out=s["out"])
    if s["op"] == "dgrad":
        return mx.mx_grouped_gemm_bf16_dgrad(s["dy"], s["w"], s["offsets"], dx=s["out"])
    if s["op"] == "wgrad":
        return mx.mx_grouped_gemm_bf16_wgrad(s["dy"], s["x"], s["offsets"], dw=s["out"], accumulate=s["add"])
    c = None
    if s["clip"]:
        mx.mx_grad_norm(s["plan"], MAX_NORM, out=s["norm"])
        c = s["norm"][1:]
    mx.mx_adamw(s["plan"], s["steps"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, grad_scale=c)
    return _adamw_outputs(s, s["norm"][0])


def run(state):
    if own:
        return _own(state)
    return _plain_adamw(state) if state["op"] == "adamw" else _plain_products(state)


# -- work and exact values ----------------------------------------------------


def work(case):
    if case["op"] != "adamw":
        M, N, K, G = (case[k] for k in "MNKG")
        weights = min(G, M) * N * K  # experts that can have a row
        if case["op"] == "wgrad":
            each = {"bf16": 2, "fp32": 4, "fp32_add": 8}[case["out"]]
            return {"bytes": 2 * M * (N + K) + each * G * N * K, "flops": 2 * M * N * K}
        return {"bytes": 2 * (M * (N + K) + weights), "flops": 2 * M * N * K}
    n = sum(_sizes(case))
    b = {"fp32": 8, "master": 10, "bf16": 4}[case["weights"]] + {"fp32": 4, "bf16": 2}[case["grad"]]
    b += 16 if case["state"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * b, "flops": n * 16}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "adamw":
        out = s["out"].double() if case.get("out") == "fp32_add" else torch.zeros_like(s["out"], dtype=torch.float64)
        for e in range(case["G"]):
            rows = slice(s["ends"][e], s["ends"][e + 1])
            if rows.stop == rows.start:
                continue
            if case["op"] == "forward":
                out[rows] = torch.matmul(s["x"][rows].double(), s["w"][e].double().T)
            elif case["op"] == "dgrad":
                out[rows] = torch.matmul(s["dy"][rows].double(), s["w"][e].double())
            else:
                out[e] += torch.matmul(s["dy"][rows].double().T, s["x"][rows].double())
        return out
    # all tensors at once: whole flat buffers (what lies between the tensors is zero and stays so)
    t = STEPS_DONE + 1
    g = s["g"].double()
    norm = (g * g).sum().sqrt() if case["clip"] else None
    if case["clip"] and float(norm) > MAX_NORM:
        g = g / norm * MAX_NORM
    m, v = s["m"].double(), s["v"].double()
    if case["state"] == 8:
        m = (m.reshape(-1, BLOCK) * s["m_scale"].double().reshape(-1, 1)).reshape(-1)
        v = (v.reshape(-1, BLOCK) * s["v_scale"].double().reshape(-1, 1)).reshape(-1) ** 2
    m += (1 - BETA1) * (g - m)
    v += (1 - BETA2) * (g * g - v)
    w = (s["w"] if s["master"] is None else s["master"]).double()
    lengths = torch.tensor([b - a for a, b in zip(s["starts"], s["starts"][1:])], device="cuda")
    w *= torch.repeat_interleave(1 - LR * torch.tensor(s["decay"], dtype=torch.float64, device="cuda"), lengths)
    w -= LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    out = {"w": w, "m": m, "v": v}
    if s["master"] is not None:
        out["master"] = w
    if case["state"] == 8:
        for name, x in (("m", m), ("v", v.sqrt())):
            scale = torch.clamp(x.reshape(-1, BLOCK).abs().max(1).values, min=TINY) / 448
            coded = x.reshape(-1, BLOCK) / scale[:, None]
            if name == "v":
                coded = torch.where(coded > 0, coded.clamp_min(2.0 ** -9), coded)
            out[name], out[name + "_scale"] = coded.reshape(-1), scale
    if norm is not None:
        out["norm"] = norm
    return out
