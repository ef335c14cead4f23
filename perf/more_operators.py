"""Cases of the 8-bit linear layer, the norm before it, and the router of a mixture-of-experts block.

  norm         h = x + residual (rounded to the type), y = h / sqrt(mean(h^2) + eps) * gamma, and y in int8 with one scale
               per row (``rmsnorm_q8``), with the values that the codes stand for (``dequant_q8``)
  norm_grad    its gradients: dx from dy (y's) and dh (h's own), dgamma (``rmsnorm_grad``)
  linear8      y = (sum_k xq wq) * sx * sw, int8 operands with a scale per token and per output channel; x as codes and
               scales, or as rows that the call quantizes (``gemm_w8a8``)
  router       expert ids and weights of logits: softmax or sigmoid scores, a balancing bias, limited groups, top-k,
               renormalised weights (``moe_route``)
  router_grad  the gradient of the logits from the weights' (``moe_route_grad``)

int8 of a row: s = max|v| / 127, code = v / s to the nearest integer, ties to even (fp32 quotient); a zero row has s = 0.
Choice of experts: by c = score + bias, ties to the lower index; without a bias that order is the logits' own.  An expert
whose logit is minus infinity is never chosen; missing routes have id -1 and weight 0.  A group counts the sum of its
``group_top`` highest c.

``own`` false: plain torch in 32 bits (the router's choice in 64); true: the framework's calls.
"""
import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


def listed():
    return [
        # one token's hidden vector before a layer's projections: the smallest call, latency alone
        {"name": "norm one token", "op": "norm", "rows": 1, "D": 4096, "residual": True, "y": False, "dtype": "bf16"},
        # a long prompt in a wide model, the normed rows kept for the router beside their codes: the largest
        {"name": "norm prompt", "op": "norm", "rows": 8192, "D": 8192, "residual": True, "y": True, "dtype": "bf16"},
        # a small fp32 fine-tuning step, an odd width, the residual's gradient absent
        {"name": "norm gradient fp32 odd", "op": "norm_grad", "rows": 333, "D": 1001, "dh": False, "dtype": "fp32"},
        # the gradient of a training step
        {"name": "norm gradient", "op": "norm_grad", "rows": 8192, "D": 4096, "dh": True, "dtype": "bf16"},
        # the gate projection of an 8B-shaped layer for a single token: weight streaming
        {"name": "linear decode", "op": "linear8", "M": 1, "N": 14336, "K": 4096, "codes": False, "dtype": "bf16"},
        # batched decode on the down projection, an odd batch, x already in codes
        {"name": "linear batch 37", "op": "linear8", "M": 37, "N": 4096, "K": 14336, "codes": True, "dtype": "fp16"},
        # a ragged middle-sized batch through a narrow expert's projection
        {"name": "linear ragged", "op": "linear8", "M": 333, "N": 1408, "K": 2048, "codes": False, "dtype": "bf16"},
        # a long prompt through a square 70B-shaped projection: the largest product
        {"name": "linear prompt", "op": "linear8", "M": 8192, "N": 8192, "K": 8192, "codes": True, "dtype": "bf16"},
        # routing of one decode step: softmax over the two chosen of 8
        {"name": "router decode", "op": "router", "T": 5, "E": 8, "k": 2, "score": "softmax", "bias": False, "groups": 1,
         "top_groups": 1, "group_top": 1, "renorm": True, "mask": False, "dtype": "bf16"},
        # a prompt over many experts: sigmoid scores, a balancing bias, half of the groups
        {"name": "router prompt", "op": "router", "T": 8191, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "group_top": 2, "renorm": True, "mask": False, "dtype": "fp32"},
        # its gradient in a small fine-tuning step, weights not renormalised: every logit of a row gets one
        {"name": "router gradient fp32", "op": "router_grad", "T": 129, "E": 60, "k": 4, "score": "softmax", "renorm": False,
         "dtype": "fp32"},
        # the gradient of a training step
        {"name": "router gradient", "op": "router_grad", "T": 8192, "E": 256, "k": 8, "score": "sigmoid", "renorm": True,
         "dtype": "bf16"},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["norm", "norm_grad", "linear8", "linear8", "router", "router_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_grad"):
        c = {"op": op, "rows": log(1, 16384), "D": log(64, 16384), "dtype": dtype}
        while c["rows"] * c["D"] * BYTES[dtype] > 1.0e8:
            c["rows"] = c["rows"] // 2 + 1
        if op == "norm":
            return c | {"residual": rng.random() < 0.7, "y": rng.random() < 0.5}
        return c | {"dh": rng.random() < 0.7}
    if op == "linear8":
        c = {"op": op, "M": log(1, 8192), "N": log(64, 16384), "K": 16 * log(8, 896), "codes": rng.random() < 0.5, "dtype": dtype}
        while 2.0 * c["M"] * c["N"] * c["K"] > 1.0e12:
            c["M"] = c["M"] // 2
        return c
    T, score, renorm = log(1, 8192), rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6
    if op == "router_grad":
        E = log(2, 512)
        k = rng.choice([2, 2, 4, 6, 8] if renorm else [1, 2, 4, 6, 8])        # one renormalised weight is 1: no gradient
        return {"op": op, "T": T, "E": E, "k": min(k, E), "score": score, "renorm": renorm, "dtype": dtype}
    groups = rng.choice([1, 1, 4, 8])
    E = groups * log(2 if groups == 1 else 4, 512 // groups)
    top_groups = rng.randint((groups + 1) // 2, groups)
    k = min(rng.choice([1, 2, 4, 6, 8]), E // groups * top_groups)
    return {"op": op, "T": T, "E": E, "k": k, "score": score, "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups,
            "group_top": rng.choice([1, 2]), "renorm": renorm, "mask": rng.random() < 0.2, "dtype": dtype}


def work(c):
    b = BYTES[c["dtype"]]
    if c["op"] == "norm":
        n = c["rows"] * c["D"]
        # x (and the residual) and gamma read; h (where there is a residual), y, codes, scales and the codes' values written
        return {"bytes": n * (b * (1 + 2 * c["residual"] + c["y"]) + 3) + b * c["D"] + 4 * c["rows"], "flops": 8.0 * n}
    if c["op"] == "norm_grad":
        n = c["rows"] * c["D"]
        return {"bytes": n * b * (3 + c["dh"]) + (b + 4) * c["D"], "flops": 10.0 * n}
    if c["op"] == "linear8":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K * (1 if c["codes"] else b) + N * K + 4 * (M * c["codes"] + N) + b * M * N, "flops": 2.0 * M * N * K}
    if c["op"] == "router":
        return {"bytes": c["T"] * c["E"] * b + 4 * c["E"] * c["bias"] + 8 * c["T"] * c["k"], "flops": 8.0 * c["T"] * c["E"]}
    return {"bytes": 2 * c["T"] * c["E"] * b + 8 * c["T"] * c["k"], "flops": 8.0 * c["T"] * c["E"]}


# ---------------------------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _hidden(g, rows, cols):
    """fp32 N(0, 1) with a few columns of outliers (20x), as hidden states have, and a few rows of padding (zeros)."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    loud = torch.rand(cols, generator=g, device="cuda") < 0.002
    pad = torch.rand(rows, 1, generator=g, device="cuda") < 0.01
    return torch.where(pad, 0.0, torch.where(loud, x * 20.0, x))


def _logits(g, c):
    x = torch.randn(c["T"], c["E"], generator=g, device="cuda") + 0.7 * torch.randn(c["E"], generator=g, device="cuda")
    if c.get("mask"):
        x = torch.where(torch.rand(c["T"], c["E"], generator=g, device="cuda") < 0.1, float("-inf"), x)
    return x.to(DTYPE[c["dtype"]])


def prepare(c, seed):
    g, d = _gen(seed), DTYPE[c["dtype"]]
    s = dict(c)
    if c["op"] in ("norm", "norm_grad"):
        rows, D = c["rows"], c["D"]
        s["gamma"] = (1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(d)
        if c["op"] == "norm":
            s["x"] = _hidden(g, rows, D).to(d)
            s["r"] = _hidden(g, rows, D).to(d) if c["residual"] else None
        else:
            s["h"] = _hidden(g, rows, D).to(d)
            dy = torch.randn(rows, D, generator=g, device="cuda")
            s["dy"] = torch.where((s["h"] != 0).any(dim=1, keepdim=True), dy, 0.0).to(d)      # padding has no gradient
            s["d"] = torch.randn(rows, D, generator=g, device="cuda").to(d) if c["dh"] else None
        return s
    if c["op"] == "linear8":
        # the weight as a program keeps it: codes and one scale per output channel
        s["w"], s["sw"] = _int8(torch.randn(c["N"], c["K"], generator=g, device="cuda") * 0.02)
        x = _hidden(g, c["M"], c["K"])
        if c["codes"]:
            s["x"], s["sx"] = _int8(x)
        else:
            s["x"] = x.to(d)
        return s
    s["logits"] = _logits(g, c)
    if c["op"] == "router":
        s["b"] = 0.1 * torch.randn(c["E"], generator=g, device="cuda") if c["bias"] else None
        return s
    s["ids"] = torch.topk(s["logits"].float(), c["k"], dim=1).indices.to(torch.int32).contiguous()
    s["dw"] = torch.randn(c["T"], c["k"], generator=g, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------
# plain forms

def _int8(v):
    """int8 codes and fp32 scales [rows] of fp32 rows."""
    s = v.abs().amax(dim=1) / 127.0
    q = torch.where(s[:, None] > 0, torch.round(v / s[:, None]), 0.0).clamp(-127, 127)
    return q.to(torch.int8), s


def _scores(x, score):
    """Scores of logits [T][E] in x's precision; a row of minus infinities has zeros."""
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(dim=1, keepdim=True).clamp(min=-3e38))
    return e / e.sum(dim=1, keepdim=True).clamp(min=1e-30)


def _scale(s):
    """The factor of the weights (a routed branch is scaled up where they are renormalised sigmoids)."""
    return 2.5 if s["score"] == "sigmoid" and s["renorm"] else 1.0


def _route(s):
    T, E, G = s["T"], s["E"], s["groups"]
    low = float("-inf")
    x = s["logits"].double()
    value = _scores(x, s["score"])
    choice = torch.where(x > low, x if s["b"] is None else value + s["b"].double(), low)
    if G > 1:
        member = choice if s["b"] is not None or s["group_top"] == 1 else torch.where(x > low, value, low)
        best = torch.sort(member.view(T, G, E // G), dim=2, descending=True).values[:, :, :s["group_top"]]
        total = torch.where(best[:, :, 0] > low, torch.where(best > low, best, 0.0).sum(dim=2), low)
        kept = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        choice = torch.where(open_.repeat_interleave(E // G, dim=1), choice, low)
    top, ids = (v[:, :s["k"]] for v in torch.sort(choice, dim=1, descending=True, stable=True))
    weights = torch.where(top > low, value.gather(1, ids), 0.0)
    if s["renorm"]:
        weights = weights / weights.sum(dim=1, keepdim=True).clamp(min=1e-300)
    return {"ids": torch.where(top > low, ids, -1).to(torch.int32), "weights": (weights * _scale(s)).to(torch.float32)}


def _plain(s):
    d = DTYPE[s["dtype"]]
    if s["op"] == "norm":
        h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(d)
        y = h.float()
        y = y / torch.sqrt((y * y).mean(dim=1, keepdim=True) + EPS) * s["gamma"].float()
        q, scale = _int8(y)
        out = {"values": (q.float() * scale[:, None]).to(torch.bfloat16), "scale": scale}
        if s["r"] is not None:
            out["h"] = h
        if s["y"]:
            out["y"] = y.to(d)
        return out
    if s["op"] == "norm_grad":
        h, dy = s["h"].float(), s["dy"].float()
        r = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)
        n, g = h * r, dy * s["gamma"].float()
        dx = r * (g - n * (g * n).mean(dim=1, keepdim=True))
        if s["d"] is not None:
            dx = dx + s["d"].float()
        return {"dx": dx.to(d), "dgamma": (dy * n).sum(dim=0)}
    if s["op"] == "linear8":
        x, sx = (s["x"], s["sx"]) if s["codes"] else _int8(s["x"].float())
        return {"y": ((x.float() @ s["w"].float().t()) * sx[:, None] * s["sw"]).to(d)}
    if s["op"] == "router":
        return _route(s)
    x, ids, dw = s["logits"].float(), s["ids"].long(), s["dw"] * _scale(s)
    value = _scores(x, s["score"])
    zero = torch.zeros_like(x)
    if s["renorm"]:
        at = value.gather(1, ids)
        w = at / at.sum(dim=1, keepdim=True)
        dx = w * (dw - (w * dw).sum(dim=1, keepdim=True))
        if s["score"] == "sigmoid":
            dx = dx * (1.0 - at)
        return {"dx": zero.scatter_add_(1, ids, dx).to(d)}
    ds = zero.scatter_add_(1, ids, dw)
    if s["score"] == "sigmoid":
        return {"dx": (ds * value * (1.0 - value)).to(d)}
    return {"dx": (value * (ds - (value * ds).sum(dim=1, keepdim=True))).to(d)}


# ---------------------------------------------------------------------------------------------
# the framework's calls

def _framework(s):
    import gemm_uq_gb300 as uq
    if s["op"] == "norm":
        h, y, (q, scale) = uq.rmsnorm_q8(s["x"], s["gamma"], EPS, residual=s["r"], normed=s["y"])
        out = {"values": uq.dequant_q8((q, scale)), "scale": scale}
        if s["r"] is not None:
            out["h"] = h
        if s["y"]:
            out["y"] = y
        return out
    if s["op"] == "norm_grad":
        dx, dgamma = uq.rmsnorm_grad(s["dy"], s["h"], s["gamma"], EPS, dh=s["d"])
        return {"dx": dx, "dgamma": dgamma}
    if s["op"] == "linear8":
        x = (s["x"], s["sx"]) if s["codes"] else s["x"]
        return {"y": uq.gemm_w8a8(x, (s["w"], s["sw"]), dtype=DTYPE[s["dtype"]])}
    if s["op"] == "router":
        ids, weights = uq.moe_route(s["logits"], s["k"], score=s["score"], bias=s["b"], groups=s["groups"],
                                    top_groups=s["top_groups"], group_top=s["group_top"], renormalize=s["renorm"],
                                    scale=_scale(s))
        return {"ids": ids, "weights": weights}
    return {"dx": uq.moe_route_grad(s["logits"], s["ids"], s["dw"], score=s["score"], renormalize=s["renorm"], scale=_scale(s))}


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _codes64(v):
    """The values of int8 rows: scale by the definition's fp32 division, the quotient rounded to fp32, then to an integer."""
    s = (v.abs().max(dim=1).values.float() / 127.0).double()
    q = torch.round((v / torch.where(s > 0, s, 1.0)[:, None]).float().double())
    return q, s


def _chosen64(c, x, b):
    """The experts of each token in order, -1 for a missing one, by sorting (choice, index) in Python's own order."""
    of = torch.softmax(x, dim=1) if c["score"] == "softmax" else torch.sigmoid(x)
    value = (of if b is None else of + b).tolist()
    first = x.tolist() if b is None else value                     # without a bias the logits' order
    size, k, low = c["E"] // c["groups"], c["k"], float("-inf")
    out = []
    for t, row in enumerate(x.tolist()):
        on = [e for e in range(c["E"]) if row[e] > low]
        if c["groups"] > 1:
            by = first[t] if c["group_top"] == 1 else value[t]
            parts = {}
            for e in on:
                parts.setdefault(e // size, []).append(by[e])
            total = {g: sum(sorted(v, reverse=True)[:c["group_top"]]) for g, v in parts.items()}
            kept = sorted(total, key=lambda g: (-total[g], g))[:c["top_groups"]]
            on = [e for e in on if e // size in kept]
        best = sorted(on, key=lambda e: (-first[t][e], e))[:k]
        out.append(best + [-1] * (k - len(best)))
    return torch.tensor(out, dtype=torch.long).view(-1, k)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        h = s["x"].double()
        if c["residual"]:
            h = (h + s["r"].double()).to(DTYPE[c["dtype"]]).double()
        y = s["gamma"].double() * h * torch.rsqrt(h.pow(2).sum(dim=1, keepdim=True) / c["D"] + EPS)
        scale = y.abs().max(dim=1).values / 127
        values = torch.round(y / torch.where(scale > 0, scale, 1.0)[:, None]) * scale[:, None]
        out = {"values": values, "scale": scale}
        if c["residual"]:
            out["h"] = h
        if c["y"]:
            out["y"] = y
        return out
    if c["op"] == "norm_grad":
        h = s["h"].double().requires_grad_()
        gamma = s["gamma"].double().requires_grad_()
        y = h * torch.rsqrt(h.pow(2).sum(dim=1, keepdim=True) / c["D"] + EPS) * gamma
        dx, dgamma = torch.autograd.grad(y, (h, gamma), s["dy"].double())
        return {"dx": dx + s["d"].double() if c["dh"] else dx, "dgamma": dgamma}
    if c["op"] == "linear8":
        x, sx = (s["x"].double(), s["sx"].double()) if c["codes"] else _codes64(s["x"].double())
        return {"y": torch.einsum("mk,nk->mn", x, s["w"].double()) * torch.outer(sx, s["sw"].double())}
    x = s["logits"].double()
    if c["op"] == "router":
        ids = _chosen64(c, x.cpu(), s["b"].double().cpu() if c["bias"] else None).cuda()
        of = torch.softmax(x, dim=1) if c["score"] == "softmax" else torch.sigmoid(x)
        w = torch.where(ids >= 0, of.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=torch.float64, device="cuda"))
        return {"ids": None, "weights": _scale(c) * (torch.nn.functional.normalize(w, p=1, dim=1, eps=1e-300) if c["renorm"] else w)}
    x.requires_grad_()
    of = torch.softmax(x, dim=1) if c["score"] == "softmax" else torch.sigmoid(x)
    w = of.gather(1, s["ids"].long())
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return {"dx": torch.autograd.grad(_scale(c) * w, x, s["dw"].double())[0]}
