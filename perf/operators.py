"""Cases of the microscaled 4-bit operators and of the expert routing around them.

Four operators of a mixture-of-experts layer whose weights and activations are held in
microscaled 4-bit floating point:

  quantize   rows of bf16 / fp16 / fp32 -> e2m1 codes with one scale per block, and the values
             they stand for (``quantize_mx``, ``dequant_mx``)
  product    y = x^ W^T with both operands microscaled, x quantized in the call (``gemm_mx``)
  experts    the same product for rows sorted by expert, each expert with its own weight;
             ``gated``: silu(x^ Wg^T) * (x^ Wu^T) (``quantize_mx`` with ``pos``, ``gemm_mx_grouped``)
  route      tokens sorted by expert, and back with the router's weights applied
             (``moe_sort``, ``moe_gather``, ``moe_combine``); route_grad: the gradients of both
             directions (``moe_combine_grad``, ``moe_gather_grad``)

Formats.  MXFP4: blocks of 32, scale 2^e, e = floor(log2(absmax)) - 2.  NVFP4: blocks of 16, scale
the e4m3 value nearest absmax / 6.  Element: the e2m1 value nearest x / scale (ties to the even
code, at most 6 in magnitude).  A weight is in hand as codes (two per byte, low nibble = even k)
and scales in 512-byte tiles of 128 rows x 4 blocks, byte (r % 32) * 16 + (r / 32) * 4 + block.

``own`` false: plain torch in 32 bits; true: the framework's calls.
"""
import torch

own = False

BLOCK = {"MXFP4": 32, "NVFP4": 16}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token's hidden vector entering a down projection: the smallest call, latency alone
        {"name": "quantize one token", "op": "quantize", "fmt": "MXFP4", "rows": 1, "K": 14336, "dtype": "bf16"},
        # a prompt's activations, an odd number of rows, in the finer format
        {"name": "quantize prompt nvfp4", "op": "quantize", "fmt": "NVFP4", "rows": 8191, "K": 4096, "dtype": "bf16"},
        # the gate projection of an 8B-shaped layer for a single token: weight streaming
        {"name": "product decode", "op": "product", "fmt": "MXFP4", "M": 1, "N": 14336, "K": 4096, "dtype": "bf16"},
        # batched decode on the down projection, an odd batch
        {"name": "product batch 37 nvfp4", "op": "product", "fmt": "NVFP4", "M": 37, "N": 4096, "K": 14336, "dtype": "fp16"},
        # a long prompt through a square 70B-shaped projection: the largest product
        {"name": "product prompt", "op": "product", "fmt": "MXFP4", "M": 8192, "N": 8192, "K": 8192, "dtype": "bf16"},
        # gate and up of 8 experts for a decode batch of 3 tokens, 2 experts each
        {"name": "experts decode gated", "op": "experts", "fmt": "MXFP4", "T": 3, "k": 2, "E": 8, "N": 14336,
         "K": 4096, "gated": True, "drop": False, "dtype": "bf16"},
        # many small experts, a ragged middle-sized batch, some routes dropped, some experts empty
        {"name": "experts ragged nvfp4", "op": "experts", "fmt": "NVFP4", "T": 333, "k": 4, "E": 64, "N": 1408,
         "K": 2048, "gated": False, "drop": True, "dtype": "bf16"},
        # the down projection of 8 experts for a prompt
        {"name": "experts prompt", "op": "experts", "fmt": "MXFP4", "T": 4096, "k": 2, "E": 8, "N": 4096,
         "K": 14336, "gated": False, "drop": False, "dtype": "bf16"},
        # routing of one decode step
        {"name": "route decode", "op": "route", "T": 5, "k": 2, "E": 8, "H": 4096, "drop": False, "dtype": "bf16"},
        # routing of a prompt over many experts with dropped routes
        {"name": "route prompt", "op": "route", "T": 8191, "k": 8, "E": 64, "H": 4096, "drop": True, "dtype": "bf16"},
        # its gradient in a small fp32 fine-tuning step, an odd width
        {"name": "route gradient fp32 odd", "op": "route_grad", "T": 129, "k": 4, "E": 16, "H": 1001, "drop": True,
         "dtype": "fp32"},
        # the gradient of a training step
        {"name": "route gradient", "op": "route_grad", "T": 8192, "k": 4, "E": 32, "H": 4096, "drop": False,
         "dtype": "bf16"},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["quantize", "product", "product", "experts", "experts", "route", "route_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    fmt = rng.choice(["MXFP4", "NVFP4"])
    if op == "quantize":
        return {"op": op, "fmt": fmt, "rows": log(1, 8192), "K": 32 * log(4, 448), "dtype": dtype}
    half = rng.choice(["bf16", "bf16", "fp16"])
    if op == "product":
        c = {"op": op, "fmt": fmt, "M": log(1, 8192), "N": log(512, 16384), "K": 32 * log(16, 448), "dtype": half}
        while 2.0 * c["M"] * c["N"] * c["K"] > 1.0e12:
            c["M"] = c["M"] // 2
        return c
    if op == "experts":
        c = {"op": op, "fmt": fmt, "T": log(1, 4096), "k": rng.choice([1, 2, 4, 6, 8]), "E": rng.choice([8, 16, 32, 64]),
             "N": 8 * log(64, 1024), "K": 32 * log(16, 256), "gated": rng.random() < 0.4, "drop": rng.random() < 0.5,
             "dtype": half}
        while c["E"] * c["N"] * c["K"] > 4.0e8:
            c["N"] = c["N"] // 16 * 8
        while c["T"] * c["k"] > 16384:
            c["T"] = c["T"] // 2
        return c
    c = {"op": op, "T": log(1, 8192), "k": rng.choice([1, 2, 4, 6, 8]), "E": rng.choice([4, 8, 16, 60, 64, 128]),
         "H": log(64, 8192), "drop": rng.random() < 0.5, "dtype": dtype}
    while c["T"] * c["k"] * c["H"] * BYTES[dtype] > 5.0e8:
        c["T"] = c["T"] // 2 + 1
    return c


def work(c):
    if c["op"] == "quantize":
        n = c["rows"] * c["K"]
        # x read; codes and scales written; their values written
        return {"bytes": n * (BYTES[c["dtype"]] + 0.5 + 1 / BLOCK[c["fmt"]] + 2), "flops": 0}
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": 2 * M * K + N * K * (0.5 + 1 / BLOCK[c["fmt"]]) + 2 * M * N, "flops": 2.0 * M * N * K}
    R, E = c["T"] * c["k"], c["E"]
    if c["op"] == "experts":
        NW, K = c["N"] * (2 if c["gated"] else 1), c["K"]
        kept = R * (0.9 if c["drop"] else 1.0)
        active = E * (1.0 - (1.0 - 1.0 / E) ** kept)         # experts that get a row, by an even router
        return {"bytes": 2 * c["T"] * K + active * NW * K * (0.5 + 1 / BLOCK[c["fmt"]]) + 2 * R * c["N"],
                "flops": 2.0 * kept * NW * K}
    H, b = c["H"], BYTES[c["dtype"]]
    if c["op"] == "route":
        # ids in, order / pos / offsets out; x read and sorted rows written; rows and weights read, y written
        return {"bytes": 4 * R + 8 * R + 4 * (E + 1) + b * H * (c["T"] + R) + b * H * (R + c["T"]) + 4 * R,
                "flops": 2.0 * R * H}
    # dy, ys, weights read and dys, dw written; dxs read and dx written
    return {"bytes": b * H * (c["T"] + 2 * R) + 8 * R + 4 * R + b * H * (R + c["T"]), "flops": 4.0 * R * H}


# ---------------------------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _activations(g, rows, cols):
    """fp32 N(0, 1) with a few columns of outliers (20x), as hidden states have."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    loud = torch.rand(cols, generator=g, device="cuda") < 0.002
    return torch.where(loud, x * 20.0, x)


def _weight(g, experts, rows, K, fmt):
    """Codes [experts*rows][K/2], natural scales [experts*rows][K/block] and the tiled scales of each expert."""
    codes, scales, tiles = [], [], []
    for _ in range(experts):
        w = torch.randn(rows, K, generator=g, device="cuda") * 0.02
        q, s = _codes(w, fmt)
        codes.append(q[:, 0::2] | (q[:, 1::2] << 4))
        scales.append(s)
        tiles.append(_tile(s))
    return torch.cat(codes), torch.cat(scales), torch.stack(tiles)


def _tile(s):
    """Natural scales [rows][blocks] -> [row tiles][block tiles][32][4][4] uint8."""
    rows, nb = s.shape
    rt, bt = -(-rows // 128), -(-nb // 4)
    p = torch.zeros(rt * 128, bt * 4, dtype=torch.uint8, device=s.device)
    p[:rows, :nb] = s
    return p.view(rt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).contiguous()


def _routing(g, c):
    """Expert ids [T][k] (distinct per token; -1 = dropped) and fp32 weights, from a router with popular experts."""
    T, k, E = c["T"], min(c["k"], c["E"]), c["E"]
    logits = torch.randn(T, E, generator=g, device="cuda") + 0.7 * torch.randn(E, generator=g, device="cuda")
    top, ids = torch.topk(logits, k, dim=1)
    weights = torch.softmax(top, dim=1)
    ids = ids.to(torch.int32)
    if c["drop"]:
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.1, torch.full_like(ids, -1), ids)
    return ids.contiguous(), weights.contiguous()


def prepare(c, seed):
    g = _gen(seed)
    s = dict(c)
    if c["op"] == "quantize":
        x = _activations(g, c["rows"], c["K"])
        x[:, :32] = torch.where(torch.rand(c["rows"], 1, generator=g, device="cuda") < 0.1, 0.0, x[:, :32])   # zero blocks
        s["x"] = x.to(DTYPE[c["dtype"]])
        return s
    if c["op"] == "product":
        s["x"] = _activations(g, c["M"], c["K"]).to(DTYPE[c["dtype"]])
        s["codes"], s["scales"], s["tiles"] = _weight(g, 1, c["N"], c["K"], c["fmt"])
        s["tiles"] = s["tiles"][0]
        return s
    ids, weights = _routing(g, c)
    T, k = ids.shape
    if c["op"] == "route":
        s["x"] = _activations(g, T, c["H"]).to(DTYPE[c["dtype"]])
        s["ys"] = torch.randn(T * k, c["H"], generator=g, device="cuda").to(DTYPE[c["dtype"]])
        s["ids"], s["weights"] = ids, weights
        return s
    s["order"], s["pos"], s["offsets"] = _sort(ids, c["E"])
    if c["op"] == "route_grad":
        d = DTYPE[c["dtype"]]
        s["dy"] = torch.randn(T, c["H"], generator=g, device="cuda").to(d)
        s["ys"] = torch.randn(T * k, c["H"], generator=g, device="cuda").to(d)
        s["dxs"] = torch.randn(T * k, c["H"], generator=g, device="cuda").to(d)
        s["weights"] = weights
        return s
    s["x"] = _activations(g, T, c["K"]).to(DTYPE[c["dtype"]])
    for part in ("", "up_") if c["gated"] else ("",):
        codes, scales, s[part + "tiles"] = _weight(g, c["E"], c["N"], c["K"], c["fmt"])
        s[part + "codes"], s[part + "scales"] = codes.view(c["E"], c["N"], -1), scales.view(c["E"], c["N"], -1)
    # for the plain form: the rows of each expert, padded to the longest with row R (a zero row)
    off = s["offsets"].long()
    count = off[1:] - off[:-1]
    cap = max(1, int(count.max()))
    slot = off[:-1, None] + torch.arange(cap, device="cuda")[None, :]
    s["slots"] = torch.where(slot < off[1:, None], slot, T * k)
    return s


# ---------------------------------------------------------------------------------------------
# plain forms

def _codes(x, fmt):
    """e2m1 code indices (uint8 0..15) and scale bytes of fp32 rows."""
    rows, K = x.shape
    b = x.reshape(rows, K // BLOCK[fmt], BLOCK[fmt])
    amax = b.abs().amax(dim=2, keepdim=True)
    if fmt == "MXFP4":
        e = torch.where(amax > 0, (torch.frexp(amax).exponent - 3).clamp(-127, 127), -127)
        a = torch.ldexp(b, -e).abs()
        byte = (e + 127).to(torch.uint8)
    else:
        s8 = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        s = s8.to(torch.float32)
        a = torch.where(s > 0, (b / s).abs(), 0.0)
        byte = s8.view(torch.uint8)
    a = a.clamp(max=6.0)
    # half steps below 2, whole steps to 4, steps of 2 above; the multiples' parity is the code's
    code = torch.where(a < 2.0, torch.round(a * 2.0), torch.where(a < 4.0, torch.round(a) + 2.0, torch.round(a * 0.5) + 4.0))
    q = code.to(torch.uint8) | (torch.signbit(b).to(torch.uint8) << 3)
    return q.reshape(rows, K), byte.reshape(rows, K // BLOCK[fmt])


def _scale_values(byte, fmt):
    if fmt == "MXFP4":
        return torch.ldexp(torch.ones((), device=byte.device), byte.to(torch.int32) - 127)
    return byte.view(torch.float8_e4m3fn).to(torch.float32)


def _values(q, byte, fmt):
    """fp32 values of code indices [..., K] and scale bytes [..., K/block]."""
    lut = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float32, device=q.device)
    v = lut[q.to(torch.int32)]
    s = _scale_values(byte, fmt)
    return (v.view(*s.shape, BLOCK[fmt]) * s.unsqueeze(-1)).view(v.shape)


def _rounded(x, fmt):
    return _values(*_codes(x.to(torch.float32), fmt), fmt)


def _unpacked(codes):
    return torch.stack((codes & 15, codes >> 4), dim=-1).reshape(*codes.shape[:-1], -1)


def _sort(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device=ids.device)
    pos = torch.where(key < E, pos, -1)
    offsets = (key[None, :] < torch.arange(E + 1, device=ids.device)[:, None]).sum(dim=1)
    order = torch.where(torch.arange(T * k, device=ids.device) < offsets[E], order, -1)
    return order.to(torch.int32), pos.reshape(T, k).to(torch.int32), offsets.to(torch.int32)


def _taken(rows, pos):
    """fp32 rows[pos] [T][k][H], zero where pos is -1."""
    got = rows.to(torch.float32)[pos.long().clamp(min=0)]
    return torch.where((pos >= 0)[..., None], got, 0.0)


def _spread(values, pos, like):
    """values [T][k][H] laid at their rows; rows that nothing points to are zero."""
    R, H = pos.numel(), values.shape[-1]
    out = torch.zeros(R + 1, H, dtype=torch.float32, device=pos.device)
    out[torch.where(pos >= 0, pos.long(), R).reshape(-1)] = values.reshape(R, H)
    return out[:R].to(like.dtype)


def _plain(s):
    if s["op"] == "quantize":
        return {"values": _rounded(s["x"], s["fmt"]).to(torch.bfloat16)}
    if s["op"] == "product":
        w = _values(_unpacked(s["codes"]), s["scales"], s["fmt"])
        return {"y": (_rounded(s["x"], s["fmt"]) @ w.t()).to(s["x"].dtype)}
    if s["op"] == "experts":
        x = _rounded(s["x"], s["fmt"])
        R, k = s["pos"].numel(), s["pos"].shape[1]
        x = torch.cat((x, torch.zeros_like(x[:1])))
        token = torch.cat((torch.where(s["order"] >= 0, s["order"].long() // k, x.shape[0] - 1),
                           torch.full((1,), x.shape[0] - 1, device=x.device)))
        x = x[token[s["slots"]]]
        y = torch.bmm(x, _values(_unpacked(s["codes"]), s["scales"], s["fmt"]).transpose(1, 2))
        if s["gated"]:
            up = torch.bmm(x, _values(_unpacked(s["up_codes"]), s["up_scales"], s["fmt"]).transpose(1, 2))
            y = y / (1.0 + torch.exp(-y)) * up
        out = torch.zeros(R + 1, s["N"], dtype=torch.float32, device=x.device)
        out[s["slots"].reshape(-1)] = y.reshape(-1, s["N"])
        return {"y": out[:R].to(torch.bfloat16)}
    if s["op"] == "route":
        order, pos, offsets = _sort(s["ids"], s["E"])
        x = s["x"]
        xs = _spread(x.to(torch.float32)[:, None, :].expand(-1, pos.shape[1], -1), pos, x)
        y = (_taken(s["ys"], pos) * s["weights"][..., None]).sum(dim=1).to(x.dtype)
        return {"order": order, "pos": pos, "offsets": offsets, "xs": xs, "y": y}
    dy = s["dy"].to(torch.float32)[:, None, :]
    dys = _spread(dy * s["weights"][..., None], s["pos"], s["ys"])
    dw = (dy * _taken(s["ys"], s["pos"])).sum(dim=2)
    dx = _taken(s["dxs"], s["pos"]).sum(dim=1).to(s["dxs"].dtype)
    return {"dys": dys, "dw": dw, "dx": dx}


# ---------------------------------------------------------------------------------------------
# the framework's calls

def _framework(s):
    import gemm_uq_gb300 as uq
    if s["op"] == "quantize":
        q = uq.quantize_mx(s["x"], s["fmt"])
        return {"values": uq.dequant_mx(q, s["fmt"])}
    if s["op"] == "product":
        return {"y": uq.gemm_mx(s["x"], (s["codes"], s["tiles"]), s["fmt"])}
    if s["op"] == "experts":
        q = uq.quantize_mx(s["x"], s["fmt"], offsets=s["offsets"], pos=s["pos"])
        up = (s["up_codes"], s["up_tiles"]) if s["gated"] else None
        return {"y": uq.gemm_mx_grouped(q, (s["codes"], s["tiles"]), s["offsets"], s["fmt"], up=up)}
    if s["op"] == "route":
        order, pos, offsets = uq.moe_sort(s["ids"], s["E"])
        xs = uq.moe_gather(s["x"], pos, offsets)
        y = uq.moe_combine(s["ys"], pos, s["weights"])
        return {"order": order, "pos": pos, "offsets": offsets, "xs": xs, "y": y}
    dys, dw = uq.moe_combine_grad(s["dy"], s["ys"], s["pos"], s["weights"], s["offsets"])
    return {"dys": dys, "dw": dw, "dx": uq.moe_gather_grad(s["dxs"], s["pos"])}


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _exponent(a):
    """floor(log2 a) of float64 a >= 0 (-126 below 2^-126), a rounded logarithm put right at the powers of two."""
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -126)))
    return e + (torch.exp2(e + 1) <= a).double() - (torch.exp2(e) > a.clamp(min=2.0 ** -126)).double()


def _exact_rounded(x, fmt):
    """Each value's nearest representable one, in float64, from the definition by comparisons with the midpoints."""
    n = BLOCK[fmt]
    b = x.double().view(x.shape[0], -1, n)
    amax = b.abs().max(dim=2, keepdim=True).values
    if fmt == "MXFP4":
        step = torch.exp2((_exponent(amax) - 2).clamp(-127, 127))
    else:
        t = amax / 6
        unit = torch.exp2(_exponent(t).clamp(min=-6) - 3)
        step = (torch.round(t / unit) * unit).clamp(max=448.0)
    a = b.abs()
    code = torch.zeros_like(a)
    for i in range(7):
        mid = (GRID[i] + GRID[i + 1]) / 2 * step
        code += ((a > mid) | ((a == mid) & (i % 2 == 1))) & (step > 0)     # a tie goes to the even code
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    return (torch.sign(b) * grid[code.long()] * step).view(x.shape)


def _exact_weight(codes, scales, fmt):
    """float64 weight of packed codes and natural scale bytes, from the formats' bit fields."""
    c = torch.stack((codes % 16, codes // 16), dim=-1).flatten(-2).short()
    e, m = (c % 8) // 2, c % 2
    mag = torch.where(e > 0, torch.exp2(e.double() - 1) * (1 + m.double() / 2), m.double() / 2)
    v = torch.where(c >= 8, -mag, mag)
    b = scales.short()
    if fmt == "MXFP4":
        s = torch.exp2(b.double() - 127)
    else:
        f = (b % 8).double()
        x = b // 8
        s = torch.where(x > 0, torch.exp2(x.double() - 7) * (1 + f / 8), f / 512)
    return v * s.repeat_interleave(BLOCK[fmt], dim=-1)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "quantize":
        return {"values": _exact_rounded(s["x"], c["fmt"])}
    if c["op"] == "product":
        w = _exact_weight(s["codes"], s["scales"], c["fmt"])
        return {"y": _exact_rounded(s["x"], c["fmt"]) @ w.t()}
    if c["op"] == "experts":
        x = _exact_rounded(s["x"], c["fmt"])
        out = torch.zeros(s["pos"].numel(), c["N"], dtype=torch.float64, device="cuda")
        off, k = s["offsets"].tolist(), s["pos"].shape[1]
        for e in range(c["E"]):
            if off[e] == off[e + 1]:
                continue
            rows = x[s["order"][off[e]:off[e + 1]].long() // k]
            y = rows @ _exact_weight(s["codes"][e], s["scales"][e], c["fmt"]).t()
            if c["gated"]:
                y = y * torch.sigmoid(y) * (rows @ _exact_weight(s["up_codes"][e], s["up_scales"][e], c["fmt"]).t())
            out[off[e]:off[e + 1]] = y
        return {"y": out}
    if c["op"] == "route":
        ids, w = s["ids"].cpu(), s["weights"].double()
        T, k = ids.shape
        kept = sorted((e, i) for i, e in enumerate(ids.reshape(-1).tolist()) if 0 <= e < c["E"])
        pos = torch.full((T * k,), -1, dtype=torch.long)
        pos[[i for _, i in kept]] = torch.arange(len(kept))
        pos = pos.cuda()
        n = len(kept)
        xs = torch.zeros(T * k, c["H"], dtype=torch.float64, device="cuda")
        xs[:n] = s["x"].double()[torch.tensor([i // k for _, i in kept], dtype=torch.long, device="cuda")]
        y = torch.zeros(T, c["H"], dtype=torch.float64, device="cuda")
        for j in range(k):
            p = pos.view(T, k)[:, j]
            on = p >= 0
            y[on] += w[on, j, None] * s["ys"].double()[p[on]]
        return {"order": None, "pos": None, "offsets": None, "xs": xs, "y": y}
    T, k = s["pos"].shape
    dy, ys, dxs, w = s["dy"].double(), s["ys"].double(), s["dxs"].double(), s["weights"].double()
    dys, dw, dx = torch.zeros_like(ys), torch.zeros(T, k, dtype=torch.float64, device="cuda"), torch.zeros_like(dy)
    for j in range(k):
        p = s["pos"][:, j].long()
        on = p >= 0
        dys[p[on]] = w[on, j, None] * dy[on]
        dw[on, j] = torch.einsum("th,th->t", dy[on], ys[p[on]])
        dx[on] += dxs[p[on]]
    return {"dys": dys, "dw": dw, "dx": dx}
