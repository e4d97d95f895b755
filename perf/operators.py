"""Cases of the 8-bit projection steps and of the gated linear recurrence, with their plain forms.

The operators are the steps of a linear-recurrence layer whose projections run in 8 bits:
the RMSNorm with the residual's addition and an e4m3 output with scales, the quantisation of the
other operands (weights, activations), the product of two such operands, and the recurrence
h_t = a_t h_{t-1} + x_t with a gate per channel, forward and backward.
"""
import math

import torch

own = False

BLOCK = 128            # columns (and, for weights, rows) that share a scale
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # one decoding step of a few requests: the projection output added to the residual stream
        {"name": "norm_step", "op": "norm", "rows": 8, "d": 2048, "x": "bf16", "res": "fp32"},
        # the packed 5% tails of 8 hits of a 32K prefix, a wide model
        {"name": "norm_tails", "op": "norm", "rows": 13112, "d": 4096, "x": "bf16", "res": "fp32"},
        # an input projection's weight, quantised in tiles as it is loaded
        {"name": "quant_weight", "op": "quant", "rows": 6176, "cols": 2048, "x": "bf16", "tile": 128},
        # the FFN's hidden activation of a batch of tails, ragged rows
        {"name": "quant_hidden", "op": "quant", "rows": 13112, "cols": 5632, "x": "bf16", "tile": 1},
        # a decoding step's input projection: the weight is read for 8 tokens
        {"name": "proj_step", "op": "proj", "t": 8, "n": 6176, "k": 2048, "y": "bf16"},
        # a short tail and sizes that fill no tile, fp32 out (the residual stream's type)
        {"name": "proj_ragged", "op": "proj", "t": 205, "n": 1001, "k": 2000, "y": "fp32"},
        # the 5% tail of a 32K prefix through one input projection
        {"name": "proj_tail", "op": "proj", "t": 1639, "n": 6176, "k": 2048, "y": "bf16"},
        # the packed tails of 8 hits through the wide model's projection
        {"name": "proj_tails", "op": "proj", "t": 13112, "n": 12352, "k": 4096, "y": "bf16"},
        # one token of 256 requests: the states are read and written
        {"name": "rec_step", "op": "rec", "t": 256, "n_seqs": 256, "c": 4096, "x": "bf16", "g": "bf16",
         "logits": True, "h0": True, "step": True},
        # the packed tails of 64 requests of mixed lengths, zero start
        {"name": "rec_tails", "op": "rec", "t": 65536, "n_seqs": 64, "c": 4096, "x": "bf16", "g": "bf16",
         "logits": True, "h0": False, "step": False},
        # training on one long sequence, fp32 log decays
        {"name": "rec_back_long", "op": "rec_back", "t": 32768, "n_seqs": 1, "c": 2048, "x": "bf16",
         "g": "fp32", "logits": False, "h0": False, "step": False},
        # training on short packed sequences of an odd width, fp32, from given states
        {"name": "rec_back_ragged", "op": "rec_back", "t": 1639, "n_seqs": 13, "c": 1023, "x": "fp32",
         "g": "fp32", "logits": True, "h0": True, "step": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quant", "proj", "rec", "rec_back"])
    x = rng.choice(["bf16", "bf16", "fp32"])
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 13000), "d": 16 * _log(rng, 16, 256), "x": x,
                "res": rng.choice(["none", "bf16", "fp32"])}
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 13000), "cols": 16 * _log(rng, 8, 352), "x": x,
                "tile": rng.choice([1, 128])}
    if op == "proj":
        return {"op": op, "t": _log(rng, 1, 8000), "n": _log(rng, 100, 12000), "k": 16 * _log(rng, 8, 256),
                "y": rng.choice(["bf16", "bf16", "fp32"])}
    c = _log(rng, 64, 4096)
    step = op == "rec" and rng.random() < 0.3
    t = _log(rng, 1, 1024) if step else _log(rng, 16, min(65536, 2 ** 26 // c))
    return {"op": op, "t": t, "n_seqs": t if step else _log(rng, 1, min(t, 256)), "c": c, "x": x,
            "g": rng.choice(["bf16", "fp32"]), "logits": rng.random() < 0.5,
            "h0": step or rng.random() < 0.5, "step": step}


def _blocks(n):
    return -(-n // BLOCK)


def _randn(shape, seed, i, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1000 + i) & 0x7FFFFFFFFFFFFFFF)
    return torch.randn(shape, generator=g, device="cuda") * std


def _lengths(case, seed):
    """Offsets of the packed sequences: random cuts, so that some are short and a few empty."""
    t, n = case["t"], case["n_seqs"]
    if case["step"]:
        return torch.arange(n + 1, dtype=torch.int32)
    g = torch.Generator()
    g.manual_seed(seed * 1000 + 99)
    cuts = torch.randint(0, t + 1, (n - 1,), generator=g).sort().values.to(torch.int32)
    return torch.cat([torch.zeros(1, dtype=torch.int32), cuts, torch.full((1,), t, dtype=torch.int32)])


def prepare(case, seed):
    op = case["op"]
    if op == "norm":
        rows, d = case["rows"], case["d"]
        res = None if case["res"] == "none" else _randn((rows, d), seed, 2, 3.0).to(TYPES[case["res"]])
        return {"case": case, "x": _randn((rows, d), seed, 1).to(TYPES[case["x"]]), "res": res,
                "gain": 1 + _randn((d,), seed, 3, 0.1)}
    if op == "quant":
        std = 0.02 if case["tile"] > 1 else 1.0
        return {"case": case, "x": _randn((case["rows"], case["cols"]), seed, 1, std).to(TYPES[case["x"]])}
    if op == "proj":
        a, sa = _quantize(_randn((case["t"], case["k"]), seed, 1), 1)
        w, sw = _quantize(_randn((case["n"], case["k"]), seed, 2, 0.02), BLOCK)
        return {"case": case, "a": a, "sa": sa, "w": w, "sw": sw}
    t, c, n = case["t"], case["c"], case["n_seqs"]
    # gates around 0.95, as a trained gate's bias puts them: sigmoid(3 + noise), and its logarithm
    gate = _randn((t, c), seed, 1) - 3.0
    gate = (gate if case["logits"] else torch.nn.functional.logsigmoid(-gate)).to(TYPES[case["g"]])
    host = _lengths(case, seed)
    s = {"case": case, "x": _randn((t, c), seed, 2).to(TYPES[case["x"]]), "gate": gate,
         "cu": (host, host.cuda()), "h0": _randn((n, c), seed, 3) if case["h0"] else None}
    if op == "rec_back":
        # what the forward pass left, and the gradients that reach its outputs
        s["y"], _ = _recurrence(s)
        s["dh"] = _randn((n, c), seed, 5) if case["h0"] else None
        s["x"], s["dy"] = None, _randn((t, c), seed, 4).to(TYPES[case["x"]])
    return s


# ------------------------------------------------------------------ plain forms (32 bits)

def _quantize(x, tile):
    """e4m3 values and fp32 scales of x [rows, cols], one scale per tile x 128 block."""
    rows, cols = x.shape
    kb, rb = _blocks(cols), -(-rows // tile)
    full = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - cols, 0, rb * tile - rows))
    full = full.view(rb, tile, kb, BLOCK)
    scale = (full.abs().amax(dim=(1, 3)) / E4M3_MAX).clamp_min(SCALE_MIN)
    q = (full * (1.0 / scale)[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(F8)
    return q.view(rb * tile, kb * BLOCK)[:rows, :cols].contiguous(), scale


def _dequantize(q, scale, tile):
    rows, cols = q.shape
    s = scale.repeat_interleave(tile, 0)[:rows] if tile > 1 else scale
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :cols]


def _norm(s):
    r = s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()
    n = r * torch.rsqrt(r.square().mean(dim=1, keepdim=True) + 1e-6) * s["gain"]
    q, scale = _quantize(n, 1)
    return (q, scale) if s["res"] is None else (q, scale, r.to(s["res"].dtype))


def _decay(s):
    g = s["gate"].float()
    return torch.sigmoid(-g) if s["case"]["logits"] else torch.exp(g)


def _prefix(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis (a = 0 where a sequence begins), by doubling:
    pass d joins every position with the one 2^d before it, log2 of the longest sequence passes."""
    d = 1
    while d < longest:
        b = torch.cat([b[:d], torch.addcmul(b[d:], a[d:], b[:-d])])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _ends(s):
    """Per sequence the index of its first and last token, whether it holds any [n, 1], and the
    longest length. An empty one gets the first or last token of another."""
    cu = s["cu"][1].long()
    t, host = s["gate"].shape[0], s["cu"][0]
    first, last = cu[:-1], cu[1:] - 1
    return (torch.where(first < t, first, 0), torch.where(last >= 0, last, t - 1),
            (cu[1:] > cu[:-1])[:, None], int((host[1:] - host[:-1]).max()))


def _recurrence(s):
    first, last, some, longest = _ends(s)
    a, h = _decay(s), s["x"].float()
    if s["h0"] is not None:
        h = h.index_add(0, first, torch.where(some, a[first] * s["h0"], 0.0))
    h = _prefix(a.index_fill(0, first, 0.0), h, longest)
    return h.to(s["x"].dtype), torch.where(some, h[last], 0.0 if s["h0"] is None else s["h0"])


def _recurrence_backward(s):
    first, last, some, longest = _ends(s)
    a, dy, y = _decay(s), s["dy"].float(), s["y"].float()
    # G_t = dy_t + a_{t+1} G_{t+1}, run from the last token to the first
    after = torch.cat([a[1:], torch.zeros_like(a[:1])]).index_fill(0, last, 0.0)
    before = torch.cat([torch.zeros_like(y[:1]), y[:-1]]).index_fill(0, first, 0.0)
    if s["h0"] is not None:
        dy = dy.index_add(0, last, torch.where(some, s["dh"], 0.0))
        before = before.index_add(0, first, torch.where(some, s["h0"], 0.0))
    g = _prefix(after.flip(0), dy.flip(0), longest).flip(0)
    u = a * g
    dg = u * before
    if s["case"]["logits"]:
        dg = -dg * torch.sigmoid(s["gate"].float())
    dx = g.to(s["dy"].dtype), dg.to(s["gate"].dtype)
    return dx if s["h0"] is None else (*dx, torch.where(some, u[first], s["dh"]))


def run(s):
    op = s["case"]["op"]
    if own:
        import linear_attention_state_zero_b200 as tr
        if op == "norm":
            out = tr.rmsnorm_fp8(s["x"], s["gain"], residual=s["res"])
            return out[:2] if s["res"] is None else out
        if op == "quant":
            return tr.quantize_fp8(s["x"], block_rows=s["case"]["tile"])
        if op == "proj":
            return tr.projection_fp8(s["a"], s["sa"], s["w"], s["sw"], out_dtype=TYPES[s["case"]["y"]])
        if op == "rec":
            return tr.linear_recurrence(s["x"], s["gate"], s["cu"], h0=s["h0"],
                                        gate_logits=s["case"]["logits"])
        out = tr.linear_recurrence_backward(s["dy"], s["gate"], s["y"], s["cu"], h0=s["h0"], dh_final=s["dh"],
                                            gate_logits=s["case"]["logits"])
        return out[:2] if s["h0"] is None else out
    if op == "norm":
        return _norm(s)
    if op == "quant":
        return _quantize(s["x"], s["case"]["tile"])
    if op == "proj":
        y = _dequantize(s["a"], s["sa"], 1) @ _dequantize(s["w"], s["sw"], BLOCK).t()
        return y.to(TYPES[s["case"]["y"]])
    return _recurrence(s) if op == "rec" else _recurrence_backward(s)


def work(case):
    op = case["op"]
    if op == "norm":
        rows, d, r = case["rows"], case["d"], SIZE.get(case["res"], 0)
        return {"bytes": rows * (d * (SIZE[case["x"]] + 2 * r + 1) + 4 * _blocks(d)) + 4 * d, "flops": 6 * rows * d}
    if op == "quant":
        rows, cols = case["rows"], case["cols"]
        return {"bytes": rows * cols * (SIZE[case["x"]] + 1) + 4 * -(-rows // case["tile"]) * _blocks(cols),
                "flops": 2 * rows * cols}
    if op == "proj":
        t, n, k = case["t"], case["n"], case["k"]
        return {"bytes": (t + n) * k + 4 * _blocks(k) * (t + _blocks(n)) + t * n * SIZE[case["y"]],
                "flops": 2 * t * n * k}
    tc, nc = case["t"] * case["c"], case["n_seqs"] * case["c"]
    x, g = SIZE[case["x"]], SIZE[case["g"]]
    if op == "rec":
        return {"bytes": tc * (2 * x + g) + 4 * nc * (2 if case["h0"] else 1), "flops": 2 * tc}
    return {"bytes": tc * (3 * x + 2 * g) + (4 * nc * 3 if case["h0"] else 0), "flops": 4 * tc}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_quantized(v, tile):
    """Scales of v (64 bits) block by block, and the e4m3 values nearest to v / scale."""
    rows, cols = v.shape
    out = torch.empty_like(v)
    scales = torch.empty((-(-rows // tile), _blocks(cols)), dtype=torch.float64, device=v.device)
    for b in range(scales.shape[1]):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        top = part.abs().max(dim=1).values
        if tile > 1:
            top = torch.stack([p.max() for p in top.split(tile)])
        scales[:, b] = torch.maximum(top / 448, torch.full_like(top, 2.0 ** -126))
        each = scales[:, b] if tile == 1 else scales[:, b].repeat_interleave(tile)[:rows]
        z = part / each[:, None]
        # e4m3 spacing: 2^(e-3) in [2^e, 2^(e+1)), at least 2^-9; round half to even
        step = torch.exp2(torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6))) - 3)
        out[:, b * BLOCK:(b + 1) * BLOCK] = (torch.round(z / step) * step).clamp(-448, 448)
    return out, scales


def _exact_walk(a, b, lo, hi, start, out):
    """h = a h + b from `start` over tokens lo, lo +- 1, ..., hi; each h is kept in out."""
    h = start
    for t in range(lo, hi + 1) if lo <= hi else range(lo, hi - 1, -1):
        h = torch.addcmul(b[t], a[t], h, out=out[t])
    return h


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "quant"):
        v = s["x"].double()
        if op == "quant":
            return _exact_quantized(v, case["tile"])
        if s["res"] is not None:
            v = v + s["res"].double()
        q = _exact_quantized(v / (v.pow(2).sum(1, keepdim=True) / case["d"] + 1e-6).sqrt() * s["gain"].double(), 1)
        return q if s["res"] is None else (*q, v)
    if op == "proj":
        a = torch.empty(s["a"].shape, dtype=torch.float64, device="cuda")
        w = torch.empty(s["w"].shape, dtype=torch.float64, device="cuda")
        for b in range(_blocks(case["k"])):
            cols = slice(b * BLOCK, (b + 1) * BLOCK)
            a[:, cols] = s["a"][:, cols].double() * s["sa"][:, b:b + 1].double()
            w[:, cols] = s["w"][:, cols].double() * s["sw"][:, b].double().repeat_interleave(BLOCK)[:case["n"], None]
        return torch.matmul(a, w.T)
    g = s["gate"].double()
    a = 1 / (1 + g.exp()) if case["logits"] else g.exp()
    cu = s["cu"][0].tolist()
    zero = torch.zeros(case["c"], dtype=torch.float64, device="cuda")
    h0 = [zero if s["h0"] is None else s["h0"][i].double() for i in range(case["n_seqs"])]
    out, ends = torch.empty_like(a), []
    if op == "rec":
        x = s["x"].double()
        for i, (lo, hi) in enumerate(zip(cu[:-1], cu[1:])):
            ends.append(_exact_walk(a, x, lo, hi - 1, h0[i], out) if hi > lo else h0[i])
        return out, torch.stack(ends)
    dy, y, u, before = s["dy"].double(), s["y"].double(), torch.empty_like(a), torch.empty_like(a)
    ady = a * dy
    # u_t = a_t G_t is what reaches h_{t-1}: u_t = a_t u_{t+1} + a_t dy_t, and G_t = dy_t + u_{t+1}
    for i, (lo, hi) in enumerate(zip(cu[:-1], cu[1:])):
        dh = zero if s["dh"] is None else s["dh"][i].double()
        if hi > lo:
            out[hi - 1] = dh
            before[lo], before[lo + 1:hi] = h0[i], y[lo:hi - 1]
            _exact_walk(a, ady, hi - 1, lo, dh, u)
            out[lo:hi - 1] = u[lo + 1:hi]
        ends.append(u[lo].clone() if hi > lo else dh)
    dg = u * before
    if case["logits"]:
        dg = -dg / (1 + (-g).exp())
    return (dy + out, dg) if s["h0"] is None else (dy + out, dg, torch.stack(ends))
