"""Measured cases of the FP8 linear layer with a scale per block of 128, the products grouped by
expert, the routing around them, and the mixture-of-experts MLP that runs them together.

Operators, each in a plain form (elementary torch operations in 32 bits) and as the framework's
kernels:

* linear: bf16 rows quantised to E4M3 with one fp32 scale per 128 elements along K (scale =
  amax / 448, code = E4M3(448 x / amax)), the product with E4M3 weights that have one fp32 scale per
  128 x 128 block, bias, bf16 out;
* grouped: rows sorted by expert, expert e owning rows [offsets[e], offsets[e + 1]), each multiplied
  with its expert's weights, in that format or in MXFP8 (E4M3, one E8M0 scale per 32 along K); the
  rows are given in order, or picked from a token tensor by an index;
* route: the k largest logits of each token (ties to the lowest expert), their softmax or sigmoid
  weights, the rows sorted by expert; then, once the experts' outputs exist, each token's weighted sum;

and "experts", the MLP block that runs them together: route, gather and quantise, gate and up
products, silu(gate) * up, down products, weighted sum.
"""

import math
import random

import torch

own = False

OUTLIERS = 1e-3       # share of x that is 100 times larger
ZERO_BLOCKS = 1e-2    # share of 32-element blocks of x that are all zero
FORMATS = ["mxfp8", "fp8_128"]


def listed():
    return [
        # one token through a projection of a block-scaled checkpoint: the smallest serving call
        {"name": "lin_decode_1", "op": "linear", "b": 1, "m": 1, "n": 4096, "k": 4096, "x": "bf16", "bias": True},
        # a decode batch through the MLP's first projection
        {"name": "lin_decode_48", "op": "linear", "b": 1, "m": 48, "n": 14336, "k": 4096, "x": "bf16", "bias": False},
        # a chunk of prompt with ragged rows, columns and K (a last block of 16 along K, of 104 along N)
        {"name": "lin_ragged", "op": "linear", "b": 1, "m": 333, "n": 1000, "k": 4112, "x": "bf16", "bias": True},
        # prefill, MLP up
        {"name": "lin_prefill_up", "op": "linear", "b": 1, "m": 4096, "n": 14336, "k": 4096, "x": "bf16", "bias": False},
        # one token's eight experts, the activation handed over quantised
        {"name": "grp_one_token_128", "op": "grouped", "fmt": "fp8_128", "e": 64, "active": 8, "rows": 8, "n": 2048,
         "k": 4096, "x": "codes", "gather": False},
        # a decode batch of 16 tokens, eight experts each, rows picked from the token tensor
        {"name": "grp_decode_mx", "op": "grouped", "fmt": "mxfp8", "e": 64, "active": 54, "rows": 128, "n": 2048,
         "k": 4096, "x": "bf16", "gather": True},
        # prefill, few wide experts with very uneven shares, three of them without a row
        {"name": "grp_prefill_mx", "op": "grouped", "fmt": "mxfp8", "e": 16, "active": 13, "rows": 16384, "n": 4096,
         "k": 4096, "x": "bf16", "gather": True},
        # prefill, more and smaller experts, the down projection of a block-scaled checkpoint
        {"name": "grp_prefill_128", "op": "grouped", "fmt": "fp8_128", "e": 64, "active": 61, "rows": 24576, "n": 4096,
         "k": 2048, "x": "codes", "gather": False},
        # the router of a decode batch, and of a long prompt with many experts
        {"name": "route_decode", "op": "route", "t": 16, "e": 64, "k": 8, "n": 4096, "logits": "fp32",
         "scoring": "softmax", "renormalize": True},
        {"name": "route_prefill", "op": "route", "t": 8192, "e": 256, "k": 8, "n": 4096, "logits": "bf16",
         "scoring": "sigmoid", "renormalize": True},
        # the whole block: a decoding sequence, and a prompt
        {"name": "experts_decode_mx", "op": "experts", "fmt": "mxfp8", "t": 4, "e": 64, "k": 8, "h": 2048, "f": 1024},
        {"name": "experts_prefill_128", "op": "experts", "fmt": "fp8_128", "t": 2048, "e": 64, "k": 8, "h": 2048,
         "f": 1024},
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], even over the logarithm."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))) / step) * step
    return max(-(-lo // step) * step, min(hi // step * step, v))


def draw(rng):
    op = rng.choice(["linear", "linear", "grouped", "grouped", "route", "experts"])
    fmt = rng.choice(FORMATS)
    k_step = 128 if fmt == "mxfp8" else 16
    while True:
        if op == "linear":
            b = rng.choice([1, 1, 1, rng.randint(2, 16)])
            c = {"op": op, "b": b, "m": _log_int(rng, 1, 8192 if b == 1 else 512),
                 "n": _log_int(rng, 256, 14336 if b == 1 else 1024, 8), "k": _log_int(rng, 512, 14336, 16),
                 "x": rng.choice(["bf16", "bf16", "codes"]), "bias": rng.random() < 0.5}
            if b * c["m"] * c["n"] * c["k"] <= 4096 * 14336 * 4096:
                return c
        elif op == "grouped":
            e = _log_int(rng, 2, 256)
            rows = _log_int(rng, 1, 24576)
            gather = rng.random() < 0.5
            c = {"op": op, "fmt": fmt, "e": e, "active": rng.randint(max(1, min(e, rows) // 2), min(e, rows)), "rows": rows,
                 "n": _log_int(rng, 256, 4096, 8), "k": _log_int(rng, 512, 4096, k_step),
                 "x": "bf16" if gather else rng.choice(["bf16", "codes"]), "gather": gather}
            if e * c["n"] * c["k"] <= 64 * 2048 * 4096 and rows * c["n"] * c["k"] <= 16384 * 4096 * 4096:
                return c
        elif op == "route":
            e = _log_int(rng, 8, 512)
            k = rng.randint(1, min(16, e))
            c = {"op": op, "t": _log_int(rng, 1, 16384), "e": e, "k": k, "n": _log_int(rng, 512, 8192, 8),
                 "logits": rng.choice(["fp32", "bf16"]), "scoring": rng.choice(["softmax", "sigmoid"]),
                 "renormalize": rng.random() < 0.5}
            if c["t"] * k * c["n"] <= 8192 * 8 * 4096:
                return c
        else:
            e = _log_int(rng, 8, 128)
            c = {"op": op, "fmt": fmt, "t": _log_int(rng, 1, 2048), "e": e, "k": rng.randint(1, 8),
                 "h": _log_int(rng, 512, 2048, 128), "f": _log_int(rng, 256, 1024, 128)}
            if c["e"] * c["h"] * c["f"] <= 64 * 2048 * 1024:
                return c


# ------------------------------------------------------------------ plain quantisation (32 bits)
def _pow2(e):
    """2 ** e in fp32 for whole e in [-127, 127], from its bit pattern."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _e4m3(t):
    return t.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _blocks128(y):
    """[..., K] as [..., ceil(K / 128), 128], the last block filled up with zeros."""
    k = y.shape[-1]
    if k % 128:
        y = torch.nn.functional.pad(y, (0, -k % 128))
    return y.unflatten(-1, (-1, 128))


def _quantise(y, fmt):
    """fp32 y [..., K] -> (E4M3 codes, scale values fp32 per block along K)."""
    k = y.shape[-1]
    if fmt == "mxfp8":
        yb = y.unflatten(-1, (-1, 32))
        top = yb.abs().amax(-1, keepdim=True)
        e = (torch.frexp(top).exponent - 9).clamp(-127, 127)
        e = torch.where(top > 0, e, -127)
        return _e4m3(yb * _pow2(-e)).flatten(-2), _pow2(e).squeeze(-1)
    yb = _blocks128(y)
    top = yb.abs().amax(-1, keepdim=True)
    # 448 y / top: the product with 7 / 8 is exact for y of 16 bits, so ties are met as ties
    q = _e4m3(torch.where(top > 0, yb * 0.875 / top, 0.0) * 512.0)
    return q.flatten(-2)[..., :k].contiguous(), (top / 448.0).squeeze(-1)


def _spread(s, n, block):
    """One scale per block as one per element, of ``n`` elements."""
    return s.repeat_interleave(block, -1)[..., :n]


def _dequantise(q, s, fmt):
    return q.float() * _spread(s, q.shape[-1], 32 if fmt == "mxfp8" else 128)


def _fake(y, fmt):
    return _dequantise(*_quantise(y, fmt), fmt)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _acts(gen, *shape):
    """bf16 activations: normal, a few outliers, a few all-zero blocks of 32."""
    k = shape[-1]
    x = torch.randn(shape, device="cuda", generator=gen)
    x = torch.where(torch.rand(shape, device="cuda", generator=gen) < OUTLIERS, x * 100.0, x)
    dead = torch.rand((*shape[:-1], -(-k // 32)), device="cuda", generator=gen) < ZERO_BLOCKS
    return x.masked_fill_(_spread(dead, k, 32), 0.0).to(torch.bfloat16)


def _weights(gen, fmt, *shape):
    """Quantised weights as a checkpoint holds them: E4M3 codes [..., N, K] and scales, E8M0 bytes
    [..., N, K / 32] or fp32 [..., ceil(N / 128), ceil(K / 128)]."""
    if len(shape) == 3:  # expert by expert: the fp32 draws of all of them would be large
        each = [_weights(gen, fmt, *shape[1:]) for _ in range(shape[0])]
        return {"q": torch.stack([w["q"] for w in each]), "s": torch.stack([w["s"] for w in each])}
    w = torch.randn(shape, device="cuda", generator=gen) * 0.02
    if fmt == "mxfp8":
        q, s = _quantise(w, fmt)
        return {"q": q.view(torch.uint8), "s": s.to(torch.float8_e8m0fnu).view(torch.uint8)}
    n, k = shape
    s = _blocks128(_blocks128(w.abs()).amax(-1).mT).amax(-1).mT / 448.0
    return {"q": _e4m3(w / _block_scales(s, n, k)).view(torch.uint8), "s": s.contiguous()}


def _block_scales(s, n, k):
    """Scales of 128 x 128 blocks as one per element of [n, k]."""
    return _spread(_spread(s.mT, n, 128).mT, k, 128)


def _weight_values(w, fmt):
    """fp32 weights of the plain form."""
    v = w["q"].view(torch.float8_e4m3fn).float()
    if fmt == "mxfp8":
        return v.mul_(_spread(_pow2(w["s"].int() - 127), v.shape[-1], 32))
    return v.mul_(_block_scales(w["s"], *v.shape[-2:]))


def _laid_out(w, fmt):
    """The weights as a program keeps them for its calls: processed once for the framework's
    kernels, or plain fp32."""
    if not own:
        return _weight_values(w, fmt)
    from mxfp8_block_scaled_02_gb300 import ops
    return ops.process_weights(w["q"], w["s"]) if fmt == "mxfp8" else ops.process_weights_fp8_128(w["q"], w["s"])


def _counts(case, seed):
    """Rows of each expert: ``active`` of them have at least one, the others none, the shares spread as
    a trained router's are (log-normal)."""
    rng = random.Random(seed * 7919 + case["rows"])
    n = [0] * case["e"]
    busy = rng.sample(range(case["e"]), case["active"])
    for e in busy:
        n[e] = 1
    for e in rng.choices(busy, [math.exp(0.8 * rng.gauss(0, 1)) for _ in busy], k=case["rows"] - case["active"]):
        n[e] += 1
    return n


def _offsets(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return torch.tensor(at, dtype=torch.int32).cuda()


def _codes(x, fmt):
    """Codes and scales that the step before hands over."""
    q, s = _quantise(x.float(), fmt)
    return q.view(torch.uint8), s.to(torch.float8_e8m0fnu).view(torch.uint8) if fmt == "mxfp8" else s


def _raw(case, seed):
    """Everything a user has before the call, in the types they have it in."""
    gen, op = _gen(seed), case["op"]
    if op == "route":
        t, e = case["t"], case["e"]
        logits = 2.0 * torch.randn(t, e, device="cuda", generator=gen)
        y = torch.randn(t * case["k"], case["n"], device="cuda", generator=gen)
        return {"logits": logits.to(torch.bfloat16 if case["logits"] == "bf16" else torch.float32),
                "y": y.to(torch.bfloat16)}
    if op == "experts":
        t, e, h, f, fmt = case["t"], case["e"], case["h"], case["f"], case["fmt"]
        return {"x": _acts(gen, t, h), "logits": 2.0 * torch.randn(t, e, device="cuda", generator=gen),
                "add": torch.randn(t, h, device="cuda", generator=gen).to(torch.bfloat16),
                "w1": _weights(gen, fmt, e, 2 * f, h), "w2": _weights(gen, fmt, e, h, f)}
    if op == "grouped":
        fmt, rows, k = case["fmt"], case["rows"], case["k"]
        counts = _counts(case, seed)
        r = {"counts": counts, "offsets": _offsets(counts), "rows": None, "s": None,
             "w1": _weights(gen, fmt, case["e"], case["n"], k)}
        if case["gather"]:
            tokens = -(-rows // 8)
            r["x"] = _acts(gen, tokens, k)
            r["rows"] = torch.randint(tokens, (rows,), device="cuda", generator=gen, dtype=torch.int32)
        else:
            r["x"] = _acts(gen, rows, k)
            if case["x"] == "codes":
                r["x"], r["s"] = _codes(r["x"], fmt)
        return r
    lead = (case["b"],) if case["b"] > 1 else ()
    r = {"x": _acts(gen, *lead, case["m"], case["k"]), "s": None,
         "w1": _weights(gen, "fp8_128", *lead, case["n"], case["k"]),
         "bias": (0.1 * torch.randn(case["n"], device="cuda", generator=gen)).to(torch.bfloat16) if case["bias"] else None}
    if case["x"] == "codes":
        r["x"], r["s"] = _codes(r["x"], "fp8_128")
    return r


def prepare(case, seed):
    st = _raw(case, seed)
    st["case"] = case
    for name in ("w1", "w2"):
        if name in st:
            st[name] = _laid_out(st[name], case.get("fmt", "fp8_128"))
    if own and case["op"] == "experts":
        from mxfp8_block_scaled_02_gb300 import mlp
        st["mlp"] = mlp.ExpertMLP(st["w1"], st["w2"], case["k"], renormalize=True)
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from mxfp8_block_scaled_02_gb300 import ops
    case = st["case"]
    if case["op"] == "linear":
        return ops.linear_fp8_128(st["x"], st["w1"], st["bias"], st["s"])
    if case["op"] == "grouped":
        return ops.grouped_linear(st["x"], st["w1"], st["offsets"], st["s"], rows=st["rows"])
    if case["op"] == "experts":
        return st["mlp"](st["x"], st["logits"], add=st["add"])
    r = ops.route(st["logits"], case["k"], scoring=case["scoring"], renormalize=case["renormalize"])
    return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "rows": r.rows, "positions": r.positions,
            "out": ops.combine(st["y"], r)}


def _route(logits, k, scoring, renormalize):
    """Experts, weights and the sorted order of their rows; every logit is finite here."""
    t, e = logits.shape
    z = logits.float()
    best, ids = torch.sort(z, dim=-1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    if scoring == "softmax":
        top = z.amax(-1, keepdim=True)
        w = torch.exp(best - top) / torch.exp(z - top).sum(-1, keepdim=True)
    else:
        w = 1.0 / (1.0 + torch.exp(-best))
    if renormalize:
        w = w / w.sum(-1, keepdim=True)
    order = torch.sort(ids.flatten(), stable=True).indices  # by expert, then by token
    positions = torch.empty_like(order)
    positions[order] = torch.arange(t * k, device=order.device)
    ends = torch.cumsum((ids.reshape(-1, 1) == torch.arange(e, device=ids.device)).sum(0), 0)
    i32 = torch.int32
    return {"ids": ids.to(i32), "weights": w, "offsets": torch.nn.functional.pad(ends, (1, 0)).to(i32),
            "rows": (order // k).to(i32), "positions": positions.reshape(t, k).to(i32)}


def _combine(y, r, add=None):
    out = (y.float()[r["positions"].long()] * r["weights"].unsqueeze(-1)).sum(1)
    return (out if add is None else out + add.float()).to(torch.bfloat16)


def _grouped(x, w, counts):
    """fp32 rows, one product an expert, rounded to bf16."""
    out = torch.empty(x.shape[0], w.shape[1], dtype=torch.bfloat16, device=x.device)
    at = 0
    for e, n in enumerate(counts):
        if n:
            out[at:at + n] = (x[at:at + n] @ w[e].T).to(torch.bfloat16)
        at += n
    return out


def _silu_mul(gate_up):
    gate, up = gate_up.float().chunk(2, -1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _scale_values(s, fmt):
    return _pow2(s.int() - 127) if fmt == "mxfp8" else s


def _values(st, fmt):
    """fp32 values of x: handed over quantised, or quantised here."""
    if st["s"] is None:
        return _fake(st["x"].float(), fmt)
    return _dequantise(st["x"].view(torch.float8_e4m3fn), _scale_values(st["s"], fmt), fmt)


def _run_plain(st):
    case, fmt = st["case"], st["case"].get("fmt", "fp8_128")
    if case["op"] == "linear":
        out = _values(st, fmt) @ st["w1"].mT
        return (out if st["bias"] is None else out + st["bias"].float()).to(torch.bfloat16)
    if case["op"] == "grouped":
        x = _values(st, fmt)
        return _grouped(x if st["rows"] is None else x[st["rows"].long()], st["w1"], st["counts"])
    if case["op"] == "experts":
        r = _route(st["logits"], case["k"], "softmax", True)
        counts = r["offsets"].diff().tolist()  # an eager program asks the device how many rows each expert has
        h = _grouped(_fake(st["x"].float(), fmt)[r["rows"].long()], st["w1"], counts)
        y = _grouped(_fake(_silu_mul(h), fmt), st["w2"], counts)
        return _combine(y, r, st["add"])
    r = _route(st["logits"], case["k"], case["scoring"], case["renormalize"])
    r["out"] = _combine(st["y"], r)
    return r


# ------------------------------------------------------------------ what a pass cannot do without
def _weight_bytes(n, k, fmt):
    return n * k + (n * k / 32 if fmt == "mxfp8" else 4 * -(-n // 128) * -(-k // 128))


def _x_bytes(rows, k, fmt, kind):
    if kind == "bf16":
        return 2 * rows * k
    return rows * k + (rows * k / 32 if fmt == "mxfp8" else 4 * rows * -(-k // 128))


def work(case):
    op, fmt = case["op"], case.get("fmt", "fp8_128")
    if op == "linear":
        b, m, n, k = case["b"], case["m"], case["n"], case["k"]
        return {"bytes": _x_bytes(b * m, k, fmt, case["x"]) + b * _weight_bytes(n, k, fmt) + 2 * b * m * n
                + (2 * n if case["bias"] else 0), "flops": 2 * b * m * n * k}
    if op == "grouped":
        rows, n, k = case["rows"], case["n"], case["k"]
        given = -(-rows // 8) if case["gather"] else rows
        return {"bytes": _x_bytes(given, k, fmt, case["x"]) + (4 * rows if case["gather"] else 0) + 4 * (case["e"] + 1)
                + case["active"] * _weight_bytes(n, k, fmt) + 2 * rows * n, "flops": 2 * rows * n * k}
    t, e, k = case["t"], case["e"], case["k"]
    if op == "route":
        n = case["n"]
        return {"bytes": t * e * (2 if case["logits"] == "bf16" else 4) + t * k * 16 + 4 * (e + 1) + 2 * n * t * (k + 1),
                "flops": 4 * t * e + 2 * t * k * n}
    h, f = case["h"], case["f"]
    active = e * (1 - (1 - k / e) ** t)  # experts that at least one of the tokens chose
    return {"bytes": t * h * 6 + 4 * t * e + active * (_weight_bytes(2 * f, h, fmt) + _weight_bytes(h, f, fmt)),
            "flops": 2 * t * k * 3 * f * h}


# ------------------------------------------------------------------ the definitions in 64 bits
def _unit64(e):
    """2 ** e in 64 bits for whole e, from its bit pattern (ldexp is an ulp off on the GPU)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round64(a):
    """a to the nearest E4M3 value (three fraction bits, smallest normal 2^-6, largest 448), ties to even."""
    e = (torch.frexp(a.abs()).exponent - 1).clamp(min=-6)
    ulp = _unit64(e - 3)
    return (torch.round(a / ulp) * ulp).clamp(-448.0, 448.0)


def _fake64(y, fmt):
    """y quantised and back, in 64 bits."""
    k, n = y.shape[-1], 32 if fmt == "mxfp8" else 128
    full = torch.zeros(*y.shape[:-1], -(-k // n) * n, dtype=torch.float64, device=y.device)
    full[..., :k] = y
    yb = full.view(*y.shape[:-1], -1, n)
    top = yb.abs().amax(-1, keepdim=True)
    if fmt == "mxfp8":
        e = torch.where(top > 0, torch.frexp(top).exponent - 9, -127).clamp(-127, 127)
        unit = _unit64(e)
        z = _round64(yb / unit) * unit
    else:
        z = _round64(yb * 448 / torch.where(top > 0, top, 1.0)) * (top / 448)
    return z.reshape(full.shape)[..., :k]


def _weights64(q, s, fmt):
    """64-bit values of one weight matrix [N, K]."""
    v = q.view(torch.float8_e4m3fn).double()
    n, k = v.shape
    if fmt == "mxfp8":
        return (v.view(n, -1, 32) * _unit64(s.int() - 127).unsqueeze(-1)).view(n, k)
    at_n = torch.arange(n, device=v.device) // 128
    at_k = torch.arange(k, device=v.device) // 128
    return v * s.double()[at_n][:, at_k]


def _grouped64(x, w, counts, fmt):
    parts, at = [], 0
    for e, n in enumerate(counts):
        parts.append(x[at:at + n] @ _weights64(w["q"][e], w["s"][e], fmt).T)
        at += n
    return torch.cat(parts)


def _route64(logits, k, scoring, renormalize):
    z = logits.double()
    t, e = z.shape
    # the k largest one after the other, the lowest index among equals
    left, ids = z.clone(), []
    for _ in range(k):
        at = (left == left.amax(-1, keepdim=True)).to(torch.int8).argmax(-1, keepdim=True)
        ids.append(at)
        left.scatter_(1, at, -math.inf)
    ids = torch.cat(ids, 1)
    p = torch.softmax(z, -1) if scoring == "softmax" else torch.sigmoid(z)
    w = p.gather(1, ids)
    if renormalize:
        w = w / w.sum(-1, keepdim=True)
    chosen = torch.zeros(t, e, dtype=torch.int64, device=z.device).scatter_(1, ids, 1)
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=z.device)
    offsets[1:] = chosen.sum(0).cumsum(0)
    positions = (offsets[:-1] + chosen.cumsum(0) - chosen).gather(1, ids)
    rows = torch.empty(t * k, dtype=torch.int64, device=z.device)
    rows[positions.flatten()] = torch.arange(t, device=z.device).repeat_interleave(k)
    return {"ids": ids, "weights": w, "offsets": offsets, "rows": rows, "positions": positions}


def _combine64(y, r):
    out = torch.zeros(r["positions"].shape[0], y.shape[1], dtype=torch.float64, device=y.device)
    for j in range(r["positions"].shape[1]):
        out += y[r["positions"][:, j]].double() * r["weights"][:, j:j + 1]
    return out


def exact(case, seed):
    st, op, fmt = _raw(case, seed), case["op"], case.get("fmt", "fp8_128")
    if op == "route":
        r = _route64(st["logits"], case["k"], case["scoring"], case["renormalize"])
        return {**r, "out": _combine64(st["y"], r)}
    if op == "experts":
        # each operator's output is held in its own type between the steps
        r = _route64(st["logits"], case["k"], "softmax", True)
        counts = r["offsets"].diff().tolist()
        h = _grouped64(_fake64(st["x"].double(), fmt)[r["rows"]], st["w1"], counts, fmt).to(torch.bfloat16).double()
        f = h.shape[-1] // 2
        y = _grouped64(_fake64(h[:, :f] * torch.sigmoid(h[:, :f]) * h[:, f:], fmt), st["w2"], counts, fmt)
        return _combine64(y.to(torch.bfloat16), r) + st["add"].double()
    if st["s"] is None:
        x = _fake64(st["x"].double(), fmt)
    else:
        s = st["s"]
        unit = _unit64(s.int() - 127) if fmt == "mxfp8" else s.double()
        x = st["x"].view(torch.float8_e4m3fn).double()
        x = x * unit.repeat_interleave(32 if fmt == "mxfp8" else 128, -1)[..., :x.shape[-1]]
    if op == "grouped":
        return _grouped64(x if st["rows"] is None else x[st["rows"].long()], st["w1"], st["counts"], fmt)
    if case["b"] == 1:
        out = x @ _weights64(st["w1"]["q"], st["w1"]["s"], fmt).T
    else:
        out = torch.stack([x[i] @ _weights64(st["w1"]["q"][i], st["w1"]["s"][i], fmt).T for i in range(case["b"])])
    return out if st["bias"] is None else out + st["bias"].double()
