"""Measured cases of the 4-bit linear layer and of the steps on either side of it.

Four operators, each in a plain form (elementary torch operations in 32 bits) and as the
framework's kernels:

* quantise: bf16 rows to MXFP4 (E2M1 elements, one E8M0 scale per 32) or NVFP4 (E2M1 elements,
  one E4M3 scale per 16, one fp32 scale per tensor), and back to one E4M3 value per element;
* linear: that quantisation of x, the block-scaled product with 4-bit weights, bias, bf16 out;
* norm: residual addition, root-mean-square norm, output quantised to MXFP8 / MXFP4 / NVFP4;
* act: silu(gate) * up of a merged projection, output quantised the same ways;

and "mlp", the gated MLP block that runs them together.  Elements held in 4 or 8 bits are returned
as the values they stand for (float8_e4m3fn holds every E2M1 value), scales as float8 too.
"""

import math

import torch

own = False

OUTLIERS = 1e-3       # share of x that is 100 times larger
ZERO_BLOCKS = 1e-2    # share of 32-element blocks of x that are all zero
EPS = 1e-6
BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}


def listed():
    return [
        # 4-bit weights made when a checkpoint is loaded: the largest layer of the benchmark
        {"name": "quant_load_mx", "op": "quant", "fmt": "mxfp4", "m": 14336, "k": 4096},
        # one token through a projection: the smallest serving call
        {"name": "lin_decode_1_mx", "op": "linear", "fmt": "mxfp4", "b": 1, "m": 1, "n": 4096, "k": 4096,
         "x": "bf16", "bias": True},
        # a decode batch through the MLP's first projection
        {"name": "lin_decode_48_nv", "op": "linear", "fmt": "nvfp4", "b": 1, "m": 48, "n": 14336, "k": 4096,
         "x": "bf16", "bias": False},
        # prefill, MLP up
        {"name": "lin_prefill_up_mx", "op": "linear", "fmt": "mxfp4", "b": 1, "m": 4096, "n": 14336, "k": 4096,
         "x": "bf16", "bias": False},
        # prefill, MLP down, x handed over in 4 bits by the step before
        {"name": "lin_prefill_down_nv", "op": "linear", "fmt": "nvfp4", "b": 1, "m": 8192, "n": 4096, "k": 14336,
         "x": "codes", "bias": False},
        # a chunk of prompt with ragged rows, columns and K (not whole tiles)
        {"name": "lin_ragged_mx", "op": "linear", "fmt": "mxfp4", "b": 1, "m": 333, "n": 1000, "k": 4128,
         "x": "bf16", "bias": True},
        # independent products in one call (bmm)
        {"name": "lin_bmm_nv", "op": "linear", "fmt": "nvfp4", "b": 16, "m": 512, "n": 512, "k": 7168,
         "x": "bf16", "bias": False},
        # norm before a projection: a few decoding sequences, and a long prompt
        {"name": "norm_decode_mx8", "op": "norm", "fmt": "mxfp8", "m": 4, "k": 4096, "residual": "bf16"},
        {"name": "norm_prefill_mx8", "op": "norm", "fmt": "mxfp8", "m": 8192, "k": 4096, "residual": "bf16"},
        # gated activation between the MLP's projections: decode batch, and prefill
        {"name": "act_decode_mx4", "op": "act", "fmt": "mxfp4", "m": 16, "k": 14336},
        {"name": "act_prefill_mx8", "op": "act", "fmt": "mxfp8", "m": 4096, "k": 14336},
        # the whole block on a prompt chunk: norm, gate and up projection, activation, down projection
        {"name": "mlp_512_mx4", "op": "mlp", "fmt": "mxfp4", "m": 512, "k": 4096, "f": 14336},
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    v = max(lo, min(hi, int(v / step) * step))
    return v + step if v in (1536, 3072) else v


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "linear", "norm", "act", "mlp"])
    fp4 = rng.choice(["mxfp4", "nvfp4"])
    any_fmt = rng.choice(["mxfp8", "mxfp4", "nvfp4"])
    if op == "quant":
        return {"op": op, "fmt": fp4, "m": _log_int(rng, 1, 14336), "k": _log_int(rng, 512, 4096, 32)}
    if op == "norm":
        return {"op": op, "fmt": any_fmt, "m": _log_int(rng, 1, 8192), "k": _log_int(rng, 512, 4096, 32),
                "residual": rng.choice(["bf16", "fp32", "none"])}
    if op == "act":
        return {"op": op, "fmt": any_fmt, "m": _log_int(rng, 1, 4096), "k": _log_int(rng, 512, 14336, 32)}
    if op == "mlp":
        return {"op": op, "fmt": any_fmt, "m": _log_int(rng, 1, 512), "k": _log_int(rng, 512, 4096, 128),
                "f": _log_int(rng, 1024, 14336, 128)}
    b = rng.choice([1, 1, 1, 1, rng.randint(2, 16)])
    top_n = 14336 if b == 1 else 512
    while True:
        c = {"op": op, "fmt": fp4, "b": b, "m": _log_int(rng, 1, 8192 if b == 1 else 512),
             "n": _log_int(rng, 256, top_n, 8), "k": _log_int(rng, 512, 14336 if b == 1 else 7168, 32),
             "x": rng.choice(["bf16", "bf16", "codes"]), "bias": rng.random() < 0.5}
        if c["b"] * c["m"] * c["n"] * c["k"] <= 8192 * 4096 * 14336:
            return c


# ------------------------------------------------------------------ plain quantisation (32 bits)
def _blocks(y, fmt):
    return y.reshape(*y.shape[:-1], y.shape[-1] // BLOCK[fmt], BLOCK[fmt])


def _e2m1(a):
    """The nearest E2M1 value (0, .5, 1, 1.5, 2, 3, 4, 6), ties to even, saturating."""
    m = a.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return torch.copysign((torch.round(m / step) * step).clamp_(max=6.0), a)


def _pow2(e):
    """2 ** e in fp32 for whole e in [-127, 127], from its bit pattern."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantise(y, fmt, g):
    """fp32 y -> (element values fp32, scale values fp32, scale as its float8 type), per block along K."""
    yb = _blocks(y, fmt)
    amax = yb.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        s8 = (amax / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        s = s8.float()
        inv = torch.where(s > 0, 1.0 / (s * g), 0.0)
        v = _e2m1(yb * inv)
        return v.reshape(y.shape), s, s8.squeeze(-1)
    emax = 8 if fmt == "mxfp8" else 2
    e = (torch.frexp(amax).exponent - 1 - emax).clamp(-127, 127)
    e = torch.where(amax > 0, e, -127)
    t = yb * _pow2(-e)
    v = t.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float() if fmt == "mxfp8" else _e2m1(t)
    return v.reshape(y.shape), _pow2(e), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu).squeeze(-1)


def _dequantise(v, s, g, fmt):
    w = (_blocks(v, fmt) * s).reshape(v.shape)
    return w * g if fmt == "nvfp4" else w


def _pack4(v):
    """E2M1 values -> two 4-bit codes a byte, the even element in the low half."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=v.device)
    c = torch.bucketize(v.abs(), grid).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous()


def _unpack4(q):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    grid = torch.cat([grid, -grid])
    return torch.stack([grid[(q & 15).long()], grid[(q >> 4).long()]], -1).reshape(*q.shape[:-1], -1)


def _scale_bytes(s8):
    return s8.contiguous().view(torch.uint8)


def _scale_values(raw, fmt):
    if fmt == "nvfp4":
        return raw.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return _pow2(raw.int() - 127).unsqueeze(-1)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _acts(gen, *shape):
    """bf16 activations: normal, a few outliers, a few all-zero blocks."""
    x = torch.randn(shape, device="cuda", generator=gen)
    hit = torch.rand(shape, device="cuda", generator=gen)
    x = torch.where(hit < OUTLIERS, x * 100.0, x)
    xb = x.view(*shape[:-1], shape[-1] // 32, 32)
    dead = torch.rand(xb.shape[:-1], device="cuda", generator=gen) < ZERO_BLOCKS
    return xb.masked_fill_(dead.unsqueeze(-1), 0.0).view(shape).to(torch.bfloat16)


def _tensor_scale(gen, x, fmt):
    """The calibrated scale a serving program keeps for NVFP4 (None for the MX formats): up to 5 %
    of room above the largest value."""
    if fmt != "nvfp4":
        return None
    return (x.float().abs().amax() * (1 + 0.05 * torch.rand(1, device="cuda", generator=gen)) / (448.0 * 6.0)).reshape(1)


def _weights(gen, fmt, std, *shape):
    """Quantised weights as a checkpoint holds them: codes, scales, tensor scale."""
    w = (torch.randn(shape, device="cuda", generator=gen) * std).to(torch.bfloat16)
    g = _tensor_scale(gen, w, fmt)
    v, s, s8 = _quantise(w.float(), fmt, g)
    if fmt == "mxfp8":
        return {"q": v.to(torch.float8_e4m3fn).view(torch.uint8), "s": _scale_bytes(s8), "g": None}
    return {"q": _pack4(v), "s": _scale_bytes(s8), "g": g}


def _weight_values(w, fmt):
    """fp32 weights of the plain form."""
    v = w["q"].view(torch.float8_e4m3fn).float() if fmt == "mxfp8" else _unpack4(w["q"])
    return _dequantise(v, _scale_values(w["s"], fmt), w["g"], fmt)


def _laid_out(w, fmt):
    """The weights as a program keeps them for its calls: repacked once for the framework's
    kernels, or plain fp32."""
    if not own:
        return _weight_values(w, fmt)
    from mxfp8_block_scaled_02_gb300 import ops
    if fmt == "mxfp8":
        return ops.process_weights(w["q"], w["s"])
    return ops.process_weights_fp4(w["q"], w["s"], fmt, tensor_scale=w["g"])


def _raw(case, seed):
    """Everything a user has before the call, in the types they have it in."""
    gen, op, fmt = _gen(seed), case["op"], case["fmt"]
    if op == "quant":
        x = (torch.randn(case["m"], case["k"], device="cuda", generator=gen) * 0.02).to(torch.bfloat16)
        return {"x": x, "g": _tensor_scale(gen, x, fmt)}
    if op == "norm":
        m, k = case["m"], case["k"]
        r = {"x": _acts(gen, m, k), "w": (1 + 0.1 * torch.randn(k, device="cuda", generator=gen)).to(torch.bfloat16)}
        if case["residual"] != "none":
            res = torch.randn(m, k, device="cuda", generator=gen) * 3.0
            r["res"] = res.to(torch.bfloat16) if case["residual"] == "bf16" else res
        r["g"] = torch.full((1,), 8.0 / (448.0 * 6.0), device="cuda") if fmt == "nvfp4" else None
        return r
    if op == "act":
        return {"x": (2.0 * torch.randn(case["m"], 2 * case["k"], device="cuda", generator=gen)).to(torch.bfloat16),
                "g": torch.full((1,), 32.0 / (448.0 * 6.0), device="cuda") if fmt == "nvfp4" else None}
    if op == "mlp":
        m, k, f = case["m"], case["k"], case["f"]
        g = torch.full((1,), 8.0 / (448.0 * 6.0), device="cuda") if fmt == "nvfp4" else None
        return {"x": _acts(gen, m, k), "res": (3.0 * torch.randn(m, k, device="cuda", generator=gen)).to(torch.bfloat16),
                "w": (1 + 0.1 * torch.randn(k, device="cuda", generator=gen)).to(torch.bfloat16),
                "w1": _weights(gen, fmt, 0.02, 2 * f, k), "w2": _weights(gen, fmt, 0.02, k, f), "g": g}
    lead = (case["b"],) if case["b"] > 1 else ()
    x = _acts(gen, *lead, case["m"], case["k"])
    r = {"x": x, "g": _tensor_scale(gen, x, fmt), "w1": _weights(gen, fmt, 0.02, *lead, case["n"], case["k"]),
         "bias": (0.1 * torch.randn(case["n"], device="cuda", generator=gen)).to(torch.bfloat16) if case["bias"] else None}
    if case["x"] == "codes":
        v, _, s8 = _quantise(x.float(), fmt, r["g"])
        r["x"], r["s"] = _pack4(v), _scale_bytes(s8)
    return r


def prepare(case, seed):
    st = _raw(case, seed)
    st["case"] = case
    for name in ("w1", "w2"):
        if name in st:
            st[name] = _laid_out(st[name], case["fmt"])
    if own and case["op"] == "mlp":
        from mxfp8_block_scaled_02_gb300 import mlp
        st["mlp"] = mlp.GatedMLP(st["w"], st["w1"], st["w2"], eps=EPS, x_tensor_scale=st["g"], h_tensor_scale=st["g"])
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from mxfp8_block_scaled_02_gb300 import ops
    case, fmt = st["case"], st["case"]["fmt"]
    if case["op"] == "linear":
        return ops.linear_fp4(st["x"], st["w1"], st["bias"], st.get("s"), tensor_scale=st["g"])
    if case["op"] == "mlp":
        out, residual = st["mlp"](st["x"], st["res"])
        return {"out": out, "residual": residual}
    if case["op"] == "quant":
        q, s = ops.quantize_fp4(st["x"], fmt, tensor_scale=st["g"])
    elif case["op"] == "act":
        q, s = ops.silu_mul_quantize(st["x"], fmt=fmt, tensor_scale=st["g"])
    else:
        (q, s), residual = ops.rmsnorm_quantize(st["x"], st["w"], st.get("res"), eps=EPS, fmt=fmt, tensor_scale=st["g"])
    r = {"values": q.view(torch.float8_e4m3fn) if fmt == "mxfp8" else ops.unpack_fp4(q),
         "scales": s.view(torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu)}
    if case["op"] == "norm" and residual is not None:
        r["residual"] = residual
    return r


def _norm(x, res, w):
    """The sum in fp32 and its weighted root-mean-square norm."""
    t = x.float() if res is None else x.float() + res.float()
    return t, t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS) * w.float()


def _silu_mul(gate_up):
    gate, up = gate_up.float().chunk(2, -1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _product(y, fmt, g, w, bias=None):
    v, s, _ = _quantise(y, fmt, g)
    out = _dequantise(v, s, g, fmt) @ w.transpose(-1, -2)
    return (out if bias is None else out + bias.float()).to(torch.bfloat16)


def _run_plain(st):
    case, fmt = st["case"], st["case"]["fmt"]
    if case["op"] == "linear":
        if case["x"] == "codes":
            x = _dequantise(_unpack4(st["x"]), _scale_values(st["s"], fmt), st["g"], fmt)
            out = x @ st["w1"].transpose(-1, -2)
            return (out if st["bias"] is None else out + st["bias"].float()).to(torch.bfloat16)
        return _product(st["x"].float(), fmt, st["g"], st["w1"], st["bias"])
    if case["op"] == "mlp":
        t, y = _norm(st["x"], st["res"], st["w"])
        h = _silu_mul(_product(y, fmt, st["g"], st["w1"]))
        return {"out": _product(h, fmt, st["g"], st["w2"]), "residual": t.to(torch.bfloat16)}
    if case["op"] == "quant":
        v, _, s8 = _quantise(st["x"].float(), fmt, st["g"])
        return {"values": v.to(torch.float8_e4m3fn), "scales": s8}
    if case["op"] == "act":
        v, _, s8 = _quantise(_silu_mul(st["x"]), fmt, st["g"])
        return {"values": v.to(torch.float8_e4m3fn), "scales": s8}
    t, y = _norm(st["x"], st.get("res"), st["w"])
    v, _, s8 = _quantise(y, fmt, st["g"])
    r = {"values": v.to(torch.float8_e4m3fn), "scales": s8}
    if "res" in st:
        r["residual"] = t.to(st["res"].dtype)
    return r


# ------------------------------------------------------------------ what a pass cannot do without
def _tensor_bytes(rows, k, fmt):
    """Elements and scales of a quantised [rows, k] tensor."""
    return rows * k * (1.0 if fmt == "mxfp8" else 0.5) + rows * k / BLOCK[fmt]


def work(case):
    op, fmt, m, k = case["op"], case["fmt"], case["m"], case["k"]
    if op == "quant":  # x in; one E4M3 value per element and the scales out
        return {"bytes": 2 * m * k + _tensor_bytes(m, k, "mxfp8") - m * k / 32 + m * k / BLOCK[fmt], "flops": 3 * m * k}
    if op == "norm":
        res = {"bf16": 4, "fp32": 8, "none": 0}[case["residual"]]
        return {"bytes": m * k * (2 + res) + 2 * k + m * k * (1 + 1 / BLOCK[fmt]), "flops": 8 * m * k}
    if op == "act":
        return {"bytes": 4 * m * k + m * k * (1 + 1 / BLOCK[fmt]), "flops": 9 * m * k}
    if op == "mlp":
        f = case["f"]
        return {"bytes": m * k * (2 + 2 + 2 + 2) + 2 * k + _tensor_bytes(2 * f, k, fmt) + _tensor_bytes(k, f, fmt),
                "flops": 2 * m * k * 3 * f}
    b, n = case["b"], case["n"]
    x = 2 * b * m * k if case["x"] == "bf16" else _tensor_bytes(b * m, k, fmt)
    return {"bytes": x + _tensor_bytes(b * n, k, fmt) + 2 * b * m * n + (2 * n if case["bias"] else 0),
            "flops": 2 * b * m * n * k}


# ------------------------------------------------------------------ the definitions in 64 bits
def _round64(a, mant_bits, min_exp, largest):
    """a rounded to a binary format of ``mant_bits`` fraction bits, smallest normal exponent
    ``min_exp`` and largest value ``largest``: to nearest, ties to even, saturating."""
    e = torch.frexp(a.abs()).exponent.double() - 1
    ulp = torch.ldexp(torch.ones_like(a), (e.clamp_(min=min_exp) - mant_bits).int())
    return (torch.round(a / ulp) * ulp).clamp_(-largest, largest)


def _quantise64(y, fmt, g):
    """(element values, scale values) of y in 64 bits, scales without a trailing axis."""
    n = 16 if fmt == "nvfp4" else 32
    yb = y.unflatten(-1, (-1, n))
    top = yb.abs().amax(-1)
    if fmt == "nvfp4":
        s = _round64(top / (6 * g), 3, -6, 448.0)
        unit = (s * g).unsqueeze(-1)
        return _round64(torch.where(unit > 0, yb / torch.where(unit > 0, unit, 1.0), 0.0), 1, 0, 6.0).flatten(-2), s
    lead = 8 if fmt == "mxfp8" else 2
    lowest = torch.full_like(top, -127.0)
    e = torch.where(top > 0, torch.frexp(top).exponent.double() - 1 - lead, lowest).clamp(-127, 127)
    s = torch.ldexp(torch.ones_like(top), e.int())
    z = yb / s.unsqueeze(-1)
    return (_round64(z, 3, -6, 448.0) if fmt == "mxfp8" else _round64(z, 1, 0, 6.0)).flatten(-2), s


def _values64(w, fmt):
    """64-bit values of a quantised tensor given as bytes."""
    if fmt == "mxfp8":
        v = w["q"].view(torch.float8_e4m3fn).double()
    else:
        both = torch.stack([w["q"] & 15, w["q"] >> 4], -1).flatten(-2)
        mag = (both & 7).double()
        mag = torch.where(mag < 2, mag * 0.5, (1 + 0.5 * (mag % 2)) * torch.ldexp(torch.ones_like(mag), (torch.floor(mag / 2) - 1).int()))
        v = torch.where(both > 7, -mag, mag)
    n = 16 if fmt == "nvfp4" else 32
    s = w["s"].view(torch.float8_e4m3fn).double() * w["g"].double() if fmt == "nvfp4" else torch.ldexp(torch.ones_like(w["s"], dtype=torch.float64), w["s"].int() - 127)
    return (v.unflatten(-1, (-1, n)) * s.unsqueeze(-1)).flatten(-2)


def _fake64(y, fmt, g):
    """y quantised and back, in 64 bits."""
    v, s = _quantise64(y, fmt, g)
    n = 16 if fmt == "nvfp4" else 32
    r = (v.unflatten(-1, (-1, n)) * s.unsqueeze(-1)).flatten(-2)
    return r * g if fmt == "nvfp4" else r


def _norm64(st):
    t = st["x"].double()
    if "res" in st:
        t = t + st["res"].double()
    return t, t / torch.sqrt((t ** 2).mean(-1, keepdim=True) + EPS) * st["w"].double()


def _gated64(h):
    k = h.shape[-1] // 2
    return h[..., :k] * torch.sigmoid(h[..., :k]) * h[..., k:]


def exact(case, seed):
    st, op, fmt = _raw(case, seed), case["op"], case["fmt"]
    g = st["g"].double() if st["g"] is not None else None
    if op == "linear":
        x = _values64({"q": st["x"], "s": st["s"], "g": st["g"]}, fmt) if case["x"] == "codes" else _fake64(st["x"].double(), fmt, g)
        out = x @ _values64(st["w1"], fmt).mT
        return out if st["bias"] is None else out + st["bias"].double()
    if op == "mlp":
        # each operator's output is held in its own type between the steps
        t, y = _norm64(st)
        h = (_fake64(y, fmt, g) @ _values64(st["w1"], fmt).mT).to(torch.bfloat16).double()
        return {"out": _fake64(_gated64(h), fmt, g) @ _values64(st["w2"], fmt).mT, "residual": t}
    if op == "quant":
        v, s = _quantise64(st["x"].double(), fmt, g)
        return {"values": v, "scales": s}
    if op == "act":
        v, s = _quantise64(_gated64(st["x"].double()), fmt, g)
        return {"values": v, "scales": s}
    t, y = _norm64(st)
    v, s = _quantise64(y, fmt, g)
    r = {"values": v, "scales": s}
    if "res" in st:
        r["residual"] = t
    return r
