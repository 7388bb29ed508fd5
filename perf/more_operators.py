"""The operators on microscaled (MX) numbers, as cases to time and to check.

  quantize  blocks of 32 values as 4-bit (e2m1) or 8-bit (e4m3) codes under a shared power of two
  norm      r' = r + scale * gate * post_norm(y), n = pre_norm(r') as MX codes and scales
  linear    y = act(x W^T + b) + r                    and its gradients (dx, dz, db)
  gated     h = act(x Wg^T + bg) * (x Wu^T + bu), and its gradients (dx, dg, du, dbg, dbu)

W is a frozen 4-bit MX matrix; x is bfloat16, binary16, or MX codes of 8 or 4 bits.  A block's scale is
2^(floor(log2 max|v|) - e), e = 2 for e2m1 and 8 for e4m3, and a code is v / scale rounded to nearest even and cut
to the largest code.  ``run`` computes an operator in plain torch operations in binary32 (binary64 where a value is
rounded to a code), or (``own``) with the library's kernels; ``exact`` computes it in binary64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


# ---- cases ---------------------------------------------------------------------------

def listed():
    return [
        # loading a model: the wide matrix of a layer to 4 bits, and back as the values that it stands for
        dict(name="quantize weights", op="quantize", M=12288, K=4096, dtype="bf16", to="fp4"),
        # the activations of an odd number of tokens to 8 bits, at the 1B-shaped layer's inner width
        dict(name="quantize activations", op="quantize", M=1001, K=8192, dtype="bf16", to="fp8"),
        # decode: residual add and the next norm for one token, all latency
        dict(name="norm token", op="norm", M=1, D=4096, dtype="bf16", r_dtype="bf16", to="fp8", pre="rms", post="none",
             gate=0, bias=False, scale=1.0),
        # a prompt through a layer with norms on both sides of the block and a learned per-channel residual scale
        dict(name="norm prompt", op="norm", M=2048, D=4096, dtype="bf16", r_dtype="bf16", to="fp8", pre="rms", post="rms",
             gate=1, bias=False, scale=0.5),
        # decode: the down projection of the 1B-shaped layer for one token in bfloat16, onto the residual stream
        dict(name="linear token", op="linear", M=1, N=2048, K=8192, x="bf16", dtype="bf16", act="none", bias=False,
             residual=True, save=False),
        # a decode batch of 32 on the wide matrix, 8-bit activations, bias and activation
        dict(name="linear batch", op="linear", M=32, N=12288, K=4096, x="fp8", dtype="bf16", act="gelu", bias=True,
             residual=False, save=False),
        # a prompt's down projection from 8-bit activations, onto the residual stream
        dict(name="linear prompt", op="linear", M=2048, N=4096, K=12288, x="fp8", dtype="bf16", act="none", bias=True,
             residual=True, save=False),
        # training: gradients through a frozen up projection with bias and activation, an odd number of tokens
        dict(name="linear gradient", op="linear_backward", M=1001, N=8192, K=2048, dtype="bf16", act="gelu_tanh",
             bias=True),
        # decode: the feed-forward block's first half for one token, 8-bit activations from the norm before it
        dict(name="gated token", op="gated", M=1, N=12288, K=4096, x="fp8", dtype="bf16", act="silu", bias=False,
             save=False),
        # a ragged number of tokens on an odd width, 4-bit activations, binary16 output
        dict(name="gated ragged", op="gated", M=333, N=8191, K=2080, x="fp4", dtype="f16", act="silu", bias=True,
             save=False),
        # a prompt, or a training forward pass that keeps both projections
        dict(name="gated prompt", op="gated", M=2048, N=12288, K=4096, x="fp8", dtype="bf16", act="silu", bias=False,
             save=True),
        # training: gradients through both frozen projections
        dict(name="gated gradient", op="gated_backward", M=4096, N=12288, K=4096, dtype="bf16", act="silu", bias=True),
    ]


MOST_FLOPS = 4 * 4096 * 12288 * 4096     # the largest listed case's


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.random()
    if kind < 0.15:
        return dict(op="quantize", M=_log(rng, 1, 12288), K=32 * _log(rng, 1, 128), dtype=rng.choice(["bf16", "f16", "f32"]),
                    to=rng.choice(["fp4", "fp8"]))
    if kind < 0.35:
        M, D = _log(rng, 1, 8192), 32 * _log(rng, 1, 256)
        dtype = rng.choice(["bf16", "bf16", "f16"])
        bias = rng.random() < 0.5
        divisors = [d for d in range(1, M + 1) if M % d == 0]
        return dict(op="norm", M=M, D=D, dtype=dtype, r_dtype=rng.choice([dtype, dtype, "f32"]),
                    to=rng.choice(["fp8", "fp8", "fp4"]), pre="layer" if bias else "rms",
                    post=rng.choice(["none", "layer" if bias else "rms"]), gate=rng.choice([0, 1, rng.choice(divisors)]),
                    bias=bias, scale=rng.choice([1.0, 0.5]))
    op = rng.choice(["linear", "linear", "linear_backward", "gated", "gated", "gated_backward"])
    N, K = _log(rng, 16, 12288), 32 * _log(rng, 2, 384)
    each = 4 if op.startswith("gated") else 2
    M = _log(rng, 1, min(8192, max(1, MOST_FLOPS // (each * N * K))))
    case = dict(op=op, M=M, N=N, K=K, dtype="bf16", bias=rng.random() < 0.5,
                act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"] + (["none"] if op.startswith("linear") else [])))
    if not op.endswith("backward"):                       # training is in bfloat16
        case["x"] = rng.choice(["bf16", "f16", "fp8", "fp8", "fp4"])
        case["dtype"] = case["x"] if case["x"].endswith("16") else rng.choice(["bf16", "bf16", "f16"])
        case["save"] = rng.random() < 0.5
    if op == "linear":
        case["residual"] = rng.random() < 0.5
    return case


#: Bytes of a value: MX codes with their share of a scale.
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 33 / 32, "fp4": 17 / 32}


def work(case):
    if case["op"] == "quantize":
        n = case["M"] * case["K"]
        # 4-bit codes are returned as values (no torch type holds them): those are the output then
        return {"bytes": n * (SIZE[case["dtype"]] + (SIZE["fp8"] if case["to"] == "fp8" else 2)), "flops": 2 * n}
    if case["op"] == "norm":
        M, D = case["M"], case["D"]
        e, er = SIZE[case["dtype"]], SIZE[case["r_dtype"]]
        norms = 1 + (case["post"] != "none")
        small = (norms * (1 + case["bias"]) + case["gate"]) * D * e
        return {"bytes": M * D * (e + 2 * er + (SIZE["fp8"] if case["to"] == "fp8" else 2)) + small + 16 * M,
                "flops": M * D * 4 * norms}
    M, N, K = case["M"], case["N"], case["K"]
    mats = 2 if case["op"].startswith("gated") else 1
    back = "backward" in case["op"]
    rows = 2 * M * N                     # bytes of one [M, N] tensor of 16-bit values
    b = mats * N * K * SIZE["fp4"] + M * K * (2 if back else SIZE[case["x"]]) + mats * case["bias"] * N * (4 if back else 2)
    if case["op"] == "linear":
        b += rows * (1 + case["residual"] + case["save"])
    elif case["op"] == "gated":
        b += rows * (1 + 2 * case["save"])
    elif case["op"] == "linear_backward":
        b += rows if case["act"] == "none" else 3 * rows
    else:
        b += 5 * rows
    return {"bytes": b, "flops": 2 * mats * M * N * K}


# ---- the plain quantiser (binary64: values next to a border between two codes) -----------

#: Exponent of the largest code's power of two, of the smallest normal one, bits of the fraction, the largest code.
FORMS = {"fp4": (2, 0, 1, 6.0), "fp8": (8, -6, 3, 448.0)}


def _floor_log2(v):
    return torch.frexp(v)[1] - 1                          # frexp: v = m 2^e, 1/2 <= m < 1 (0 for 0)


def _power(e):
    return torch.exp2(e.double())                         # exact; torch.ldexp is not, on every device


def _round_blocks(v, to):
    """Codes' values [M, K] and the blocks' exponents [M, K / 32] of v [M, K]."""
    top, low, bits, most = FORMS[to]
    v = v.double().unflatten(1, (-1, 32))
    amax = v.abs().amax(2)
    e = torch.where(amax > 0, (_floor_log2(amax) - top).clamp(min=-127), -127)
    t = v * _power(-e[..., None])
    step = _power(torch.where(t != 0, _floor_log2(t.abs()).clamp(min=low), low) - bits)
    return (torch.round(t / step) * step).clamp(-most, most).flatten(1), e


def _codes(q, to):
    if to == "fp8":
        return q.float().to(torch.float8_e4m3fn).view(torch.uint8)
    a = (2 * q.abs()).long()                              # 0, 1, 2, 3, 4, 6, 8, 12
    c = torch.where(a <= 4, a, torch.where(a == 6, 5, torch.where(a == 8, 6, 7))) + 8 * (q < 0)
    return (c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8)


def _mx(v, to):
    """The planes (codes, scales) of v."""
    q, e = _round_blocks(v, to)
    return _codes(q, to), (e + 127).to(torch.uint8)


def _returned(q, e, to, dtype):
    """What is returned of codes of values q under exponents e: 8-bit codes and scales in torch's types of them; of
    4-bit codes, which have none, the values."""
    if to == "fp8":
        return q.float().to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return (q.unflatten(1, (-1, 32)) * _power(e[..., None])).flatten(1).to(dtype)


# ---- inputs --------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape, scale=1.0, mean=0.0, dtype=None):
        t = torch.randn(*shape, generator=gen, device="cuda") * scale + mean
        return t.to(DTYPES[dtype or case["dtype"]])

    s = {"case": dict(case)}
    if case["op"] == "quantize":
        s["v"] = normal(case["M"], case["K"], scale=0.02 if case["to"] == "fp4" else 1.0)
        return s
    if case["op"] == "norm":
        M, D, G = case["M"], case["D"], case["gate"]
        s["y"], s["r"] = normal(M, D), normal(M, D, scale=2.0, dtype=case["r_dtype"])
        s["pre_weight"] = normal(D, scale=0.1, mean=1.0)
        s["post_weight"] = normal(D, scale=0.1, mean=1.0) if case["post"] != "none" else None
        s["pre_bias"] = normal(D, scale=0.1) if case["bias"] else None
        s["post_bias"] = normal(D, scale=0.1) if case["bias"] and case["post"] != "none" else None
        s["gate"] = normal(G, D, scale=0.3, mean=0.5) if G else None
        return s
    M, N, K = case["M"], case["N"], case["K"]
    for name in ("gate", "up") if case["op"].startswith("gated") else ("w",):
        s[name] = _mx(torch.randn(N, K, generator=gen, device="cuda") * 0.02, "fp4")
        if case["bias"] and not case["op"].endswith("backward"):
            s[name + "_bias"] = normal(N, scale=0.1)
    if case["op"] == "linear":
        s["residual"] = normal(M, N, scale=2.0) if case["residual"] else None
    if case["op"] in ("linear", "gated"):
        s["x"] = normal(M, K, dtype=case["x"]) if case["x"] in DTYPES else _mx(normal(M, K), case["x"])
        return s
    # gradients: what the forward pass kept (the values before the activation) and the output's gradient
    s["dy"] = normal(M, N, scale=0.01)
    spread = 0.02 * math.sqrt(K)
    if case["op"] == "linear_backward":
        s["w_pre"] = normal(M, N, scale=spread) if case["act"] != "none" else None
    else:
        s["gate_pre"], s["up_pre"] = normal(M, N, scale=spread), normal(M, N, scale=spread)
    return s


# ---- the plain forms (binary32, one rounding at the end) ----------------------------------

def _dense(x):
    """The binary32 values of a 16-bit tensor, or of MX planes."""
    if isinstance(x, torch.Tensor):
        return x.float()
    codes, scales = x
    if codes.shape[1] == 32 * scales.shape[1]:
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        c = torch.stack([codes & 15, codes >> 4], 2).flatten(1)
        a = (c & 7).float()
        a = torch.where(a < 4, 0.5 * a, torch.where(a < 6, a - 2, 2 * a - 8))
        v = torch.where(c > 7, -a, a)
    return (v.unflatten(1, (-1, 32)) * torch.exp2(scales[..., None].float() - 127)).flatten(1)


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return torch.where(z > 0, z, 0) if act == "relu" else z


def _act_slope(z, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return (z > 0).float() if act == "relu" else torch.ones_like(z)


def _normed(v, kind, weight, bias):
    """A norm of the rows of v, their mean and reciprocal standard deviation (0 and 1 where nothing is normalised)."""
    mean, rstd = torch.zeros_like(v[:, 0]), torch.ones_like(v[:, 0])
    if kind == "layer":
        mean = v.mean(1)
    if kind != "none":
        v = v - mean[:, None]
        rstd = 1 / torch.sqrt((v * v).mean(1) + EPS)
        v = v * rstd[:, None]
    v = v * weight.double() if weight is not None else v
    return v + bias.double() if bias is not None else v, mean, rstd


def _plain(s):
    c = s["case"]
    op, dtype = c["op"], DTYPES[c["dtype"]]
    if op == "quantize":
        return _returned(*_round_blocks(s["v"], c["to"]), c["to"], torch.bfloat16)
    if op == "norm":                                      # in binary64: n is rounded to codes
        p, m0, i0 = _normed(s["y"].double(), c["post"], s["post_weight"], s["post_bias"])
        if s["gate"] is not None:
            p = p * s["gate"].double().repeat_interleave(c["M"] // c["gate"], 0)
        r = s["r"].double() + c["scale"] * p
        n, m1, i1 = _normed(r, c["pre"], s["pre_weight"], s["pre_bias"])
        return (r.to(s["r"].dtype), _returned(*_round_blocks(n, c["to"]), c["to"], torch.bfloat16),
                torch.stack([m0, i0, m1, i1], 1).float())

    def project(name):
        z = _dense(s["x"]) @ _dense(s[name]).t()
        return z + s[name + "_bias"].float() if c["bias"] else z

    if op == "linear":
        z = project("w")
        y = _act(z, c["act"])
        y = (y + s["residual"].float() if c["residual"] else y).to(dtype)
        return (y, z.to(dtype)) if c["save"] else y
    if op == "gated":
        g, u = project("gate"), project("up")
        h = (_act(g, c["act"]) * u).to(dtype)
        return (h, g.to(dtype), u.to(dtype)) if c["save"] else h
    dy = s["dy"].float()
    if op == "linear_backward":
        dz = dy * _act_slope(s["w_pre"].float(), c["act"]) if c["act"] != "none" else dy
        out = {"dx": (dz @ _dense(s["w"])).to(dtype)}
        if c["act"] != "none":
            out["dz"] = dz.to(dtype)
        return dict(out, dbias=dz.sum(0)) if c["bias"] else out
    g, u = s["gate_pre"].float(), s["up_pre"].float()
    dg, du = dy * u * _act_slope(g, c["act"]), dy * _act(g, c["act"])
    dx = dg @ _dense(s["gate"]) + du @ _dense(s["up"])
    out = {"dx": dx.to(dtype), "dgate": dg.to(dtype), "dup": du.to(dtype)}
    return dict(out, dgate_bias=dg.sum(0), dup_bias=du.sum(0)) if c["bias"] else out


# ---- the library's operators -----------------------------------------------------------

def _library(s):
    import gemv_q4_affine_amd as Q

    c = s["case"]
    op = c["op"]
    types = {"fp4": Q.Q4_MXFP4, "fp8": Q.Q4_MXFP8}

    def returned(planes):
        if c["to"] == "fp8":
            return planes[0].view(torch.float8_e4m3fn), planes[1].view(torch.float8_e8m0fnu)
        return Q.mx_dequantize(planes, dtype=torch.bfloat16)

    if op == "quantize":
        return returned(Q.mx_quantize(s["v"], types[c["to"]]))
    if op == "norm":
        norms = {"none": Q.Q4_NORM_NONE, "rms": Q.Q4_NORM_RMS, "layer": Q.Q4_NORM_LAYER}
        r, n, stats = Q.block_norm_mx(
            s["r"], s["y"], pre_norm=norms[c["pre"]], pre_weight=s["pre_weight"], pre_bias=s["pre_bias"],
            post_norm=norms[c["post"]], post_weight=s["post_weight"], post_bias=s["post_bias"], gate=s["gate"],
            scale=c["scale"], eps=EPS, n_type=types[c["to"]], save_stats=True)
        return r, returned(n), stats
    act = {"none": Q.Q4_ACT_NONE, "silu": Q.Q4_ACT_SILU, "gelu": Q.Q4_ACT_GELU, "gelu_tanh": Q.Q4_ACT_GELU_TANH,
           "relu": Q.Q4_ACT_RELU}[c["act"]]
    if op == "linear":
        return Q.mx_linear(s["w"], s["x"], bias=s.get("w_bias"), act=act, residual=s["residual"], save_pre=c["save"],
                           dtype=DTYPES[c["dtype"]])
    if op == "gated":
        return Q.mx_gated(s["gate"], s["up"], s["x"], act=act, gate_bias=s.get("gate_bias"), up_bias=s.get("up_bias"),
                          save_pre=c["save"], dtype=DTYPES[c["dtype"]])
    if op == "linear_backward":
        return Q.mx_linear_backward(s["w"], s["dy"], act=act, pre=s["w_pre"], bias_grad=c["bias"])
    return Q.mx_gated_backward(s["gate"], s["up"], s["dy"], s["gate_pre"], s["up_pre"], act=act, bias_grad=c["bias"])


def run(state):
    return _library(state) if own else _plain(state)


# ---- binary64 --------------------------------------------------------------------------

#: The magnitudes that a code can have, in the codes' order.
MAGNITUDES = {"fp4": [0, 0.5, 1, 1.5, 2, 3, 4, 6],
              "fp8": [m / 8 * 2.0 ** -6 for m in range(8)]
                     + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)]}


def _quantised64(v, to):
    """Codes' values and scales: the nearest magnitude of the sorted list, the even code where two are as near."""
    v = v.reshape(v.shape[0], -1, 32)
    most = v.abs().max(2, keepdim=True).values
    power = torch.floor(torch.log2(most))
    power = power + (torch.exp2(power + 1) <= most).double() - (torch.exp2(power) > most).double()
    scale = torch.exp2((power - (2 if to == "fp4" else 8)).clamp(min=-127.0))
    table = torch.tensor(MAGNITUDES[to], dtype=torch.float64, device=v.device)
    middle = (table[1:] + table[:-1]) / 2
    t = v.abs() / scale
    at, after = torch.bucketize(t, middle), torch.bucketize(t, middle, right=True)      # they differ at a tie
    at = torch.where((at != after) & (at % 2 == 1), after, at)
    q = table[at] * torch.sign(v)
    if to == "fp8":
        return q.flatten(1), scale[..., 0]
    return (q * scale).flatten(1)


def _wide(x):
    """The binary64 values of a tensor or of MX planes."""
    if isinstance(x, torch.Tensor):
        return x.double()
    codes, scales = x
    table = torch.tensor(MAGNITUDES["fp4" if codes.shape[1] == 16 * scales.shape[1] else "fp8"] + [math.nan],
                         dtype=torch.float64, device=codes.device)
    if codes.shape[1] == 16 * scales.shape[1]:
        values = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.uint8, device=codes.device)
        values[:, 0::2], values[:, 1::2] = codes % 16, codes // 16
        values = torch.cat([table[:8], -table[:8]])[values.int()]
    else:
        values = torch.cat([table[:128], -table[:128]])[codes.int()]
    return values.mul_(torch.exp2(scales.double() - 127).repeat_interleave(32, 1))


def _act64(z, act):
    """The activation and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * (-z * z / 2).exp() / (2 * math.pi) ** 0.5
    a = (2 / math.pi) ** 0.5
    p = torch.sigmoid(2 * a * (z + 0.044715 * z ** 3))           # (1 + tanh v) / 2 = sigmoid(2 v)
    return z * p, p + z * p * (1 - p) * 2 * a * (1 + 0.134145 * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    op, M = case["op"], case["M"]
    if op == "quantize":
        return _quantised64(s["v"], case["to"])
    if op == "norm":
        one = torch.ones((), dtype=torch.float64, device="cuda")
        gate = one if s["gate"] is None else s["gate"][torch.arange(M, device="cuda") // (M // case["gate"])]
        wide = {k: one if s[k] is None else s[k] for k in ("pre_weight", "post_weight")}
        add = {k: 0 * one if s[k] is None else s[k] for k in ("pre_bias", "post_bias")}

        def centre(v, kind):
            m = v.mean(1, keepdim=True) * (kind == "layer")
            return m, torch.ones_like(m) if kind == "none" else (v.sub(m).square().mean(1, keepdim=True) + EPS).rsqrt()

        m0, i0 = centre(s["y"], case["post"])
        r = s["r"] + case["scale"] * gate * ((s["y"] - m0) * i0 * wide["post_weight"] + add["post_bias"])
        m1, i1 = centre(r, case["pre"])
        n = (r - m1) * i1 * wide["pre_weight"] + add["pre_bias"]
        return r, _quantised64(n, case["to"]), torch.cat([m0, i0, m1, i1], 1)

    def times(name):
        z = torch.mm(_wide(s["x"]), _wide(s[name]).t())
        return z.add_(s[name + "_bias"]) if case["bias"] else z

    if op == "linear":
        z = times("w")
        y = _act64(z, case["act"])[0]
        y = y if s["residual"] is None else y + s["residual"]
        return (y, z) if case["save"] else y
    if op == "gated":
        g, u = times("gate"), times("up")
        h = _act64(g, case["act"])[0] * u
        return (h, g, u) if case["save"] else h
    if op == "linear_backward":
        dz = s["dy"] if case["act"] == "none" else s["dy"] * _act64(s["w_pre"], case["act"])[1]
        out = {"dx": torch.mm(dz, _wide(s["w"]))}
        if case["act"] != "none":
            out["dz"] = dz
        return dict(out, dbias=dz.sum(0)) if case["bias"] else out
    value, slope = _act64(s["gate_pre"], case["act"])
    dg, du = s["dy"] * s["up_pre"] * slope, s["dy"] * value
    out = {"dx": torch.mm(dg, _wide(s["gate"])) + torch.mm(du, _wide(s["up"])), "dgate": dg, "dup": du}
    return dict(out, dgate_bias=dg.sum(0), dup_bias=du.sum(0)) if case["bias"] else out
