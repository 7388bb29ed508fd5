"""The feed-forward operators on quantised weights, as cases to time and to check.

  linear  y = act(x W^T + b) + r          and its gradients (dx, dz, db)
  gated   h = act(x Wg^T + bg) * (x Wu^T + bu), and its gradients (dx, dg, du, dbg, dbu)
  norm    r' = r + scale * gate * post_norm(y), n = pre_norm(r'), and its gradients

W is a frozen matrix in one of the library's formats (Q4_0, affine 4-bit, affine 8-bit).  ``run`` computes an
operator in plain torch operations in binary32, or (``own``) with the library's kernels; ``exact`` computes it in
binary64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


# ---- cases ---------------------------------------------------------------------------

def listed():
    return [
        # decode: residual add and the next norm for one token, all latency
        dict(name="norm token", op="norm", M=1, D=2048, dtype="bf16", r_dtype="bf16", pre="rms", post="none", gate=0,
             bias=False, scale=1.0),
        # prompt: a layer with norms on both sides of the block and a learned per-channel residual scale
        dict(name="norm prompt", op="norm", M=2048, D=4096, dtype="bf16", r_dtype="bf16", pre="rms", post="rms", gate=1,
             bias=False, scale=0.5),
        # layer norms with biases at an odd width, binary32 residual stream, a conditioning gate per sequence of 125 tokens
        dict(name="norm ragged", op="norm", M=1000, D=1537, dtype="f16", r_dtype="f32", pre="layer", post="layer", gate=8,
             bias=True, scale=1.0),
        # training: the backward pass of the two-norm layer, a gate per sequence
        dict(name="norm gradient", op="norm_backward", M=8192, D=4096, dtype="bf16", r_dtype="bf16", pre="rms", post="rms",
             gate=4, bias=False, scale=1.0),
        # decode: the down projection of the 1B-shaped layer for one token, onto the residual stream
        dict(name="linear token", op="linear", fmt="q4_0", M=1, N=2048, K=8192, dtype="bf16", act="none", bias=False,
             residual=True, save=False),
        # a decode batch of 32 on the wide matrix, bias and activation
        dict(name="linear batch", op="linear", fmt="affine4", M=32, N=12288, K=4096, dtype="bf16", act="gelu", bias=True,
             residual=False, save=False),
        # a prompt's down projection in 8 bits, onto the residual stream
        dict(name="linear prompt", op="linear", fmt="affine8", M=2048, N=4096, K=12288, dtype="bf16", act="none", bias=True,
             residual=True, save=False),
        # training: gradients through a frozen up projection with bias and activation, an odd number of tokens
        dict(name="linear gradient", op="linear_backward", fmt="q4_0", M=1001, N=8192, K=2048, dtype="bf16",
             act="gelu_tanh", bias=True),
        # decode: the feed-forward block's first half for one token
        dict(name="gated token", op="gated", fmt="q4_0", M=1, N=12288, K=4096, dtype="bf16", act="silu", bias=False,
             save=False),
        # a ragged decode batch on the 1B-shaped layer in binary16
        dict(name="gated batch", op="gated", fmt="affine4", M=17, N=8192, K=2048, dtype="f16", act="silu", bias=False,
             save=False),
        # a prompt, or a training forward pass that keeps both projections
        dict(name="gated prompt", op="gated", fmt="q4_0", M=2048, N=12288, K=4096, dtype="bf16", act="silu", bias=False,
             save=True),
        # training: gradients through both frozen projections
        dict(name="gated gradient", op="gated_backward", fmt="affine8", M=4096, N=12288, K=4096, dtype="bf16", act="silu",
             bias=True),
    ]


MOST_FLOPS = 4 * 4096 * 12288 * 4096     # the largest listed case's


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.3:
        M, D = _log(rng, 1, 8192), _log(rng, 16, 8192)
        dtype = rng.choice(["bf16", "bf16", "f16"])
        bias = rng.random() < 0.5
        divisors = [d for d in range(1, M + 1) if M % d == 0]
        return dict(op=rng.choice(["norm", "norm_backward"]), M=M, D=D, dtype=dtype,
                    r_dtype=rng.choice([dtype, dtype, "f32"]), pre="layer" if bias else "rms",
                    post=rng.choice(["none", "layer" if bias else "rms"]), gate=rng.choice([0, 1, rng.choice(divisors)]),
                    bias=bias, scale=rng.choice([1.0, 0.5]))
    op = rng.choice(["linear", "linear", "linear_backward", "gated", "gated", "gated_backward"])
    fmt = rng.choice(["q4_0", "affine4", "affine8"])
    unit = 32 if fmt == "q4_0" else 64
    N = _log(rng, 16, 12288)
    K = unit * _log(rng, 2, 12288 // unit)
    each = 4 if op.startswith("gated") else 2
    M = _log(rng, 1, min(8192, max(1, MOST_FLOPS // (each * N * K))))
    dtype = "bf16" if op.endswith("backward") else rng.choice(["bf16", "bf16", "f16"])      # training is in bfloat16
    case = dict(op=op, fmt=fmt, M=M, N=N, K=K, dtype=dtype, bias=rng.random() < 0.5,
                act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"] + (["none"] if op.startswith("linear") else [])))
    if op == "linear":
        case["residual"] = rng.random() < 0.5
    if op in ("linear", "gated"):
        case["save"] = rng.random() < 0.5
    return case


def work(case):
    if case["op"].startswith("norm"):
        M, D = case["M"], case["D"]
        e, er = (4 if case[k] == "f32" else 2 for k in ("dtype", "r_dtype"))
        norms = 1 + (case["post"] != "none")
        small = (norms * (1 + case["bias"]) + case["gate"]) * D * e
        if case["op"] == "norm":
            return {"bytes": M * D * 2 * (e + er) + small + 16 * M, "flops": M * D * 4 * norms}
        back = norms * (1 + case["bias"]) * D * 4 + case["gate"] * D * e
        return {"bytes": M * D * (3 * e + 3 * er) + small + back + 16 * M, "flops": M * D * 10 * norms}
    M, N, K = case["M"], case["N"], case["K"]
    mats = 2 if case["op"].startswith("gated") else 1
    bits = 8.5 if case["fmt"] == "affine8" else 4.5
    rows = 2 * M * N                     # bytes of one [M, N] tensor of 16-bit values
    b = mats * N * K * bits / 8 + 2 * M * K + mats * case["bias"] * N * (4 if "backward" in case["op"] else 2)
    if case["op"] == "linear":
        b += rows * (1 + case["residual"] + case["save"])
    elif case["op"] == "gated":
        b += rows * (1 + 2 * case["save"])
    elif case["op"] == "linear_backward":
        b += rows if case["act"] == "none" else 3 * rows
    else:
        b += 5 * rows
    return {"bytes": b, "flops": 2 * mats * M * N * K}


# ---- inputs --------------------------------------------------------------------------

def _quantise(w, fmt):
    """The planes of a weight matrix [N, K] in one of the library's formats."""
    N, K = w.shape
    if fmt == "q4_0":
        v = w.view(N, K // 32, 32)
        d = v.gather(2, v.abs().argmax(2, keepdim=True)) / -8
        q = torch.clamp(torch.floor(v / d + 8.5), 0, 15).to(torch.uint8)
        return q[..., :16] | (q[..., 16:] << 4), d[..., 0].half().view(torch.int16)
    steps = 15 if fmt == "affine4" else 255
    v = w.view(N, K // 64, 64)
    low = v.amin(2, keepdim=True)
    s, b = ((v.amax(2, keepdim=True) - low) / steps).bfloat16(), low.bfloat16()
    q = torch.clamp(torch.floor((v - b.float()) / s.float() + 0.5), 0, steps).to(torch.uint8).view(N, K)
    if fmt == "affine4":
        q = q[:, 0::2] | (q[:, 1::2] << 4)
    return q.contiguous(), s[..., 0].contiguous().view(torch.int16), b[..., 0].contiguous().view(torch.int16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape, scale=1.0, mean=0.0, dtype=None):
        t = torch.randn(*shape, generator=gen, device="cuda") * scale + mean
        return t.to(DTYPES[dtype or case["dtype"]])

    s = {"case": dict(case)}
    if case["op"].startswith("norm"):
        M, D, G = case["M"], case["D"], case["gate"]
        s["y"], s["r"] = normal(M, D), normal(M, D, scale=2.0, dtype=case["r_dtype"])
        s["pre_weight"] = normal(D, scale=0.1, mean=1.0)
        s["post_weight"] = normal(D, scale=0.1, mean=1.0) if case["post"] != "none" else None
        s["pre_bias"] = normal(D, scale=0.1) if case["bias"] else None
        s["post_bias"] = normal(D, scale=0.1) if case["bias"] and case["post"] != "none" else None
        s["gate"] = normal(G, D, scale=0.3, mean=0.5) if G else None
        if case["op"] == "norm_backward":
            # what the forward pass keeps: r' (in place of r), y and the statistics of both norms
            s["dn"], s["dr"] = normal(M, D, scale=0.01), normal(M, D, scale=0.01, dtype=case["r_dtype"])
            s["stats"] = torch.cat([torch.stack(_stats(s[k].float(), case[w]), 1) for k, w in (("y", "post"), ("r", "pre"))], 1)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    for name in ("gate", "up") if case["op"].startswith("gated") else ("w",):
        s[name] = _quantise(torch.randn(N, K, generator=gen, device="cuda") * 0.02, case["fmt"])
        if case["bias"] and not case["op"].endswith("backward"):
            s[name + "_bias"] = normal(N, scale=0.1)
    if case["op"] == "linear":
        s["residual"] = normal(M, N, scale=2.0) if case["residual"] else None
    if case["op"] in ("linear", "gated"):
        s["x"] = normal(M, K)
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

def _dense(planes, fmt):
    if fmt == "q4_0":
        q, d = planes
        codes = torch.cat([q & 15, q >> 4], 2).float() - 8
        return (codes * d.view(torch.float16).float()[..., None]).flatten(1)
    q, s, b = planes
    if fmt == "affine4":
        q = torch.stack([q & 15, q >> 4], 2).flatten(1)
    q = q.float().view(q.shape[0], -1, 64)
    return (q * s.view(torch.bfloat16).float()[..., None] + b.view(torch.bfloat16).float()[..., None]).flatten(1)


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


def _stats(v, kind):
    """Mean and reciprocal standard deviation of the rows; 0 and 1 where nothing is normalised."""
    if kind == "none":
        return torch.zeros_like(v[:, 0]), torch.ones_like(v[:, 0])
    mean = v.mean(1) if kind == "layer" else torch.zeros_like(v[:, 0])
    return mean, 1 / torch.sqrt(((v - mean[:, None]) ** 2).mean(1) + EPS)


def _normed(v, stats, weight, bias):
    v = (v - stats[0][:, None]) * stats[1][:, None]
    v = v * weight.float() if weight is not None else v
    return v + bias.float() if bias is not None else v


def _norm_slope(dn, v, mean, rstd, weight, kind):
    """Gradients (input, weight, bias) of a norm of the rows of v."""
    hat = (v - mean[:, None]) * rstd[:, None]
    t = dn * weight.float()
    d = t - hat * (t * hat).mean(1, keepdim=True)
    if kind == "layer":
        d = d - t.mean(1, keepdim=True)
    return d * rstd[:, None], (dn * hat).sum(0), dn.sum(0)


def _rows_of(gate, M):
    return gate.float().repeat_interleave(M // gate.shape[0], 0) if gate is not None else 1.0


def _plain(s):
    c = s["case"]
    op, dtype = c["op"], DTYPES[c["dtype"]]
    if op == "norm":
        y, r = s["y"].float(), s["r"].float()
        post = _stats(y, c["post"])
        r = r + c["scale"] * _rows_of(s["gate"], c["M"]) * _normed(y, post, s["post_weight"], s["post_bias"])
        pre = _stats(r, c["pre"])
        n = _normed(r, pre, s["pre_weight"], s["pre_bias"])
        return r.to(s["r"].dtype), n.to(dtype), torch.stack(post + pre, 1)
    if op == "norm_backward":
        y, r, dn, stats, gate = s["y"].float(), s["r"].float(), s["dn"].float(), s["stats"], _rows_of(s["gate"], c["M"])
        d, pre_dw, pre_db = _norm_slope(dn, r, stats[:, 2], stats[:, 3], s["pre_weight"], c["pre"])
        d = d + s["dr"].float()
        dp = c["scale"] * gate * d
        out = {"dr": d.to(s["r"].dtype), "pre_dw": pre_dw}
        if s["gate"] is not None:
            p = _normed(y, (stats[:, 0], stats[:, 1]), s["post_weight"], s["post_bias"])
            out["dgate"] = (c["scale"] * d * p).view(c["gate"], -1, c["D"]).sum(1).to(dtype)
        post_db = None
        if c["post"] != "none":
            dp, out["post_dw"], post_db = _norm_slope(dp, y, stats[:, 0], stats[:, 1], s["post_weight"], c["post"])
        out["dy"] = dp.to(dtype)
        if c["bias"]:
            out["pre_db"] = pre_db
            if post_db is not None:
                out["post_db"] = post_db
        return out

    def project(name):
        z = s["x"].float() @ _dense(s[name], c["fmt"]).t()
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
        out = {"dx": (dz @ _dense(s["w"], c["fmt"])).to(dtype)}
        if c["act"] != "none":
            out["dz"] = dz.to(dtype)
        return dict(out, dbias=dz.sum(0)) if c["bias"] else out
    g, u = s["gate_pre"].float(), s["up_pre"].float()
    dg, du = dy * u * _act_slope(g, c["act"]), dy * _act(g, c["act"])
    dx = dg @ _dense(s["gate"], c["fmt"]) + du @ _dense(s["up"], c["fmt"])
    out = {"dx": dx.to(dtype), "dgate": dg.to(dtype), "dup": du.to(dtype)}
    return dict(out, dgate_bias=dg.sum(0), dup_bias=du.sum(0)) if c["bias"] else out


# ---- the library's operators -----------------------------------------------------------

def _library(s):
    import gemv_q4_affine_amd as Q

    c = s["case"]
    op = c["op"]
    norms = {"none": Q.Q4_NORM_NONE, "rms": Q.Q4_NORM_RMS, "layer": Q.Q4_NORM_LAYER}
    acts = {"none": Q.Q4_ACT_NONE, "silu": Q.Q4_ACT_SILU, "gelu": Q.Q4_ACT_GELU, "gelu_tanh": Q.Q4_ACT_GELU_TANH,
            "relu": Q.Q4_ACT_RELU}
    if op.startswith("norm"):
        how = dict(pre_norm=norms[c["pre"]], pre_weight=s["pre_weight"], pre_bias=s["pre_bias"], post_norm=norms[c["post"]],
                   post_weight=s["post_weight"], post_bias=s["post_bias"], gate=s["gate"], scale=c["scale"])
        if op == "norm":
            return Q.block_norm(s["r"], s["y"], eps=EPS, save_stats=True, **how)
        return Q.block_norm_backward(s["r"], s["y"], s["stats"], s["dn"], s["dr"], **how)
    act = acts[c["act"]]
    if op == "linear":
        return Q.q4_linear(s["w"], s["x"], bias=s.get("w_bias"), act=act, residual=s["residual"], save_pre=c["save"])
    if op == "gated":
        return Q.q4_gated(s["gate"], s["up"], s["x"], act=act, gate_bias=s.get("gate_bias"), up_bias=s.get("up_bias"),
                          save_pre=c["save"])
    if op == "linear_backward":
        return Q.q4_linear_backward(s["w"], s["dy"], act=act, pre=s["w_pre"], bias_grad=c["bias"])
    return Q.q4_gated_backward(s["gate"], s["up"], s["dy"], s["gate_pre"], s["up_pre"], act=act, bias_grad=c["bias"])


def run(state):
    return _library(state) if own else _plain(state)


# ---- binary64 --------------------------------------------------------------------------

def _weights64(planes, fmt):
    bits = {"q4_0": torch.float16}.get(fmt, torch.bfloat16)
    scale = planes[1].view(bits).double()
    offset = -8 * scale if fmt == "q4_0" else planes[2].view(bits).double()
    q, (N, groups) = planes[0].reshape(planes[0].shape[0], -1), scale.shape
    W = torch.empty(N, groups, 32 if fmt == "q4_0" else 64, dtype=torch.float64, device=q.device)
    if fmt == "q4_0":
        W[:, :, :16], W[:, :, 16:] = q.view(N, groups, 16) % 16, q.view(N, groups, 16) // 16
    elif fmt == "affine4":
        W[:, :, 0::2], W[:, :, 1::2] = q.view(N, groups, 32) % 16, q.view(N, groups, 32) // 16
    else:
        W.copy_(q.view(N, groups, 64))
    return W.mul_(scale.unsqueeze(2)).add_(offset.unsqueeze(2)).view(N, -1)


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
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in prepare(case, seed).items()}
    op, M = case["op"], case["M"]
    if op.startswith("norm"):
        one = torch.ones((), dtype=torch.float64, device="cuda")
        gate = one if s["gate"] is None else s["gate"][torch.arange(M, device="cuda") // (M // case["gate"])]
        wide = {k: one if s[k] is None else s[k] for k in ("pre_weight", "post_weight")}
        add = {k: 0 * one if s[k] is None else s[k] for k in ("pre_bias", "post_bias")}

        def centre(v, kind):
            m = v.mean(1, keepdim=True) * (kind == "layer")
            return m, torch.ones_like(m) if kind == "none" else (v.sub(m).square().mean(1, keepdim=True) + EPS).rsqrt()

        if op == "norm":
            m0, i0 = centre(s["y"], case["post"])
            r = s["r"] + case["scale"] * gate * ((s["y"] - m0) * i0 * wide["post_weight"] + add["post_bias"])
            m1, i1 = centre(r, case["pre"])
            return r, (r - m1) * i1 * wide["pre_weight"] + add["pre_bias"], torch.cat([m0, i0, m1, i1], 1)
        m0, i0, m1, i1 = s["stats"].split(1, 1)
        hat1, t1 = (s["r"] - m1) * i1, s["dn"] * wide["pre_weight"]
        total = s["dr"] + i1 * (t1 - hat1 * t1.mul(hat1).mean(1, keepdim=True) - (case["pre"] == "layer") * t1.mean(1, keepdim=True))
        hat0, back = (s["y"] - m0) * i0, case["scale"] * gate * total
        out = {"dr": total, "pre_dw": torch.sum(s["dn"] * hat1, 0)}
        if s["gate"] is not None:
            out["dgate"] = case["scale"] * (total * (hat0 * wide["post_weight"] + add["post_bias"])).view(case["gate"], -1, case["D"]).sum(1)
        if case["bias"]:
            out["pre_db"] = s["dn"].sum(0)
            if case["post"] != "none":
                out["post_db"] = back.sum(0)
        if case["post"] != "none":
            out["post_dw"] = torch.sum(back * hat0, 0)
            t0 = back * wide["post_weight"]
            back = i0 * (t0 - hat0 * t0.mul(hat0).mean(1, keepdim=True) - (case["post"] == "layer") * t0.mean(1, keepdim=True))
        return dict(out, dy=back)

    def times(name):
        z = torch.mm(s["x"], _weights64(s[name], case["fmt"]).t())
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
        out = {"dx": torch.mm(dz, _weights64(s["w"], case["fmt"]))}
        if case["act"] != "none":
            out["dz"] = dz
        return dict(out, dbias=dz.sum(0)) if case["bias"] else out
    value, slope = _act64(s["gate_pre"], case["act"])
    dg, du = s["dy"] * s["up_pre"] * slope, s["dy"] * value
    out = {"dx": torch.mm(dg, _weights64(s["gate"], case["fmt"])) + torch.mm(du, _weights64(s["up"], case["fmt"])),
           "dgate": dg, "dup": du}
    return dict(out, dgate_bias=dg.sum(0), dup_bias=du.sum(0)) if case["bias"] else out
