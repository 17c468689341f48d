"""Cases for the operators of a Mixture-of-Experts block that serve a few tokens or join the layer to its residual
stream: the whole layer for 1 to 128 tokens (bf16 weights, or e4m3 codes), and the norms before and after the block fused
with its gate and residual scale, forward and backward.

`run` computes them in their plain form (elementary torch operations in 32 bits) or, where `own` is true, through the
framework's entry points."""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------- the cases
def _decode(name, T, h, f, E, k, bias=False, fp8=False):
    return {"name": name, "op": "decode_fp8" if fp8 else "decode", "T": T, "h": h, "f": f, "E": E, "k": k, "bias": bias}


def _norm(name, op, T, h, res, gate, post=True, pre=True, alpha=1.0, beta=1.0):
    return {"name": name, "op": op, "T": T, "h": h, "res": res, "gate": gate, "post": post, "pre": pre, "alpha": alpha, "beta": beta}


def listed():
    return [
        # one user's next token through the DeepSeekMoE-shaped layer: the latency of a small model's decode step
        _decode("one token, 64 experts", 1, 2048, 1408, 64, 6),
        # a small batch through the Mixtral-8x7B-shaped layer: long rows, few wide experts
        _decode("4 tokens, 8 wide experts", 4, 4096, 14336, 8, 2),
        # a server's batch through the DeepSeekMoE-shaped layer: nearly every expert is hit, by a few tokens each
        _decode("32 tokens, 64 experts", 32, 2048, 1408, 64, 6),
        # the Internal-352B-shaped layer with its skewed router: the largest set of weights
        _decode("16 tokens, 32 skewed", 16, 4096, 14336, 32, 3, bias=True),
        # the largest batch the operator takes, Mixtral-8x7B-shaped
        _decode("128 tokens, 8 wide experts", 128, 4096, 14336, 8, 2),
        # odd sizes: multiples of 64 that fill no tile, a token count that fills no tile, a router bias
        _decode("13 tokens, odd sizes", 13, 1088, 704, 10, 3, bias=True),
        # single-token decode on e4m3 weights, Mixtral-8x7B-shaped
        _decode("one token, e4m3", 1, 4096, 14336, 8, 2, fp8=True),
        # a server's batch on e4m3 weights, DeepSeekMoE-shaped
        _decode("24 tokens, e4m3", 24, 2048, 1408, 64, 6, fp8=True),
        # between two blocks in training: post-norm, channel gate, residual, next pre-norm
        _norm("norms forward, training", "norm_fwd", 16384, 4096, "bf16", "channel", alpha=1.0, beta=0.5),
        # the same around a decode step: a few rows, an fp32 residual stream, a gate for each token
        _norm("norms forward, 7 rows", "norm_fwd", 7, 6400, "fp32", "token", alpha=1.25),
        # the backward of the first, in training
        _norm("norms backward, training", "norm_bwd", 16384, 4096, "bf16", "channel", alpha=1.0, beta=0.5),
        # an odd row count and width, an fp32 residual stream, a gate for each token
        _norm("norms backward, odd", "norm_bwd", 1021, 2056, "fp32", "token", alpha=1.25),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode_fp8", "norm_fwd", "norm_bwd"])
    if op.startswith("decode"):
        unit = 64 if op == "decode" else 128
        while True:
            E = _logint(rng, 2, 64)
            k = rng.randint(1, min(8, E))
            T = _logint(rng, 1, 128)
            h = unit * _logint(rng, 512 // unit, 6400 // unit)
            f = unit * _logint(rng, 256 // unit, 18304 // unit)
            if 3072 not in (h, f) and 1 << 24 <= E * h * f <= 32 * 4096 * 14336:
                break
        c = _decode("", T, h, f, E, k, bias=rng.random() < 0.4, fp8=op == "decode_fp8")
    else:
        while True:
            T, h = _logint(rng, 1, 32768), 8 * _logint(rng, 64, 1024)
            if h != 3072 and T != 3072 and T * h <= 16384 * 4096:
                break
        post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
        c = _norm("", op, T, h, rng.choice(["bf16", "fp32"]), rng.choice(["none", "channel", "token"]), post, pre,
                  rng.choice([1.0, 1.25]), rng.choice([1.0, 0.5]))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _router_bias(c, device):
    """A fixed bias that skews the load: the share of expert e falls as its rank grows."""
    return -0.8 * torch.log1p(torch.arange(c["E"], dtype=torch.float32, device=device))


def _quant_last(v):
    """e4m3 codes and one float32 scale for each row of the last axis: scale = amax / 448, 1 for a row of zeros."""
    s = v.float().abs().amax(-1, keepdim=True) / E4M3_MAX
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (v.float() / s).to(torch.float8_e4m3fn), s.squeeze(-1)


def _up(n):
    return -(-n // 256) * 256


def _qw_parts(c):
    """The quantised-weight buffer that the framework's header documents: each part's byte offset and shape."""
    E, h, f = c["E"], c["h"], c["f"]
    at, parts = 0, {}
    for name, shape, size in (("W13q", (E, 2 * f, h), 1), ("W2q", (E, h, f), 1), ("s1", (E, f), 4), ("s3", (E, f), 4), ("s2", (E, h), 4)):
        n = math.prod(shape) * size
        parts[name] = (at, n, shape)
        at += _up(n)
    return parts, at


def _qw_view(c, qw, name):
    at, n, shape = _qw_parts(c)[0][name]
    return qw[at:at + n].view(torch.float8_e4m3fn if name.endswith("q") else torch.float32).view(shape)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(dev).manual_seed(seed)

    def normal(shape, std=1.0, dtype=torch.bfloat16):
        v = torch.empty(shape, dtype=dtype, device=dev)
        return v.normal_(0.0, std, generator=g)

    if c["op"].startswith("decode"):
        T, h, f, E = c["T"], c["h"], c["f"], c["E"]
        s = {"case": c, "x": normal((T, h)), "Wg": normal((h, E), h ** -0.5, torch.float32),
             "b": _router_bias(c, dev) if c["bias"] else None}
        W1, W3, W2 = normal((E, h, f), h ** -0.5), normal((E, h, f), h ** -0.5), normal((E, f, h), f ** -0.5)
        if c["op"] == "decode":
            return dict(s, W1=W1, W3=W3, W2=W2)
        # the weights as a server keeps them: e4m3 codes with the contraction index last, a scale for each output column;
        # W1 and W3 columns alternate in groups of 128
        s["qw"] = torch.zeros(_qw_parts(c)[1], dtype=torch.uint8, device=dev)
        for e in range(E):
            q1, s1 = _quant_last(W1[e].t())
            q3, s3 = _quant_last(W3[e].t())
            q2, s2 = _quant_last(W2[e].t())
            groups = torch.stack([q1.view(torch.uint8).view(f // 128, 128, h), q3.view(torch.uint8).view(f // 128, 128, h)], 1)
            _qw_view(c, s["qw"], "W13q")[e].view(torch.uint8).copy_(groups.reshape(2 * f, h))
            _qw_view(c, s["qw"], "W2q")[e].view(torch.uint8).copy_(q2.view(torch.uint8))
            for name, v in (("s1", s1), ("s3", s3), ("s2", s2)):
                _qw_view(c, s["qw"], name)[e].copy_(v)
        return s
    T, h = c["T"], c["h"]
    res = torch.bfloat16 if c["res"] == "bf16" else torch.float32
    s = {"case": c, "r": normal((T, h), 2.0, res), "y": normal((T, h), 0.7),
         "w_post": 1 + normal((h,), 0.1, torch.float32) if c["post"] else None,
         "w_pre": 1 + normal((h,), 0.1, torch.float32) if c["pre"] else None,
         "gate": {"none": lambda: None, "channel": lambda: normal((h,), 0.5, torch.float32),
                  "token": lambda: torch.sigmoid(normal((T,), 1.0, torch.float32))}[c["gate"]]()}
    if c["op"] == "norm_bwd":
        s["dr_out"], s["du"] = normal((T, h), 1.0, res), normal((T, h)) if c["pre"] else None
    return s


# ---------------------------------------------------------------- the plain forms
EPS = 1e-5


def _route(s, k):
    """Expert ids (largest logit first, ties to the lower id) and the renormalised gates."""
    logits = s["x"].float() @ s["Wg"]
    if s["b"] is not None:
        logits = logits + s["b"]
    top, idx = torch.sort(logits, dim=-1, descending=True, stable=True)
    e = torch.exp(top[:, :k] - top[:, :1])
    return idx[:, :k].to(torch.int32), e / e.sum(-1, keepdim=True)


def _plain_decode(s):
    """Every token through every expert that some token chose, weighted by its gate or by zero."""
    c = s["case"]
    idx, gates = _route(s, c["k"])
    act = torch.unique(idx).long()
    weight = (gates.unsqueeze(-1) * (idx.unsqueeze(-1) == act)).sum(1)  # [T, active]
    if c["op"] == "decode":
        x = s["x"].float()
        a, b = torch.matmul(x, s["W1"][act].float()), torch.matmul(x, s["W3"][act].float())
        o = torch.matmul(a / (1 + torch.exp(-a)) * b, s["W2"][act].float())
    else:
        xq, sx = _quant_last(s["x"])
        f = c["f"]
        w13 = _qw_view(c, s["qw"], "W13q").view(torch.uint8)[act].view(torch.float8_e4m3fn).float().view(len(act), f // 128, 2, 128, c["h"])
        w1, w3 = w13[:, :, 0].reshape(len(act), f, -1), w13[:, :, 1].reshape(len(act), f, -1)
        a = torch.matmul(xq.float(), w1.transpose(1, 2)) * (sx[:, None] * _qw_view(c, s["qw"], "s1")[act][:, None, :])
        b = torch.matmul(xq.float(), w3.transpose(1, 2)) * (sx[:, None] * _qw_view(c, s["qw"], "s3")[act][:, None, :])
        hq, sh = _quant_last((a / (1 + torch.exp(-a)) * b).to(torch.bfloat16))  # H is quantised from its bf16 value
        w2 = _qw_view(c, s["qw"], "W2q").view(torch.uint8)[act].view(torch.float8_e4m3fn).float()
        o = torch.matmul(hq.float(), w2.transpose(1, 2)) * (sh[..., None] * _qw_view(c, s["qw"], "s2")[act][:, None, :])
    return {"y": (o * weight.t().unsqueeze(-1)).sum(0).to(torch.bfloat16), "topk_idx": idx, "gates": gates}


def _gate_of(s):
    g = s["gate"]
    return 1.0 if g is None else g[:, None] if s["case"]["gate"] == "token" else g


def _plain_norm_fwd(s):
    """r_out = alpha r + beta gate * rms(y) w_post, u = rms(r_out) w_pre: the second norm is of the stored value."""
    c = s["case"]
    z = s["y"].float()
    if c["post"]:
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * s["w_post"]
    out = (c["alpha"] * s["r"].float() + c["beta"] * _gate_of(s) * z).to(s["r"].dtype)
    if not c["pre"]:
        return {"r_out": out}
    v = out.float()
    return {"r_out": out, "u": (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["w_pre"]).to(torch.bfloat16)}


def _plain_norm_bwd(s):
    c = s["case"]
    v, y, G = s["r"].float(), s["y"].float(), s["dr_out"].float()
    out = {}
    if c["pre"]:  # s["r"] is the forward's r_out
        rs = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
        t = s["du"].float() * s["w_pre"]
        G = G + rs * (t - v * rs.square() * (t * v).mean(-1, keepdim=True))
        out["dw_pre"] = (s["du"].float() * v * rs).sum(0)
    out["dr"] = (c["alpha"] * G).to(s["r"].dtype)
    G = c["beta"] * G
    n, ry = y, None
    if c["post"]:
        ry = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
        n = y * ry
        out["dw_post"] = (G * _gate_of(s) * n).sum(0)
    w = s["w_post"] if c["post"] else 1.0
    if c["gate"] != "none":
        out["dgate"] = (G * n * w).sum(0 if c["gate"] == "channel" else 1)
    t = G * _gate_of(s) * w
    if c["post"]:
        t = ry * (t - n * (t * n).mean(-1, keepdim=True))
    out["dy"] = t.to(torch.bfloat16)
    return out


# ---------------------------------------------------------------- one pass
def _own_decode(s):
    from routing_grouped_expert_router_gb300 import binding as mb
    c = s["case"]
    if "ws" not in s:  # a program keeps these from step to step
        fp8 = c["op"] == "decode_fp8"
        s["d"] = mb.dims(c["T"], c["h"], c["f"], c["E"], c["k"], has_bias=c["bias"])
        s["ws"] = torch.zeros(mb.moe_workspace_bytes(s["d"], mb.OP_LAYER_DECODE_FP8 if fp8 else mb.OP_LAYER_DECODE), dtype=torch.uint8, device="cuda")
        s["out"] = {"y": torch.empty_like(s["x"]), "topk_idx": torch.empty((c["T"], c["k"]), dtype=torch.int32, device="cuda"),
                    "gates": torch.empty((c["T"], c["k"]), dtype=torch.float32, device="cuda")}
    o = s["out"]
    if c["op"] == "decode":
        mb.moe_layer_decode(s["d"], s["x"], s["Wg"], s["b"], s["W1"], s["W3"], s["W2"], o["y"], o["topk_idx"], o["gates"], s["ws"])
    else:
        mb.moe_layer_decode_fp8(s["d"], s["x"], s["Wg"], s["b"], s["qw"], o["y"], o["topk_idx"], o["gates"], s["ws"])
    return o


def _own_norm(s):
    from routing_grouped_expert_router_gb300 import binding as mb
    c = s["case"]
    if "nd" not in s:
        s["nd"] = mb.norm_dims(c["T"], c["h"], res_f32=c["res"] == "fp32", gate={"none": mb.GATE_NONE, "channel": mb.GATE_CHANNEL, "token": mb.GATE_TOKEN}[c["gate"]],
                               eps=EPS, alpha=c["alpha"], beta=c["beta"])
        new = torch.empty_like
        if c["op"] == "norm_fwd":
            s["out"] = {"r_out": new(s["r"])} | ({"u": new(s["y"])} if c["pre"] else {})
        else:
            s["ws"] = torch.zeros(mb.moe_norm_workspace_bytes(s["nd"]), dtype=torch.uint8, device="cuda")
            s["out"] = {"dr": new(s["r"]), "dy": new(s["y"])}
            s["out"] |= {n: new(s[p]) for n, p in (("dw_pre", "w_pre"), ("dw_post", "w_post"), ("dgate", "gate")) if s[p] is not None}
    o = s["out"]
    if c["op"] == "norm_fwd":
        mb.moe_block_norm_fwd(s["nd"], s["r"], s["y"], s["w_post"], s["gate"], s["w_pre"], o["r_out"], o.get("u"))
    else:
        mb.moe_block_norm_bwd(s["nd"], s["r"], s["y"], s["w_post"], s["gate"], s["w_pre"], s["du"], s["dr_out"], o["dr"], o["dy"],
                              o.get("dw_post"), o.get("dgate"), o.get("dw_pre"), s["ws"])
    return o


def run(state):
    op = state["case"]["op"]
    if op.startswith("decode"):
        return _own_decode(state) if own else _plain_decode(state)
    if own:
        return _own_norm(state)
    return _plain_norm_fwd(state) if op == "norm_fwd" else _plain_norm_bwd(state)


# ---------------------------------------------------------------- the work
def _active(c):
    """How many experts the tokens choose, on average over draws of the router's logits."""
    r = np.random.RandomState(1)
    bias = -0.8 * np.log1p(np.arange(c["E"])) if c["bias"] else 0.0
    n = [len(np.unique(np.argsort(-(r.randn(c["T"], c["E"]) + bias), axis=1)[:, :c["k"]])) for _ in range(16)]
    return float(np.mean(n))


def work(case):
    c = case
    T, h = c["T"], c["h"]
    if c["op"].startswith("decode"):
        f, E, k = c["f"], c["E"], c["k"]
        size = 2 if c["op"] == "decode" else 1
        weights = _active(c) * (3 * h * f * size + (0 if size == 2 else 4 * (2 * f + h)))
        return {"bytes": weights + 4 * h * E + (4 * E if c["bias"] else 0) + 4 * T * h + 8 * T * k,
                "flops": 6.0 * T * k * h * f + 2.0 * T * h * E}
    n, r = T * h, 4 if c["res"] == "fp32" else 2
    small = 4 * ((h if c["post"] else 0) + (h if c["pre"] else 0) + {"none": 0, "channel": h, "token": T}[c["gate"]])
    if c["op"] == "norm_fwd":
        return {"bytes": n * (2 * r + 2 + (2 if c["pre"] else 0)) + small, "flops": 12.0 * n}
    reads = r + 2 + ((r + 2) if c["pre"] else 0)  # dr_out and y; r_out and du for the norm before the next block
    return {"bytes": n * (reads + r + 2) + 2 * small, "flops": 30.0 * n}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"].startswith("decode"):
        T, k = c["T"], c["k"]
        logits = s["x"].double() @ s["Wg"].double()
        if s["b"] is not None:
            logits += s["b"].double()
        p = torch.softmax(logits, -1)
        idx = torch.argsort(logits, dim=-1, descending=True, stable=True)[:, :k]
        gates = torch.gather(p, 1, idx)
        gates = gates / gates.sum(-1, keepdim=True)
        y = torch.zeros((T, c["h"]), dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            t, j = torch.nonzero(idx == e, as_tuple=True)
            if not len(t):
                continue
            x = s["x"][t]
            if c["op"] == "decode":
                a, b = x.double() @ s["W1"][e].double(), x.double() @ s["W3"][e].double()
                o = (a * torch.sigmoid(a) * b) @ s["W2"][e].double()
            else:
                groups = _qw_view(c, s["qw"], "W13q")[e].double().view(c["f"] // 128, 2, 128, c["h"])
                w1, w3, w2 = groups[:, 0].reshape(c["f"], -1), groups[:, 1].reshape(c["f"], -1), _qw_view(c, s["qw"], "W2q")[e].double()
                q, sc = _quant_last(x)
                x64 = q.double() * sc.double()[:, None]
                a, b = (x64 @ w1.t()) * _qw_view(c, s["qw"], "s1")[e].double(), (x64 @ w3.t()) * _qw_view(c, s["qw"], "s3")[e].double()
                q, sc = _quant_last((a * torch.sigmoid(a) * b).to(torch.bfloat16))
                o = ((q.double() * sc.double()[:, None]) @ w2.t()) * _qw_view(c, s["qw"], "s2")[e].double()
            y.index_add_(0, t, o * gates[t, j][:, None])
        return {"y": y, "topk_idx": None, "gates": gates}
    d = lambda v: None if v is None else v.double()  # noqa: E731
    y, wq, wp, al, be = d(s["y"]), d(s["w_post"]), d(s["w_pre"]), c["alpha"], c["beta"]
    gate = torch.ones((), dtype=torch.float64, device="cuda") if s["gate"] is None else d(s["gate"])
    gate = gate.view(-1, 1) if c["gate"] == "token" else gate
    rms = lambda v: torch.sqrt((v * v).sum(-1, keepdim=True) / c["h"] + EPS)  # noqa: E731
    z = y / rms(y) * wq if c["post"] else y
    if c["op"] == "norm_fwd":
        r = al * d(s["r"]) + be * gate * z
        r = r.to(s["r"].dtype).double() if c["res"] == "bf16" else r
        return {"r_out": r, "u": r / rms(r) * wp} if c["pre"] else {"r_out": r}
    # the gradients as sums over each row's Jacobian: d(v_i / rms) / d v_j = delta_ij / rms - v_i v_j / (h rms^3)
    G, out = d(s["dr_out"]), {}
    if c["pre"]:
        v, du = d(s["r"]), d(s["du"])
        q = rms(v)
        G = G + du * wp / q - v * (du * wp * v).sum(-1, keepdim=True) / (c["h"] * q ** 3)
        out["dw_pre"] = (du * v / q).sum(0)
    out["dr"] = al * G
    dz = be * G
    if c["gate"] != "none":
        out["dgate"] = (dz * z).sum(1 if c["gate"] == "token" else 0)
    dz = dz * gate
    if c["post"]:
        q = rms(y)
        out["dw_post"] = (dz * y / q).sum(0)
        dz = dz * wq
        dz = dz / q - y * (dz * y).sum(-1, keepdim=True) / (c["h"] * q ** 3)
    out["dy"] = dz
    return out
