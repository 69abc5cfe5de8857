"""Cases of the norm in front of a Mixture-of-Experts layer and of its experts with 4-bit weights.

norm          layer norm or RMS norm of the residual stream's rows, after adding the previous
              layer's output to them
norm_grad     its gradient: of the rows, the weight and the bias
experts4      every expert's matrix product on its segment of the receive rows with weights of 4
              bits and a scale a group, with bias, activation (plain or gated) and residual

A case holds T (tokens) and H (row width); the experts' also E (experts), k (experts a token), R
(virtual ranks) and N (output width).  Receive rows are ordered by (expert, token), so an expert's
rows are consecutive.  4-bit formats: "int4" stands for scale * (code - 8) with bf16 scales, "e2m1"
for scale * the OCP E2M1 value with power-of-two scales (E8M0); two codes a byte, the lower nibble
first.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
GATED = ("swiglu", "geglu")
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-5


def listed():
    return [
        # One decode step of 16 sequences in front of the DeepSeek-V3-like workload's layer: the
        # combine's output is added to the stream and normed.  Latency.
        dict(name="norm decode", op="norm", T=16, H=7168, kind="rms", residual=True, beta=False,
             x="bf16", y="bf16", stats=False),
        # The non-divisible batch with a float32 stream, normed to the bf16 rows that the dispatch
        # takes, keeping what the gradient needs.
        dict(name="norm nondiv", op="norm", T=32768, H=2048, kind="layer", residual=True, beta=True,
             x="f32", y="bf16", stats=True),
        # The tiny shuffle's batch: latency.
        dict(name="norm grad tiny", op="norm_grad", T=128, H=256, kind="layer", residual=False,
             beta=True, x="f32", y="f32"),
        # Odd sizes: a row count and a width that no block divides, a float32 stream.
        dict(name="norm grad ragged", op="norm_grad", T=4099, H=1000, kind="rms", residual=True,
             beta=False, x="f32", y="bf16"),
        # The DeepSeek-V3-like training batch, with the stream's own gradient joining in.
        dict(name="norm grad train", op="norm_grad", T=16384, H=7168, kind="layer", residual=True,
             beta=True, x="bf16", y="bf16"),
        # One token through the gated first product of OLMoE-like experts: latency.
        dict(name="experts4 token", op="experts4", T=1, E=64, k=8, R=4, H=2048, N=1024, act="swiglu",
             bias=False, residual=False, zipf=0.0, format="int4", group=128),
        # One decode step of 16 sequences: bound by reading the weights.
        dict(name="experts4 decode", op="experts4", T=16, E=64, k=8, R=4, H=2048, N=1024,
             act="swiglu", bias=False, residual=False, zipf=0.0, format="e2m1", group=32),
        # A decode step of 16 sequences through the DeepSeek-V3-like layer's first product.
        dict(name="experts4 decode large", op="experts4", T=16, E=256, k=8, R=64, H=7168, N=1024,
             act="swiglu", bias=False, residual=False, zipf=0.0, format="int4", group=128),
        # The second product of Qwen3-like experts on a decode step of 64 sequences under Zipf
        # popularity, with bias and residual, in small groups.
        dict(name="experts4 decode zipf", op="experts4", T=64, E=128, k=8, R=8, H=1024, N=4096,
             act="none", bias=True, residual=True, zipf=1.2, format="int4", group=32),
        # The OLMoE-like prefill batch.
        dict(name="experts4 prefill", op="experts4", T=4096, E=64, k=8, R=4, H=2048, N=1024,
             act="swiglu", bias=False, residual=False, zipf=0.0, format="int4", group=128),
        # Odd sizes: rows that end inside every tile, widths that no tile and no group divides.
        dict(name="experts4 ragged", op="experts4", T=1021, E=30, k=4, R=8, H=776, N=1000,
             act="gelu", bias=True, residual=False, zipf=0.0, format="e2m1", group=32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "experts4", "experts4"])
    if op != "experts4":
        c = dict(op=op, T=_log_int(rng, 1, 32768), H=8 * _log_int(rng, 8, 1024),
                 kind=rng.choice(["layer", "rms"]), residual=rng.random() < 0.6,
                 beta=rng.random() < 0.5, x=rng.choice(["f32", "bf16"]), y=rng.choice(["f32", "bf16"]))
        if op == "norm":
            c["stats"] = rng.random() < 0.5
    else:
        E = _log_int(rng, 4, 256)
        c = dict(op=op, T=_log_int(rng, 1, 4096), E=E, k=rng.randint(1, min(8, E)))
        c.update(R=rng.randint(1, min(E, 16)), H=8 * _log_int(rng, 8, 896), N=8 * _log_int(rng, 8, 512),
                 act=rng.choice(["none", "relu", "silu", "gelu", "swiglu", "geglu"]),
                 bias=rng.random() < 0.4, residual=rng.random() < 0.4,
                 zipf=rng.choice([0.0, 0.0, 0.6, 1.2]))
        c["format"], c["group"] = rng.choice([("int4", 32), ("int4", 64), ("int4", 128), ("e2m1", 32)])
    most = {}
    for x in listed():
        if (x["op"] == "experts4") == (op == "experts4"):
            w = work(x)
            most = {m: max(most.get(m, 0), w[m]) for m in w}
    while c["T"] > 1 or c["H"] > 64:  # a pass that costs no more than the largest listed one
        w = work(c)
        if all(w[m] <= most[m] for m in w):
            break
        if c["T"] > 1:
            c["T"] = (c["T"] * 3) // 4
        else:
            c["H"] = 8 * max(8, c["H"] // 16)
    return c


def _device():
    return torch.device("cuda", torch.cuda.current_device())


def _normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=g.device) * scale).to(dtype)


def _stream_rows(g, c):
    """Rows of a residual stream: a few channels are much larger than the others."""
    wide = torch.rand((c["H"],), generator=g, device=g.device) < 0.01
    x = torch.randn((c["T"], c["H"]), generator=g, device=g.device)
    return (x * torch.where(wide, 8.0, 1.0) + torch.where(wide, 3.0, 0.1)).to(DTYPES[c["x"]])


def _routing(s, c, g):
    """A routing as a router gives it, and the receive layout that it implies."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = _normal(g, (T, E))
    if c["zipf"]:
        logits = logits - c["zipf"] * torch.log(torch.arange(1, E + 1, device=g.device))
    s["topk_idx"] = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    s["rows_of"] = torch.bincount(s["topk_idx"].reshape(-1).long(), minlength=E).tolist()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=_device())
    g.manual_seed(seed)
    s = dict(c)
    T, H = c["T"], c["H"]
    if c["op"] != "experts4":
        s["rows"] = _stream_rows(g, c)
        s["gamma"] = 1 + _normal(g, (H,), scale=0.2)
        if c["op"] == "norm":
            s["added"] = _normal(g, (T, H), DTYPES[c["x"]], 0.5) if c["residual"] else None
            s["bias"] = _normal(g, (H,), scale=0.2) if c["beta"] else None
        else:
            s["grad_y"] = _normal(g, (T, H), DTYPES[c["y"]])
            s["grad_total"] = _normal(g, (T, H), DTYPES[c["x"]]) if c["residual"] else None
            # the forward pass stores each row's mean (0 for the RMS norm) and 1 / deviation
            r = s["rows"].double()
            mean = r.mean(1, keepdim=True) if c["kind"] == "layer" else torch.zeros_like(r[:, :1])
            rstd = 1 / torch.sqrt((r - mean).square().mean(1, keepdim=True) + EPS)
            s["stats"] = torch.cat([mean, rstd], 1).float().contiguous()
    else:
        E, k, N = c["E"], c["k"], c["N"]
        Z = 2 * N if c["act"] in GATED else N   # width of the product itself
        groups = -(-H // c["group"])
        _routing(s, c, g)
        s["x"] = _normal(g, (T * k, H), torch.bfloat16)
        # Codes and scales as a checkpoint holds them: weights of variance 1 / H, quantized.
        s["codes"] = torch.empty((E, Z, H // 2), dtype=torch.uint8, device=g.device)
        for e in range(E):
            v = torch.randn((Z, H), generator=g, device=g.device)
            if c["format"] == "int4":
                q = (torch.round(v * 2.6) + 8).clamp(0, 15).to(torch.uint8)
            else:
                q = torch.bucketize((v * 2.2).abs(), v.new_tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]))
                q = q.to(torch.uint8) + 8 * (v < 0).to(torch.uint8)
            s["codes"][e] = q[:, 0::2] + 16 * q[:, 1::2]
        if c["format"] == "int4":
            u = torch.rand((E, Z, groups), generator=g, device=g.device)
            s["scales"] = ((0.7 + 0.6 * u) / (2.6 * math.sqrt(H))).to(torch.bfloat16)
        else:
            base = 127 + round(math.log2(1 / (2.2 * math.sqrt(H))))
            s["scales"] = torch.randint(base - 1, base + 2, (E, Z, groups), generator=g, device=g.device,
                                        dtype=torch.uint8)
        s["b"] = _normal(g, (E, Z), torch.float32, 0.5) if c["bias"] else None
        s["added"] = _normal(g, (T * k, N), torch.bfloat16) if c["residual"] else None
    if own:
        # The plan is the handle that a program keeps for a routing; the weights are laid out once.
        import combine_shuffling_amd as cs

        if c["op"] != "experts4":
            s["plan"] = cs.Plan(T, H, 1, 1, 1)
        else:
            s["plan"] = cs.Plan(T, 8, c["E"], c["k"], c["R"]).route(s["topk_idx"])
            s["w4"] = cs.pack_experts4(s["codes"], s["scales"], c["format"], c["group"])
    return s


# ---- the framework's calls

def _run_own(s):
    p = s["plan"]
    if s["op"] == "norm":
        y, total, stats = p.norm(s["rows"], s["gamma"], s["bias"], residual=s["added"], kind=s["kind"],
                                 eps=EPS, out_dtype=DTYPES[s["y"]], save_stats=s["stats"])
        return {"y": y, "total": total, "stats": stats}
    if s["op"] == "norm_grad":
        grad_x, grad_gamma, grad_beta = p.norm_backward(
            s["grad_y"], s["rows"], s["stats"], s["gamma"], grad_total=s["grad_total"],
            kind=s["kind"], beta_grad=s["beta"])
        return {"grad_x": grad_x, "grad_gamma": grad_gamma, "grad_beta": grad_beta}
    return {"y": p.expert_linear4(s["x"], s["w4"], bias=s["b"], residual=s["added"],
                                  activation=s["act"])}


# ---- the plain form

def _norm(s):
    x = s["rows"].float()
    total = None
    if s["added"] is not None:
        total = (x + s["added"].float()).to(s["rows"].dtype)
        x = total.float()
    if s["kind"] == "layer":
        mean = x.sum(1, keepdim=True) / s["H"]
    else:
        mean = torch.zeros_like(x[:, :1])
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).sum(1, keepdim=True) / s["H"] + EPS)
    y = d * rstd * s["gamma"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(DTYPES[s["y"]]), "total": total,
            "stats": torch.cat([mean, rstd], 1) if s["stats"] else None}


def _norm_grad(s):
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    h = (s["rows"].float() - mean) * rstd
    gy = s["grad_y"].float()
    g = gy * s["gamma"]
    d = g - h * ((g * h).sum(1, keepdim=True) / s["H"])
    if s["kind"] == "layer":
        d = d - g.sum(1, keepdim=True) / s["H"]
    d = d * rstd
    if s["grad_total"] is not None:
        d = d + s["grad_total"].float()
    return {"grad_x": d.to(s["rows"].dtype), "grad_gamma": (gy * h).sum(0),
            "grad_beta": gy.sum(0) if s["beta"] else None}


def _act(kind, z):
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind in ("silu", "swiglu"):
        return z / (1 + torch.exp(-z))
    if kind in ("gelu", "geglu"):
        return z * 0.5 * (1 + torch.erf(z / math.sqrt(2.0)))
    return z


def _weights(s, e):
    """Expert e's weights [Z, H] in float32."""
    c = s["codes"][e]
    q = torch.stack([c & 15, c >> 4], 2).reshape(c.shape[0], -1).long()
    if s["format"] == "int4":
        v, scale = (q - 8).float(), s["scales"][e].float()
    else:
        table = torch.tensor(E2M1 + tuple(-m for m in E2M1), device=c.device)
        v, scale = table[q], torch.exp2(s["scales"][e].float() - 127)
    return v * scale.repeat_interleave(s["group"], 1)[:, : s["H"]]


def _experts4(s):
    parts = []
    for e, a in enumerate(torch.split(s["x"], s["rows_of"])):
        if a.shape[0]:
            z = a.float() @ _weights(s, e).t()
            parts.append(z if s["b"] is None else z + s["b"][e])
    z = torch.cat(parts)
    if s["act"] in GATED:
        y = _act(s["act"], z[:, : s["N"]]) * z[:, s["N"]:]
    else:
        y = _act(s["act"], z)
    if s["added"] is not None:
        y = y + s["added"].float()
    return {"y": y.to(torch.bfloat16)}


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm, "norm_grad": _norm_grad, "experts4": _experts4}[state["op"]](state)


# ---- what a pass cannot do without

def work(case):
    c = case
    T, H = c["T"], c["H"]
    if c["op"] != "experts4":
        xs, ys = (4 if c[n] == "f32" else 2 for n in ("x", "y"))
        params = 4 * H * (1 + c["beta"])
        if c["op"] == "norm":
            b = T * H * (xs + ys) + params
            b += (2 * T * H * xs if c["residual"] else 0) + (8 * T if c["stats"] else 0)
            return {"bytes": b, "flops": 8 * T * H}
        b = T * H * (2 * xs + ys) + (T * H * xs if c["residual"] else 0) + 8 * T + 4 * H + params
        return {"bytes": b, "flops": 12 * T * H}
    E, k, N = c["E"], c["k"], c["N"]
    rows, Z = T * k, 2 * N if c["act"] in GATED else N
    # experts with rows, on average: each token leaves an expert out with its share
    share = np.arange(1, E + 1) ** -float(c["zipf"])
    hit = float((1 - (1 - np.minimum(k * share / share.sum(), 1.0)) ** T).sum())
    groups = -(-H // c["group"])
    b = hit * Z * (H / 2 + groups * (2 if c["format"] == "int4" else 1))
    b += rows * (H + N) * 2 + (hit * 4 * Z if c["bias"] else 0) + (rows * N * 2 if c["residual"] else 0)
    return {"bytes": b, "flops": 2.0 * rows * H * Z}


# ---- the definition, in 64 bits

def _exact_experts4(s):
    T, E, k, H, N = s["T"], s["E"], s["k"], s["H"], s["N"]
    of_row = torch.sort(s["topk_idx"].long().reshape(-1)).values
    Z = s["codes"].shape[1]
    dev = of_row.device
    values = torch.empty(16, dtype=torch.float64, device=dev)
    for q in range(16):
        if s["format"] == "int4":
            values[q] = q - 8
        else:   # sign, two bits of exponent, one of mantissa
            e, m = (q >> 1) & 3, q & 1
            values[q] = (-1.0) ** (q >> 3) * (m * 0.5 if e == 0 else (1 + m * 0.5) * 2.0 ** (e - 1))
    group_of = torch.arange(H, device=dev) // s["group"]
    z = torch.zeros((T * k, Z), dtype=torch.float64, device=dev)
    for e in range(E):
        at = (of_row == e).nonzero()[:, 0]
        if at.numel() == 0:
            continue
        w = torch.empty((Z, H), dtype=torch.float64, device=dev)
        w[:, 0::2] = values[(s["codes"][e] % 16).int()]
        w[:, 1::2] = values[(s["codes"][e] // 16).int()]
        scale = s["scales"][e].double()
        if s["format"] != "int4":
            scale = torch.ldexp(torch.ones_like(scale), s["scales"][e].int() - 127)
        w *= scale[:, group_of]
        z[at] = torch.mm(s["x"][at].double(), w.t().contiguous())
        if s["b"] is not None:
            z[at] += s["b"][e].double()
    gate = z[:, :N]
    if s["act"] == "relu":
        y = torch.relu(gate)
    elif s["act"] in ("silu", "swiglu"):
        y = gate * torch.sigmoid(gate)
    elif s["act"] in ("gelu", "geglu"):
        y = gate * torch.special.ndtr(gate)
    else:
        y = gate
    if Z > N:
        y = y * z[:, N:]
    if s["added"] is not None:
        y = y + s["added"].double()
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "experts4":
        return _exact_experts4(s)
    n = s["H"]
    if s["op"] == "norm":
        total = None
        x = s["rows"]
        if s["added"] is not None:     # by definition the float32 sum, stored in the rows' type
            total = x.float().add(s["added"].float()).to(x.dtype)
            x = total
        x = x.double()
        mu = x.mean(1) if s["kind"] == "layer" else x.new_zeros(s["T"])
        var = torch.linalg.vecdot(x - mu[:, None], x - mu[:, None]) / n
        rs = torch.pow(var + EPS, -0.5)
        y = (x - mu[:, None]) * torch.outer(rs, s["gamma"].double())
        if s["bias"] is not None:
            y += s["bias"].double()[None, :]
        return {"y": y, "total": None if total is None else total.double(),
                "stats": torch.stack([mu, rs], 1) if s["stats"] else None}
    mu, rs = s["stats"].double().unbind(1)
    h = (s["rows"].double() - mu[:, None]).mul_(rs[:, None])
    gy = s["grad_y"].double()
    out = {"grad_gamma": torch.linalg.vecdot(gy, h, dim=0), "grad_beta": gy.sum(0) if s["beta"] else None}
    g = gy.mul_(s["gamma"].double())
    along = torch.linalg.vecdot(g, h) / n
    d = g - h.mul_(along[:, None])
    if s["kind"] == "layer":
        d -= g.mean(1, keepdim=True)
    d *= rs[:, None]
    if s["grad_total"] is not None:
        d += s["grad_total"].double()
    out["grad_x"] = d
    return out
