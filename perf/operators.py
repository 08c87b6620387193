"""The 16-bit expert layer's operators as calls to be timed: matrix products grouped by expert (forward, both
gradients), the dense product with bias, activation and residual (forward and backward), the gated activation between
an expert's products, and the weighted combine of a token's expert outputs, the last two with their gradients.

own = False computes each operator in its plain form, from elementary torch operations in 32 bits; own = True makes
the calls of bit_moe_amd.  Sizes follow the layer this library runs (hidden 7168, expert width 2048, 256 experts,
top-8), an expert-parallel share of it (32 experts) and its ranges.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---------------------------------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token's eight experts in a 256-expert layer: the up projection of a decode step, bound by the weights
        {"name": "experts_decode", "op": "experts", "dtype": "fp16", "T": 1, "k": 8, "E": 256, "N": 2048, "K": 7168,
         "zipf": 0.0, "idle": 0, "gather": True, "scatter": False},
        # a 2048-token prompt on the whole layer: about 64 rows an expert, every expert's weights read once
        {"name": "experts_prefill", "op": "experts", "dtype": "bf16", "T": 2048, "k": 8, "E": 256, "N": 2048, "K": 7168,
         "zipf": 0.0, "idle": 0, "gather": True, "scatter": False},
        # the down projection of a 32-expert share in training: skewed routing, an idle expert, rows back in pair order
        {"name": "experts_train", "op": "experts", "dtype": "bf16", "T": 4096, "k": 8, "E": 32, "N": 7168, "K": 2048,
         "zipf": 1.2, "idle": 1, "gather": False, "scatter": True},
        # its gradients: gate and up stacked (4096 outputs), dx of every pair and dw of every expert
        {"name": "experts_dx", "op": "experts_dx", "dtype": "bf16", "T": 2048, "k": 8, "E": 32, "N": 4096, "K": 7168,
         "zipf": 1.2, "idle": 1, "gather": False, "scatter": True},
        {"name": "experts_dw", "op": "experts_dw", "dtype": "bf16", "T": 2048, "k": 8, "E": 32, "N": 4096, "K": 7168,
         "zipf": 1.2, "idle": 1, "gather": True, "scatter": False},
        # a dense projection for one token: the latency of a single small product
        {"name": "linear_decode", "op": "linear", "dtype": "fp16", "T": 1, "N": 2048, "K": 7168, "act": "gelu",
         "bias": True, "residual": True, "pre": False},
        # the same for a 2048-token prompt, its pre-activation kept for a backward pass
        {"name": "linear_prompt", "op": "linear", "dtype": "bf16", "T": 2048, "N": 2048, "K": 7168, "act": "silu",
         "bias": True, "residual": True, "pre": True},
        # backward of the dense projection over 8192 tokens
        {"name": "linear_backward", "op": "linear_backward", "dtype": "bf16", "T": 8192, "N": 2048, "K": 7168,
         "act": "gelu_tanh", "bias": True},
        # SwiGLU of one token's eight expert rows (the smallest call), and its backward over 8192 tokens' pairs
        {"name": "swiglu_decode", "op": "swiglu", "dtype": "fp16", "R": 8, "I": 2048},
        {"name": "swiglu_backward", "op": "swiglu_backward", "dtype": "bf16", "R": 65536, "I": 2048},
        # the weighted sum of each token's eight expert rows onto the residual stream, and its backward
        {"name": "combine_prompt", "op": "combine", "dtype": "bf16", "T": 8192, "k": 8, "H": 7168, "residual": True},
        {"name": "combine_backward", "op": "combine_backward", "dtype": "bf16", "T": 8192, "k": 8, "H": 7168},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A feature size: mostly a multiple of 8, as 16-byte rows need, one in four any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(8, n // 8 * 8)


def draw(rng):
    most = [work(c) for c in listed()]
    flops, nbytes = max(w["flops"] for w in most), max(w["bytes"] for w in most)
    ops = ("experts", "experts", "experts_dx", "experts_dw", "linear", "linear", "linear_backward", "swiglu",
           "swiglu_backward", "combine", "combine_backward")
    while True:
        op = rng.choice(ops)
        c = {"op": op, "dtype": rng.choice(("bf16", "bf16", "fp16"))}
        if op.startswith("experts"):
            c["E"] = _log(rng, 1, 256)
            c["k"] = rng.randint(1, min(8, c["E"]))
            c.update(T=_log(rng, 1, 8192), N=_width(rng, 64, 8192), K=_width(rng, 64, 8192),
                     zipf=rng.choice((0.0, 0.6, 1.2)), gather=rng.random() < 0.5, scatter=rng.random() < 0.5)
            c["idle"] = rng.randint(0, (c["E"] - c["k"]) // 4)
            if op == "experts_dw":
                c["scatter"] = False
        elif op.startswith("linear"):
            c.update(T=_log(rng, 1, 16384), N=_width(rng, 64, 8192), K=_width(rng, 64, 8192), act=rng.choice(ACTS),
                     bias=rng.random() < 0.7)
            if op == "linear":
                c.update(residual=rng.random() < 0.5, pre=rng.random() < 0.3)
        elif op.startswith("swiglu"):
            c.update(R=_log(rng, 1, 65536), I=_width(rng, 64, 8192))
        else:
            c.update(T=_log(rng, 1, 16384), k=rng.randint(1, 8), H=_width(rng, 64, 8192))
            if op == "combine":
                c["residual"] = rng.random() < 0.5
        w = work(c)
        if w["flops"] <= flops and w["bytes"] <= nbytes:
            return c


def _popularity(c):
    """Each expert's share of the routing (0 for the idle ones, which are the last)."""
    n = c["E"] - c["idle"]
    p = [1.0 / (e + 1) ** c["zipf"] for e in range(n)]
    s = sum(p)
    return [v / s for v in p] + [0.0] * c["idle"]


def work(case):
    c, b = case, 2
    if c["op"].startswith("experts"):
        R, N, K = c["T"] * c["k"], c["N"], c["K"]
        # experts that some token chose, on average; rows of x are read once each where they are gathered
        active = sum(1.0 - max(0.0, 1.0 - min(1.0, c["k"] * p)) ** c["T"] for p in _popularity(c))
        active = max(active, float(c["k"]))
        rows = c["T"] if c["gather"] and c["op"] != "experts_dx" else R
        weights = (c["E"] if c["op"] == "experts_dw" else active) * N * K * b
        return {"bytes": weights + rows * K * b + R * N * b, "flops": 2.0 * R * N * K}
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": b * (T * K + N * K + T * N * (1 + c["residual"] + c["pre"]) + N * c["bias"]),
                "flops": 2.0 * T * N * K}
    if c["op"] == "linear_backward":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": b * (2 * T * N + 2 * T * K + 2 * N * K + N * c["bias"]), "flops": 4.0 * T * N * K}
    if c["op"] == "swiglu":
        return {"bytes": 3.0 * b * c["R"] * c["I"], "flops": 8.0 * c["R"] * c["I"]}
    if c["op"] == "swiglu_backward":
        return {"bytes": 5.0 * b * c["R"] * c["I"], "flops": 16.0 * c["R"] * c["I"]}
    n = c["T"] * c["H"]
    if c["op"] == "combine":
        return {"bytes": b * n * (c["k"] + 1 + c["residual"]) + 4.0 * c["T"] * c["k"], "flops": 2.0 * n * c["k"]}
    return {"bytes": b * n * (2 * c["k"] + 1) + 8.0 * c["T"] * c["k"], "flops": 3.0 * n * c["k"]}


# ---------------------------------------------------------------------------------------------------------------
# the inputs
# ---------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    c, dt, dev = case, DTYPES[case["dtype"]], "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device=dev).normal_(0.0, scale, generator=g)

    s = {"case": c}
    if c["op"].startswith("experts"):
        E, k, T, N, K = c["E"], c["k"], c["T"], c["N"], c["K"]
        # k distinct experts a token, drawn by popularity; then the pairs grouped by expert, in pair order within one
        score = torch.tensor(_popularity(c), device=dev).log()
        u = torch.empty(T, E, device=dev).uniform_(1e-6, 1.0 - 1e-6, generator=g)
        ids = (score - (-u.log()).log()).topk(k, dim=1).indices.flatten()
        counts = torch.bincount(ids, minlength=E)
        s["perm"] = torch.argsort(ids, stable=True).to(torch.int32)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["counts"] = counts.tolist()
        R = T * k
        if c["op"] != "experts_dw":
            s["w"] = normal(E, N, K, scale=1.0 / math.sqrt(K if c["op"] == "experts" else N))
        if c["op"] != "experts_dx":
            s["x"] = normal(T if c["gather"] else R, K)
        if c["op"] != "experts":
            s["dy"] = normal(R, N, scale=0.05)
    elif c["op"].startswith("linear"):
        T, N, K = c["T"], c["N"], c["K"]
        s["x"] = normal(T, K)
        s["w"] = normal(N, K, scale=1.0 / math.sqrt(K))
        if c["op"] == "linear":
            s["bias"] = normal(N, scale=0.5) if c["bias"] else None
            s["residual"] = normal(T, N) if c["residual"] else None
        else:
            s["pre"] = normal(T, N) if c["act"] != "none" else None
            s["dy"] = normal(T, N, scale=0.05)
    elif c["op"].startswith("swiglu"):
        # gate and up as the two halves of one product's output
        s["z"] = normal(c["R"], 2 * c["I"])
        if c["op"] == "swiglu_backward":
            s["dh"] = normal(c["R"], c["I"], scale=0.05)
    else:
        T, k, H = c["T"], c["k"], c["H"]
        s["o"] = normal(T * k, H)
        s["w"] = torch.softmax(normal(T, k, dtype=torch.float32), dim=1)
        if c["op"] == "combine":
            s["residual"] = normal(T, H) if c["residual"] else None
        else:
            s["dy"] = normal(T, H, scale=0.05)
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def run(state):
    return _call(state) if own else _plain(state)


def _call(s):
    import bit_moe_amd as bm
    c = s["case"]
    op = c["op"]
    if op == "experts":
        return bm.expert_matmul(s["x"], s["w"], s["offsets"], x_rows=s["perm"] if c["gather"] else None, x_div=c["k"],
                                y_rows=s["perm"] if c["scatter"] else None)
    if op == "experts_dx":
        return bm.expert_matmul_dx(s["dy"], s["w"], s["offsets"], dy_rows=s["perm"] if c["gather"] else None,
                                   dx_rows=s["perm"] if c["scatter"] else None)
    if op == "experts_dw":
        return bm.expert_matmul_dw(s["dy"], s["x"], s["offsets"], x_rows=s["perm"] if c["gather"] else None,
                                   x_div=c["k"])
    if op == "linear":
        y, pre = bm.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"], keep_pre=c["pre"])
        return [y, pre] if c["pre"] else [y]
    if op == "linear_backward":
        dx, dw, db = bm.linear_backward(s["dy"], s["x"], s["w"], act=c["act"], pre=s["pre"], need_db=c["bias"])
        return [dx, dw, db] if c["bias"] else [dx, dw]
    if op == "swiglu":
        return bm.swiglu(s["z"][:, :c["I"]], s["z"][:, c["I"]:])
    if op == "swiglu_backward":
        return list(bm.swiglu_backward(s["dh"], s["z"][:, :c["I"]], s["z"][:, c["I"]:]))
    if op == "combine":
        return bm.combine(s["o"], s["w"], residual=s["residual"])
    return list(bm.combine_backward(s["dy"], s["o"], s["w"]))


def _plain(s):
    c = s["case"]
    op, dt = c["op"], DTYPES[c["dtype"]]
    if op.startswith("experts"):
        return _plain_experts(s, op, dt)
    if op == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return [y.to(dt), z.to(dt)] if c["pre"] else [y.to(dt)]
    if op == "linear_backward":
        dz = s["dy"].float()
        if s["pre"] is not None:
            dz = dz * _act_slope(s["pre"].float(), c["act"])
        out = [(dz @ s["w"].float()).to(dt), (dz.t() @ s["x"].float()).to(dt)]
        return out + [dz.sum(0).to(dt)] if c["bias"] else out
    if op.startswith("swiglu"):
        gate, up = s["z"][:, :c["I"]].float(), s["z"][:, c["I"]:].float()
        sig = 1.0 / (1.0 + torch.exp(-gate))
        if op == "swiglu":
            return (gate * sig * up).to(dt)
        dh = s["dh"].float()
        return [(dh * up * sig * (1.0 + gate * (1.0 - sig))).to(dt), (dh * gate * sig).to(dt)]
    T, k, H = c["T"], c["k"], c["H"]
    o = s["o"].view(T, k, H).float()
    if op == "combine":
        y = (o * s["w"][:, :, None]).sum(1)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(dt)
    dy = s["dy"].float()[:, None, :]
    return [(s["w"][:, :, None] * dy).to(dt).view(T * k, H), (o * dy).sum(2)]


def _plain_experts(s, op, dt):
    """One product per expert that has rows, on its rows of the gathered operand."""
    c, perm = s["case"], s["perm"].long()
    R = c["T"] * c["k"]
    a = s["dy"] if op == "experts_dx" else s["x"]
    if c["gather"]:
        a = a[perm] if op == "experts_dx" else a[perm // c["k"]]
    if op == "experts_dw":
        out = torch.zeros(c["E"], c["N"], c["K"], dtype=dt, device=a.device)
    else:
        out = torch.empty(R, c["N"] if op == "experts" else c["K"], dtype=dt, device=a.device)
    r = 0
    for e, n in enumerate(s["counts"]):
        if not n:
            continue
        rows = a[r:r + n].float()
        if op == "experts_dw":
            out[e] = s["dy"][r:r + n].float().t() @ rows
        else:
            w = s["w"][e].float()
            y = (rows @ (w.t() if op == "experts" else w)).to(dt)
            if c["scatter"]:
                out[perm[r:r + n]] = y
            else:
                out[r:r + n] = y
        r += n
    return out


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        return sig * (1.0 + z * (1.0 - sig))
    return torch.ones_like(z)


# ---------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    f = {n: v.double() for n, v in s.items() if torch.is_tensor(v) and v.is_floating_point() and n != "w"}
    if op.startswith("experts"):
        return _exact_experts(c, s)
    if op == "linear":
        z = torch.matmul(f["x"], s["w"].double().t())
        z = z + f["bias"] if c["bias"] else z
        y = _exact_act(z, c["act"])[0]
        y = y + f["residual"] if c["residual"] else y
        return [y, z] if c["pre"] else [y]
    if op == "linear_backward":
        dz = f["dy"] * _exact_act(f["pre"], c["act"])[1] if c["act"] != "none" else f["dy"]
        out = [torch.matmul(dz, s["w"].double()), torch.matmul(dz.t(), f["x"])]
        return out + [dz.sum(dim=0)] if c["bias"] else out
    if op.startswith("swiglu"):
        # in slices of rows, so that the 64-bit copies stay small
        parts = []
        for r in range(0, c["R"], 8192):
            gate, up = s["z"][r:r + 8192].double().split(c["I"], dim=1)
            v, slope = _exact_act(gate, "silu")
            if op == "swiglu":
                parts.append((v * up,))
            else:
                dh = s["dh"][r:r + 8192].double()
                parts.append((dh * up * slope, dh * v))
        cols = [torch.cat(p) for p in zip(*parts)]
        return cols[0] if op == "swiglu" else cols
    T, k, H = c["T"], c["k"], c["H"]
    w = s["w"].double()
    if op == "combine":
        y = f["residual"] if c["residual"] else torch.zeros(T, H, dtype=torch.float64, device=w.device)
        for j in range(k):
            y = y + w[:, j:j + 1] * s["o"][j::k].double()
        return y
    do = torch.empty(T * k, H, dtype=torch.float64, device=w.device)
    dw = torch.empty(T, k, dtype=torch.float64, device=w.device)
    for j in range(k):
        do[j::k] = w[:, j:j + 1] * f["dy"]
        dw[:, j] = (s["o"][j::k].double() * f["dy"]).sum(dim=1)
    return [do, dw]


def _exact_experts(c, s):
    perm, k, op = s["perm"].long(), c["k"], c["op"]
    starts = s["offsets"].tolist()
    dev = perm.device
    if op == "experts_dw":
        if c["E"] * c["N"] * c["K"] > 1 << 30:
            return None
        out = torch.zeros(c["E"], c["N"], c["K"], dtype=torch.float64, device=dev)
    else:
        out = torch.zeros(c["T"] * k, c["N"] if op == "experts" else c["K"], dtype=torch.float64, device=dev)
    for e in range(c["E"]):
        at = torch.arange(starts[e], starts[e + 1], device=dev)
        if not at.numel():
            continue
        if op == "experts_dx":
            src = s["dy"][perm[at] if c["gather"] else at].double()
            val = torch.matmul(src, s["w"][e].double())
        else:
            src = s["x"][torch.div(perm[at], k, rounding_mode="floor") if c["gather"] else at].double()
            if op == "experts_dw":
                out[e] = torch.matmul(s["dy"][at].double().t(), src)
                continue
            val = torch.matmul(src, s["w"][e].double().t())
        out[perm[at] if c["scatter"] else at] = val
    return out


def _exact_act(z, act):
    """Activation and slope."""
    if act == "relu":
        return z.clamp(min=0.0), (z > 0).double()
    if act == "gelu":
        phi = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * phi, phi + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        # 0.5 (1 + tanh(u)) is the logistic function of 2 u
        u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
        p = torch.sigmoid(2.0 * u)
        du = math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * z ** 2)
        return z * p, p + 2.0 * z * p * (1.0 - p) * du
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1.0 - p)
    return z, torch.ones_like(z)
