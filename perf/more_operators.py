"""The expert layer's operators in 8 bits and the norms around the layer as calls to be timed: matrix products in 8-bit
integers with a scale for each token and channel (grouped by expert and dense), activation checkpoints in 8 bits and
their use in the backward pass, and the norms before and after a block with its gate and residual scale.

own = False computes each operator in its plain form, from elementary torch operations in 32 bits; own = True makes
the calls of bit_moe_amd.  Sizes follow the layer this library runs (hidden 7168, expert width 2048, 256 experts,
top-8), an expert-parallel share of it (32 experts) and its ranges.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token's eight experts of 256, gate and up stacked: a decode step's first product, bound by the weights
        {"name": "i8_decode", "op": "i8", "dtype": "fp16", "T": 1, "k": 8, "E": 256, "N": 4096, "K": 7168,
         "zipf": 0.0, "idle": 0, "gather": True, "scatter": False},
        # a 2048-token prompt on the whole layer: about 64 rows an expert, every expert's weights read once
        {"name": "i8_prefill", "op": "i8", "dtype": "bf16", "T": 2048, "k": 8, "E": 256, "N": 2048, "K": 7168,
         "zipf": 0.0, "idle": 0, "gather": True, "scatter": False},
        # from gate and up to the down projection's outputs, over a 32-expert share: skewed routing, an idle expert
        {"name": "i8_down", "op": "i8_swiglu", "dtype": "bf16", "T": 4096, "k": 8, "E": 32, "N": 7168, "K": 2048,
         "zipf": 1.2, "idle": 1, "gather": False, "scatter": True},
        # the shared expert's gate and up for an 8192-token prompt: one dense product, bound by the matrix cores
        {"name": "i8_dense", "op": "i8", "dtype": "bf16", "T": 8192, "k": 1, "E": 1, "N": 4096, "K": 7168,
         "zipf": 0.0, "idle": 0, "gather": False, "scatter": False},
        # a pruned layer's sizes, no row of which begins on a 16-byte address
        {"name": "i8_odd", "op": "i8", "dtype": "fp16", "T": 333, "k": 2, "E": 8, "N": 1001, "K": 2047,
         "zipf": 0.6, "idle": 1, "gather": True, "scatter": True},
        # a few tokens' gate and up kept in 8 bits by the forward pass and read by the backward: the smallest step
        {"name": "checkpoint_small", "op": "checkpoint", "dtype": "fp16", "R": 64, "I": 2048, "block": 64},
        # the same over 8192 tokens' pairs, what a training step keeps of an expert layer
        {"name": "checkpoint_train", "op": "checkpoint", "dtype": "bf16", "R": 65536, "I": 2048, "block": 64},
        # 16384 tokens' hidden states kept in 8 bits and restored for a weights' gradient
        {"name": "checkpoint_rows", "op": "rows", "dtype": "bf16", "R": 16384, "I": 7168, "block": 64},
        # one token between two blocks: the norm after the first, the residual stream, the norm before the next
        {"name": "norm_decode", "op": "norm", "dtype": "fp16", "T": 1, "H": 7168, "gate": "none", "stream": "fp16"},
        # the same for 8192 tokens, a gate for each channel, the residual stream kept in 32 bits
        {"name": "norm_prompt", "op": "norm", "dtype": "bf16", "T": 8192, "H": 7168, "gate": "channel",
         "stream": "fp32"},
        # its backward over 8192 tokens, the stream in 16 bits
        {"name": "norm_backward", "op": "norm_backward", "dtype": "bf16", "T": 8192, "H": 7168, "gate": "channel",
         "stream": "bf16"},
        # the backward at a pruned width, with a gate for each token and channel
        {"name": "norm_gated_backward", "op": "norm_backward", "dtype": "fp16", "T": 3001, "H": 2047, "gate": "token",
         "stream": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A feature size: mostly a multiple of 16, as 16-byte rows of 8 bits need, one in four any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(16, n // 16 * 16)


def draw(rng):
    most = [work(c) for c in listed()]
    flops, nbytes = max(w["flops"] for w in most), max(w["bytes"] for w in most)
    while True:
        op = rng.choice(("i8", "i8", "i8", "i8_swiglu", "checkpoint", "checkpoint", "rows", "norm", "norm",
                         "norm_backward", "norm_backward"))
        c = {"op": op, "dtype": rng.choice(("bf16", "bf16", "fp16"))}
        if op.startswith("i8"):
            dense = op == "i8" and rng.random() < 0.3
            c["E"] = 1 if dense else _log(rng, 1, 256)
            c["k"] = rng.randint(1, min(8, c["E"]))
            c.update(T=_log(rng, 1, 8192), N=_width(rng, 64, 8192), K=_width(rng, 64, 8192),
                     zipf=rng.choice((0.0, 0.6, 1.2)), gather=not dense and op == "i8" and rng.random() < 0.5,
                     scatter=not dense and rng.random() < 0.5)
            c["idle"] = rng.randint(0, (c["E"] - c["k"]) // 4)
        elif op in ("checkpoint", "rows"):
            c.update(R=_log(rng, 1, 65536), I=_width(rng, 64, 8192), block=rng.choice((32, 64, 128)))
        else:
            c.update(T=_log(rng, 1, 16384), H=_width(rng, 64, 8192), gate=rng.choice(("none", "channel", "token")),
                     stream=rng.choice((c["dtype"], "fp32")))
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
    c = case
    if c["op"].startswith("i8"):
        R, N, K = c["T"] * c["k"], c["N"], c["K"]
        # experts that some token chose, on average; rows of x are read once each where they are gathered
        active = sum(1.0 - max(0.0, 1.0 - min(1.0, c["k"] * p)) ** c["T"] for p in _popularity(c))
        active = max(active, float(c["k"]))
        rows = (c["T"] if c["gather"] else R) * (2 if c["op"] == "i8_swiglu" else 1)
        return {"bytes": active * N * (K + 4) + 2.0 * rows * K + 2.0 * R * N, "flops": 2.0 * R * N * K}
    if c["op"] == "checkpoint":
        # z and dh read, h and the gradients written, the checkpoint written and read
        n = float(c["R"]) * c["I"]
        return {"bytes": n * (12 + 4 * (1 + 4.0 / c["block"])), "flops": 40.0 * n}
    if c["op"] == "rows":
        n = float(c["R"]) * c["I"]
        return {"bytes": n * (4 + 2 * (1 + 4.0 / c["block"])), "flops": 8.0 * n}
    n, st = float(c["T"]) * c["H"], 4 if c["stream"] == "fp32" else 2
    gate = 2 * n if c["gate"] == "token" else 0.0
    if c["op"] == "norm":
        return {"bytes": n * (4 + 2 * st) + gate, "flops": 10.0 * n}
    return {"bytes": n * (6 + 3 * st) + 2 * gate, "flops": 30.0 * n}


# ---------------------------------------------------------------------------------------------------------------
# the inputs
# ---------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    c, dt, dev = case, DTYPES[case["dtype"]], "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, mean=0.0, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device=dev).normal_(mean, scale, generator=g)

    s = {"case": c}
    if c["op"].startswith("i8"):
        E, k, T, N, K = c["E"], c["k"], c["T"], c["N"], c["K"]
        if E > 1:
            # k distinct experts a token, drawn by popularity; then the pairs grouped by expert, in pair order within one
            score = torch.tensor(_popularity(c), device=dev).log()
            u = torch.empty(T, E, device=dev).uniform_(1e-6, 1.0 - 1e-6, generator=g)
            ids = (score - (-u.log()).log()).topk(k, dim=1).indices.flatten()
            counts = torch.bincount(ids, minlength=E)
            s["perm"] = torch.argsort(ids, stable=True).to(torch.int32)
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
            s["counts"] = counts.tolist()
        else:
            s["perm"] = torch.arange(T, dtype=torch.int32, device=dev)
            s["offsets"], s["counts"] = None, [T]
        # normal weights, in 8 bits with a scale for each output channel, an expert at a time
        s["w"] = torch.empty(E, N, K, dtype=torch.int8, device=dev)
        s["w_scale"] = torch.empty(E, N, device=dev)
        for e in range(E):
            v = normal(N, K, scale=1.0 / math.sqrt(K), dtype=torch.float32)
            m = v.abs().amax(1)
            s["w"][e] = (v * (127.0 / m)[:, None]).round_().clamp_(-127, 127)
            s["w_scale"][e] = m / 127.0
        # hidden states have a few channels far larger than the rest
        R = T * k
        wide = 1.0 + 7.0 * (torch.arange(K, device=dev) % 97 == 5)
        if c["op"] == "i8":
            s["x"] = normal(T if c["gather"] else R, K).mul_(wide.to(dt))
        else:
            s["z"] = normal(R, 2 * K)
    elif c["op"] == "checkpoint":
        # gate and up as the two halves of one product's output
        s["z"] = normal(c["R"], 2 * c["I"])
        s["dh"] = normal(c["R"], c["I"], scale=0.05)
    elif c["op"] == "rows":
        s["x"] = normal(c["R"], c["I"])
    else:
        T, H, st = c["T"], c["H"], DTYPES[c["stream"]]
        s["o"] = normal(T, H, scale=0.5)
        s["w_after"], s["w_before"] = normal(H, scale=0.1, mean=1.0), normal(H, scale=0.1, mean=1.0)
        s["gate"] = None if c["gate"] == "none" else normal(*([H] if c["gate"] == "channel" else [T, H]), scale=0.3, mean=0.5)
        s["scale"] = 0.875
        if c["op"] == "norm":
            s["residual"] = normal(T, H, scale=2.0, dtype=st)
        else:
            s["s"] = normal(T, H, scale=2.0, dtype=st)
            s["ds"], s["dn"] = normal(T, H, scale=0.05, dtype=st), normal(T, H, scale=0.05)
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def run(state):
    return _call(state) if own else _plain(state)


def _call(s):
    import bit_moe_amd as bm
    c = s["case"]
    op, dt = c["op"], DTYPES[c["dtype"]]
    if op.startswith("i8"):
        w = bm.Rows8(s["w"], s["w_scale"])
        if op == "i8":
            x = bm.quantize_rows(s["x"])
        else:
            x = bm.swiglu_rows8(s["z"][:, :c["K"]], s["z"][:, c["K"]:])
        return bm.expert_matmul_i8(x, w, s["offsets"], x_rows=s["perm"] if c["gather"] else None, x_div=c["k"],
                                   y_rows=s["perm"] if c["scatter"] else None, out_dtype=dt)
    if op == "checkpoint":
        h, gate, up = bm.swiglu_checkpoint(s["z"][:, :c["I"]], s["z"][:, c["I"]:], block=c["block"])
        dgate, dup = bm.swiglu_checkpoint_backward(s["dh"], gate, up)[:2]
        return [h, dgate, dup]
    if op == "rows":
        return bm.dequantize_rows(bm.quantize_rows(s["x"], block=c["block"]), dtype=dt)
    if op == "norm":
        return list(bm.block_norm(s["o"], s["residual"], w_after=s["w_after"], gate=s["gate"], scale=s["scale"],
                                  w_before=s["w_before"], eps=EPS))
    d = bm.block_norm_backward(s["dn"], s["ds"], s["s"], s["o"], w_after=s["w_after"], gate=s["gate"],
                               scale=s["scale"], w_before=s["w_before"], eps=EPS)
    return [d.d_o, d.dresidual, d.dw_after, d.dw_before] + ([] if s["gate"] is None else [d.dgate])


def _codes(x, block=0):
    """(codes, scales) of rows in 8 bits, in float32; the last block may be a part of one."""
    n = x.shape[1]
    b = block or n
    x = torch.nn.functional.pad(x, (0, -n % b)).view(x.shape[0], -1, b)
    m = x.abs().amax(2, keepdim=True)
    return torch.where(m > 0, torch.round(x * 127.0 / m), torch.zeros_like(x)), m / 127.0


def _kept(x, block):
    """What the rows stand for in 8 bits, in float32."""
    q, scale = _codes(x, block)
    return (q * scale).view(x.shape[0], -1)[:, :x.shape[1]]


def _plain(s):
    c = s["case"]
    op, dt = c["op"], DTYPES[c["dtype"]]
    if op.startswith("i8"):
        if op == "i8":
            x = s["x"].float()
        else:
            gate, up = s["z"][:, :c["K"]].float(), s["z"][:, c["K"]:].float()
            x = gate / (1.0 + torch.exp(-gate)) * up
        q, scale = _codes(x)
        return _plain_experts(s, q[:, 0], scale[:, 0], dt)
    if op == "checkpoint":
        gate, up = s["z"][:, :c["I"]].float(), s["z"][:, c["I"]:].float()
        h = (gate / (1.0 + torch.exp(-gate)) * up).to(dt)
        gate, up, dh = _kept(gate, c["block"]), _kept(up, c["block"]), s["dh"].float()
        sig = 1.0 / (1.0 + torch.exp(-gate))
        return [h, (dh * up * sig * (1.0 + gate * (1.0 - sig))).to(dt), (dh * gate * sig).to(dt)]
    if op == "rows":
        return _kept(s["x"].float(), c["block"]).to(dt)
    o, wa, wb = s["o"].float(), s["w_after"].float(), s["w_before"].float()
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    a = torch.rsqrt((o * o).mean(1, keepdim=True) + EPS)
    if op == "norm":
        y = s["scale"] * s["residual"].float() + gate * (o * a * wa)
        b = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        return [y.to(s["residual"].dtype), (y * b * wb).to(dt)]
    y, ds, dn = s["s"].float(), s["ds"].float(), s["dn"].float()
    b = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
    p = dn * wb
    t = ds + b * (p - y * (b * b * (p * y).mean(1, keepdim=True)))
    v = gate * t * wa
    out = [(a * (v - o * (a * a * (v * o).mean(1, keepdim=True)))).to(dt), (s["scale"] * t).to(s["ds"].dtype),
           (gate * t * o * a).sum(0).to(dt), (dn * y * b).sum(0).to(dt)]
    if s["gate"] is not None:
        dg = t * o * a * wa
        out.append((dg.sum(0) if c["gate"] == "channel" else dg).to(dt))
    return out


def _plain_experts(s, q, scale, dt):
    """One product per expert that has rows, on its rows of the gathered operand."""
    c, perm = s["case"], s["perm"].long()
    if c["gather"]:
        q, scale = q[perm // c["k"]], scale[perm // c["k"]]
    out = torch.empty(c["T"] * c["k"], c["N"], dtype=dt, device=q.device)
    r = 0
    for e, n in enumerate(s["counts"]):
        if not n:
            continue
        y = ((q[r:r + n] @ s["w"][e].float().t()) * scale[r:r + n] * s["w_scale"][e]).to(dt)
        if c["scatter"]:
            out[perm[r:r + n]] = y
        else:
            out[r:r + n] = y
        r += n
    return out


# ---------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def _exact_rows8(x, width):
    """Codes and scales of rows in float64, `width` columns a scale."""
    q, scale = torch.zeros_like(x), torch.zeros_like(x)
    for c0 in range(0, x.shape[1], width):
        part = x[:, c0:c0 + width]
        most = part.abs().max(dim=1).values[:, None].expand(part.shape)
        q[:, c0:c0 + width] = torch.div(part * 127, most).round().nan_to_num(nan=0.0)
        scale[:, c0:c0 + width] = most / 127
    return q, scale


def _exact_silu(z):
    """Value and slope."""
    p = torch.sigmoid(z)
    return z * p, p + z * p * (1.0 - p)


def _exact_slices(rows, body):
    """body(r0, r1)'s outputs over slices of rows, so that the 64-bit copies stay small."""
    parts = [body(r, min(r + 4096, rows)) for r in range(0, rows, 4096)]
    return [torch.cat(p) for p in zip(*parts)]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op.startswith("i8"):
        K, perm = c["K"], s["perm"].long()

        def codes(r0, r1):
            if op == "i8":
                v = s["x"][r0:r1].double()
            else:
                v = _exact_silu(s["z"][r0:r1, :K].double())[0] * s["z"][r0:r1, K:].double()
            q, scale = _exact_rows8(v, K)
            return q.to(torch.int8), scale[:, :1]
        q, scale = _exact_slices((s["x"] if op == "i8" else s["z"]).shape[0], codes)
        out = torch.zeros(c["T"] * c["k"], c["N"], dtype=torch.float64, device=q.device)
        starts = [0, c["T"]] if s["offsets"] is None else s["offsets"].tolist()
        for e in range(c["E"]):
            at = torch.arange(starts[e], starts[e + 1], device=q.device)
            if not at.numel():
                continue
            src = torch.div(perm[at], c["k"], rounding_mode="floor") if c["gather"] else at
            val = torch.matmul(q[src].double(), s["w"][e].double().t()) * scale[src] * s["w_scale"][e].double()
            out[perm[at] if c["scatter"] else at] = val
        return out
    if op == "checkpoint":
        I = c["I"]

        def step(r0, r1):
            gate, up = s["z"][r0:r1].double().split(I, dim=1)
            h = _exact_silu(gate)[0] * up
            gate, up = (torch.mul(*_exact_rows8(v, c["block"])) for v in (gate, up))
            v, slope = _exact_silu(gate)
            dh = s["dh"][r0:r1].double()
            return h, dh * up * slope, dh * v
        return _exact_slices(c["R"], step)
    if op == "rows":
        return _exact_slices(c["R"], lambda r0, r1: (torch.mul(*_exact_rows8(s["x"][r0:r1].double(), c["block"])),))[0]
    H, wa, wb = c["H"], s["w_after"].double(), s["w_before"].double()

    def gate_of(r0, r1):
        if s["gate"] is None:
            return torch.ones(1, H, dtype=torch.float64, device=wa.device)
        return s["gate"][r0:r1].double() if c["gate"] == "token" else s["gate"].double()[None]

    def unit(v):
        """The norm's output without weights, and its length."""
        length = (v.square().sum(dim=1, keepdim=True) / H + EPS).sqrt()
        return v / length, length

    if op == "norm":
        def forward(r0, r1):
            y = unit(s["o"][r0:r1].double())[0] * wa * gate_of(r0, r1) + s["scale"] * s["residual"][r0:r1].double()
            return y, unit(y)[0] * wb
        return _exact_slices(c["T"], forward)
    sums = [torch.zeros(H, dtype=torch.float64, device=wa.device) for _ in range(3)]

    def into_norm(dv, v, length):
        """The gradient of unit()'s input."""
        return (dv - v * (dv * v).sum(dim=1, keepdim=True) / H) / length

    def backward(r0, r1):
        v, long_v = unit(s["o"][r0:r1].double())
        y, long_y = unit(s["s"][r0:r1].double())
        dn, gate = s["dn"][r0:r1].double(), gate_of(r0, r1)
        t = s["ds"][r0:r1].double() + into_norm(dn * wb, y, long_y)
        dg = t * v * wa
        for total, term in zip(sums, (t * gate * v, dn * y, dg)):
            total += term.sum(dim=0)
        return into_norm(t * gate * wa, v, long_v), t * s["scale"], dg
    d_o, dres, dg = _exact_slices(c["T"], backward)
    out = [d_o, dres, sums[0], sums[1]]
    return out + ([] if s["gate"] is None else [dg if c["gate"] == "token" else sums[2]])
