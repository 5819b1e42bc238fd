"""The operators of an MoE layer around its expert GEMMs, as cases to be timed.

Four operators, each in the form in which a program with 4-bit experts calls it:

* ``matvec``   few tokens times the routed experts' MXFP4 weights (decoding), plain or with
               the SwiGLU of a gate/up projection as its epilogue;
* ``tokens``   token rows sorted by expert and back with the router's weights, and the
               gradients of both directions;
* ``swiglu``   the activation between an expert's two projections, written as the next GEMM's
               FP8 input, with an 8-bit checkpoint of its own input, and the backward pass
               from that checkpoint;
* ``router``   the top-k softmax gate and its gradient.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the
library's kernels.
"""
import math

import torch

own = False

W_GROUP = 32        # weights of one E8M0 scale
A_GROUP = 128       # activations of one E8M0 scale
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------- cases --

def listed():
    return [
        # The smallest call: one token through one dense 4-bit projection of odd height.
        dict(name="matvec dense small", op="matvec", M=1, k=1, E=1, N=500, K=640, per_slot=False,
             swiglu=False),
        # Decoding one token: gate and up projection of its eight experts, SwiGLU fused.
        dict(name="matvec gate-up 1 token", op="matvec", M=1, k=8, E=32, N=4096, K=6144,
             per_slot=False, swiglu=True),
        # The same token's down projection: every expert has an input row of its own.
        dict(name="matvec down 1 token", op="matvec", M=1, k=8, E=32, N=6144, K=2048,
             per_slot=True, swiglu=False),
        # A small decoding batch on few experts: each expert's weights serve several tokens.
        dict(name="matvec batch 13", op="matvec", M=13, k=8, E=12, N=6144, K=3584,
             per_slot=False, swiglu=False),
        # A prompt's tokens copied into expert order.
        dict(name="dispatch prompt", op="tokens", way="dispatch", M=768, k=8, E=32, N=6144,
             weighted=False, drop=0.0),
        # Gradient of a weighted dispatch for a short odd batch, some ids dropped by the router.
        dict(name="dispatch bwd short", op="tokens", way="dispatch_bwd", M=37, k=4, E=64, N=2056,
             weighted=True, drop=0.2),
        # Gradient of the combine at a training batch's size: the largest case.
        dict(name="combine bwd train", op="tokens", way="combine_bwd", M=16384, k=8, E=32, N=6144,
             weighted=True, drop=0.0),
        # Serving: the activation of a few routed rows, nothing kept for a backward pass.
        dict(name="swiglu serve", op="swiglu", way="fwd", R=40, F=2048, checkpoint=False),
        # Training: the activation of a whole batch's routed rows with its 8-bit checkpoint.
        dict(name="swiglu train", op="swiglu", way="fwd", R=131072, F=2048, checkpoint=True),
        # The backward pass from the checkpoint, an odd number of rows.
        dict(name="swiglu bwd", op="swiglu", way="bwd", R=9223, F=2048, checkpoint=True),
        # Serving: the gate of a handful of tokens.
        dict(name="router serve", op="router", way="fwd", M=5, E=32, k=8, renorm=True,
             masked=False),
        # Training: gate and gradient for a batch, some experts masked out per token.
        dict(name="router train", op="router", way="train", M=16384, E=160, k=6, renorm=False,
             masked=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("matvec", "tokens", "swiglu", "router"))
    if op == "matvec":
        while True:
            E = rng.choice((1, 2, 4, 8, 12, 16, 32, 64))
            M = _log_int(rng, 1, 16)
            k = rng.randint(1, min(8, E))
            swiglu = rng.random() < 0.5
            N = _log_int(rng, 64, 8192)
            N += N % 2 if swiglu else 0
            K = 128 * _log_int(rng, 1, 56)
            if E * N * K <= 1 << 30 and N != 3072 and K != 3072:
                return dict(op=op, M=M, k=k, E=E, N=N, K=K,
                            per_slot=rng.random() < 0.5, swiglu=swiglu)
    if op == "tokens":
        while True:
            M, E = _log_int(rng, 1, 16384), rng.choice((8, 12, 32, 64))
            k = rng.randint(1, 8)
            N = 8 * _log_int(rng, 16, 1024)
            way = rng.choice(("dispatch", "dispatch_bwd", "combine_bwd"))
            if M * k * N <= 16384 * 8 * 6144 and 3072 not in (M, N):
                return dict(op=op, way=way, M=M, k=k, E=E, N=N,
                            weighted=way == "combine_bwd" or rng.random() < 0.5,
                            drop=0.1 if way == "dispatch_bwd" and rng.random() < 0.5 else 0.0)
    if op == "swiglu":
        while True:
            R, F = _log_int(rng, 1, 131072), 128 * _log_int(rng, 1, 64)
            if R * F <= 131072 * 2048 and 3072 not in (R, F):
                way = rng.choice(("fwd", "bwd"))
                return dict(op=op, way=way, R=R, F=F,
                            checkpoint=way == "bwd" or rng.random() < 0.5)
    M = _log_int(rng, 1, 16384)
    E = _log_int(rng, 4, 512)
    return dict(op=op, way=rng.choice(("fwd", "train")), M=M + (M == 3072), E=E,
                k=rng.randint(1, min(8, E)), renorm=rng.random() < 0.5,
                masked=rng.random() < 0.5)


def work(case):
    c = case
    if c["op"] == "matvec":
        slots = c["M"] * c["k"]
        touched = c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["M"])   # experts of M random tokens
        out = slots * (c["N"] // 2 if c["swiglu"] else c["N"])
        weights = touched * c["N"] * (c["K"] / 2 + c["K"] / W_GROUP)
        x = (slots if c["per_slot"] else c["M"]) * c["K"]
        return {"bytes": weights + 2 * x + 4 * slots + 2 * out,
                "flops": 2.0 * slots * c["N"] * c["K"]}
    if c["op"] == "tokens":
        rows, n = c["M"] * c["k"], c["N"]
        kept = rows * (1.0 - c["drop"])
        index = rows * (4 + (4 if c["weighted"] else 0))
        if c["way"] == "dispatch":
            return {"bytes": 2.0 * n * (c["M"] + rows) + index, "flops": 1.0 * rows * n}
        if c["way"] == "dispatch_bwd":
            x = 2.0 * n * c["M"] + 4 * rows if c["weighted"] else 0.0
            return {"bytes": 2.0 * n * (kept + c["M"]) + x + index,
                    "flops": (4.0 if c["weighted"] else 1.0) * kept * n}
        return {"bytes": 2.0 * n * (c["M"] + 2 * rows) + index + 4 * rows,
                "flops": 3.0 * rows * n}
    if c["op"] == "swiglu":
        n = c["R"] * c["F"]
        if c["way"] == "bwd":
            return {"bytes": n * (2 + 2 + 2 / A_GROUP + 4), "flops": 12.0 * n}
        kept = (2 + 2 / A_GROUP) if c["checkpoint"] else 0
        return {"bytes": n * (4 + 1 + 1 / A_GROUP + kept), "flops": 8.0 * n}
    n = c["M"] * c["E"]
    if c["way"] == "fwd":
        return {"bytes": 4.0 * n + 8 * c["M"] * c["k"], "flops": 4.0 * n}
    return {"bytes": 8.0 * n + 12 * c["M"] * c["k"], "flops": 8.0 * n}


# ---------------------------------------------------------------- inputs --

def _pow2_exponent(amax, qmax):
    """Smallest integer e with amax <= qmax * 2^e, 0 for amax = 0, in [-127, 127]."""
    a = amax.double()
    safe = torch.where(a > 0, a, torch.ones_like(a))
    e = torch.ceil(torch.log2(safe / qmax))
    e = torch.where(safe > qmax * torch.exp2(e), e + 1, e)
    e = torch.where(safe <= qmax * torch.exp2(e - 1), e - 1, e)
    return torch.where(a > 0, e, torch.zeros_like(e)).clamp(-127, 127).to(torch.int32)


def _quantize_weights(w):
    """FP32 [N, K] -> E2M1 codes packed two to a byte, E8M0 codes of 32-element groups."""
    N, K = w.shape
    g = w.view(N, K // W_GROUP, W_GROUP)
    e = _pow2_exponent(g.abs().amax(-1), 6.0)
    q = torch.ldexp(g, -e.unsqueeze(-1))
    mid = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=w.device)
    code = torch.bucketize(q.abs(), mid).to(torch.uint8) | ((q < 0).to(torch.uint8) << 3)
    code = code.view(N, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _quantize_acts(x):
    """FP32 [R, K] -> E4M3 codes [R, K], E8M0 codes [R, K/128] (both as bytes)."""
    R, K = x.shape
    g = x.view(R, K // A_GROUP, A_GROUP)
    e = _pow2_exponent(g.abs().amax(-1), 448.0)
    codes = torch.ldexp(g, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).view(R, K), (e + 127).to(torch.uint8)


def _decode_acts(codes, scale):
    R, K = codes.shape
    v = codes.view(torch.float8_e4m3fn).float().view(R, K // A_GROUP, A_GROUP)
    return torch.ldexp(v, (scale.int() - 127).unsqueeze(-1)).view(R, K)


def _routing(gen, M, E, k, drop):
    """Expert ids of M tokens (k distinct ones each, unevenly loaded) and the place of each
    (token, choice) in the rows sorted by expert; -1 for ids that a router dropped."""
    logits = torch.randn(M, E, generator=gen, device="cuda")
    logits += torch.randn(E, generator=gen, device="cuda")
    ids = torch.argsort(logits, dim=1, descending=True)[:, :k]
    if drop:
        ids = torch.where(torch.rand(M, k, generator=gen, device="cuda") < drop, E, ids)
    flat = ids.reshape(-1)
    place = torch.empty_like(flat)
    place[torch.argsort(flat, stable=True)] = torch.arange(flat.numel(), device="cuda")
    place = torch.where(flat < E, place, -1)
    return ids.to(torch.int32).contiguous(), place.to(torch.int32)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"case": c}
    if c["op"] == "matvec":
        s["ids"], _ = _routing(gen, c["M"], c["E"], c["k"], 0.0)
        s["x"] = normal(c["M"] * (c["k"] if c["per_slot"] else 1), c["K"]).bfloat16()
        s["w"] = torch.empty(c["E"], c["N"], c["K"] // 2, dtype=torch.uint8, device="cuda")
        s["ws"] = torch.empty(c["E"], c["N"], c["K"] // W_GROUP, dtype=torch.uint8, device="cuda")
        for e in range(c["E"]):
            s["w"][e], s["ws"][e] = _quantize_weights(normal(c["N"], c["K"]) / c["K"] ** 0.5)
    elif c["op"] == "tokens":
        _, s["place"] = _routing(gen, c["M"], c["E"], c["k"], c["drop"])
        w = torch.softmax(normal(c["M"], c["k"]), dim=1)
        s["weights"] = w.contiguous() if c["weighted"] else None
        s["token"] = normal(c["M"], c["N"]).bfloat16()
        if c["way"] != "dispatch":
            s["rows"] = normal(c["M"] * c["k"], c["N"]).bfloat16()
    elif c["op"] == "swiglu":
        if c["way"] == "fwd":
            s["z"] = (1.5 * normal(c["R"], 2 * c["F"])).bfloat16()
        else:
            z = (1.5 * normal(c["R"], 2 * c["F"])).bfloat16().float()
            s["zq"], s["zs"] = _quantize_acts(z)
            s["dh"] = normal(c["R"], c["F"]).bfloat16()
    else:
        logits = 2.0 * normal(c["M"], c["E"])
        if c["masked"]:   # some experts are closed to a token; some tokens have too few, or none
            closed = torch.rand(c["M"], c["E"], generator=gen, device="cuda") < 0.3
            closed[2::16] |= (torch.arange(c["E"], device="cuda") >= c["k"] // 2)[None, :]
            closed[5::16] = True
            logits = torch.where(closed, -math.inf, logits)
        s["logits"] = logits.contiguous()
        s["dw"] = normal(c["M"], c["k"])
    return s


# ---------------------------------------------------------- plain forms --

def _plain_matvec(s):
    c, ids = s["case"], s["ids"].long().reshape(-1)
    values = torch.tensor(E2M1_VALUES, device="cuda")
    values = torch.cat([values, -values])
    gather = ids.numel() <= c["E"]            # else every expert is widened once
    w, ws = (s["w"][ids], s["ws"][ids]) if gather else (s["w"], s["ws"])
    W = values[torch.stack([w & 15, w >> 4], dim=-1).int()].view(-1, c["N"], c["K"] // W_GROUP,
                                                                 W_GROUP)
    W = torch.ldexp(W, (ws.int() - 127).unsqueeze(-1)).view(-1, c["N"], c["K"])
    x = s["x"].float()
    x = x if c["per_slot"] else x.repeat_interleave(c["k"], dim=0)
    if gather:
        y = torch.bmm(W, x.unsqueeze(-1)).squeeze(-1)
    else:
        y = torch.matmul(x, W.transpose(1, 2))[ids, torch.arange(ids.numel(), device="cuda")]
    if c["swiglu"]:
        g, u = y.chunk(2, dim=1)
        y = g / (1 + torch.exp(-g)) * u
    return y.bfloat16()


def _plain_tokens(s):
    c, place = s["case"], s["place"].long()
    M, k, N = c["M"], c["k"], c["N"]
    ok = (place >= 0).float().view(M, k, 1)
    w = s["weights"].view(M, k, 1) if c["weighted"] else 1.0
    token = s["token"].float().view(M, 1, N)
    if c["way"] == "dispatch":
        out = torch.empty(M * k, N, dtype=torch.bfloat16, device="cuda")
        out[place] = (token * w).expand(M, k, N).reshape(M * k, N).bfloat16()
        return out
    rows = s["rows"][place.clamp(min=0)].float().view(M, k, N) * ok
    dw = (rows * token).sum(-1)
    if c["way"] == "dispatch_bwd":
        dx = (rows * w).sum(1).bfloat16()
        return (dx, dw) if c["weighted"] else (dx,)
    dy = torch.empty(M * k, N, dtype=torch.bfloat16, device="cuda")
    dy[place] = (token * w).reshape(M * k, N).bfloat16()
    return dy, dw


def _typed(codes, scale):
    """Bytes as the number formats that they are."""
    return codes.view(torch.float8_e4m3fn), scale.view(torch.float8_e8m0fnu)


def _plain_quantize(x):
    R, K = x.shape
    g = x.view(R, K // A_GROUP, A_GROUP)
    m, p = torch.frexp(g.abs().amax(-1))                 # amax = m * 2^p, m in [0.5, 1)
    e = torch.where(m > 0, p - 9 + (m > 0.875).int(), 0).clamp(-127, 127)
    codes = torch.ldexp(g, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(R, K)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _plain_swiglu(s):
    c = s["case"]
    if c["way"] == "fwd":
        z = s["z"].float()
        g, u = z.chunk(2, dim=1)
        h = _plain_quantize(g / (1 + torch.exp(-g)) * u)
        return (*_typed(*h), *_typed(*_plain_quantize(z))) if c["checkpoint"] else _typed(*h)
    g, u = _decode_acts(s["zq"], s["zs"]).chunk(2, dim=1)
    dh = s["dh"].float()
    sig = 1 / (1 + torch.exp(-g))
    return torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], dim=1).bfloat16()


def _plain_router(s):
    c, logits = s["case"], s["logits"]
    top = logits.amax(1, keepdim=True)
    p = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    p = p / p.sum(1, keepdim=True).clamp(min=1e-38)
    value, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    value, ids = value[:, :c["k"]], ids[:, :c["k"]]
    none = value == -math.inf
    w = torch.where(none, 0.0, p.gather(1, ids))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-38)
    said = torch.where(none, -1, ids).to(torch.int32)
    if c["way"] == "fwd":
        return said, w
    dw = torch.where(none, 0.0, s["dw"])
    inner = (w * dw).sum(1, keepdim=True)
    if c["renorm"]:
        d = torch.zeros_like(logits).scatter_add(1, ids, w * (dw - inner))
    else:
        d = torch.zeros_like(logits).scatter_add(1, ids, w * dw) - p * inner
    return said, w, d


# -------------------------------------------------------- library calls --

def _own(s):
    from fp8_mxfp4_grouped_gb300 import hg
    c = s["case"]
    if c["op"] == "matvec":
        f = hg.hg_expert_matvec_swiglu if c["swiglu"] else hg.hg_expert_matvec
        return f(s["x"], s["ids"], s["w"], s["ws"])
    if c["op"] == "tokens":
        if c["way"] == "dispatch":
            return hg.hg_dispatch_tokens(s["token"], c["k"], s["place"], s["weights"])
        if c["way"] == "dispatch_bwd":
            if c["weighted"]:
                return hg.hg_dispatch_tokens_bwd(s["rows"], c["k"], s["place"], s["weights"],
                                                 s["token"])
            return hg.hg_dispatch_tokens_bwd(s["rows"], c["k"], s["place"])[:1]
        return hg.hg_combine_topk_bwd(s["token"], s["rows"], s["place"], s["weights"])
    if c["op"] == "swiglu":
        if c["way"] == "bwd":
            return hg.hg_swiglu_bwd(s["dh"], s["zq"], s["zs"])
        a, asc, zq, zs = hg.hg_swiglu_quantize(s["z"], c["checkpoint"])
        return (*_typed(a, asc), *_typed(zq, zs)) if c["checkpoint"] else _typed(a, asc)
    ids, w = hg.hg_router_topk(s["logits"], c["k"], c["renorm"])
    if c["way"] == "fwd":
        return ids, w
    return ids, w, hg.hg_router_topk_bwd(s["logits"], ids, w, s["dw"], c["renorm"])


def run(state):
    if own:
        return _own(state)
    return {"matvec": _plain_matvec, "tokens": _plain_tokens, "swiglu": _plain_swiglu,
            "router": _plain_router}[state["case"]["op"]](state)


# ------------------------------------------------------ in 64 bits -------

def _exact_e4m3(q):
    """Nearest E4M3 value, ties to even, of |q| <= 448."""
    _, p = torch.frexp(q)
    step = torch.exp2((p.double() - 1).clamp(min=-6) - 3)
    return torch.round(q / step) * step


def _exact_quantize(x):
    R, K = x.shape
    g = x.view(R, K // A_GROUP, A_GROUP)
    e = _pow2_exponent(g.abs().amax(-1), 448.0).double()
    return _exact_e4m3(g * torch.exp2(-e).unsqueeze(-1)).view(R, K), torch.exp2(e)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "matvec":
        flat = s["ids"].reshape(-1).tolist()
        sign = torch.tensor((1.0, -1.0), dtype=torch.float64, device="cuda")
        mag = torch.tensor(E2M1_VALUES, dtype=torch.float64, device="cuda")
        y = torch.empty(len(flat), c["N"], dtype=torch.float64, device="cuda")
        for e in sorted(set(flat)):
            byte = s["w"][e].long()
            W = torch.empty(c["N"], c["K"], dtype=torch.float64, device="cuda")
            W[:, 0::2] = mag[byte & 7] * sign[(byte >> 3) & 1]
            W[:, 1::2] = mag[(byte >> 4) & 7] * sign[byte >> 7]
            W *= torch.exp2(s["ws"][e].double() - 127).repeat_interleave(W_GROUP, dim=1)
            at = [i for i, f in enumerate(flat) if f == e]
            x = s["x"][[i if c["per_slot"] else i // c["k"] for i in at]].double()
            y[at] = x @ W.T
        if c["swiglu"]:
            g, u = y[:, :c["N"] // 2], y[:, c["N"] // 2:]
            y = u * g * torch.sigmoid(g)
        return y
    if c["op"] == "tokens":
        M, k, N = c["M"], c["k"], c["N"]
        place = s["place"].view(M, k).long()
        w = s["weights"].double() if c["weighted"] else torch.ones(M, k, dtype=torch.float64,
                                                                   device="cuda")
        token = s["token"].double()
        if c["way"] != "dispatch_bwd":
            placed = torch.zeros(M * k, N, dtype=torch.float64, device="cuda")
            for j in range(k):
                placed[place[:, j]] = token * w[:, j:j + 1]
            if c["way"] == "dispatch":
                return placed
        dx = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        dw = torch.zeros(M, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            here = place[:, j] >= 0
            rows = s["rows"][place[here, j]].double()
            dx[here] += w[here, j:j + 1] * rows
            dw[here, j] = torch.einsum("tn,tn->t", rows, token[here])
        if c["way"] == "combine_bwd":
            return placed, dw
        return (dx, dw) if c["weighted"] else (dx,)
    if c["op"] == "swiglu":
        if c["way"] == "fwd":
            z = s["z"].double()
            h = z[:, :c["F"]] * torch.sigmoid(z[:, :c["F"]]) * z[:, c["F"]:]
            out = _exact_quantize(h)
            return (*out, *_exact_quantize(z)) if c["checkpoint"] else out
        z = s["zq"].view(torch.float8_e4m3fn).double()
        z = z * torch.exp2(s["zs"].double() - 127).repeat_interleave(A_GROUP, dim=1)
        g, u, dh = z[:, :c["F"]], z[:, c["F"]:], s["dh"].double()
        sig = torch.sigmoid(g)
        return torch.cat([dh * u * (sig + g * sig * (1 - sig)), dh * g * sig], dim=1)
    logits = s["logits"].double()
    open_ = logits > -math.inf
    p = torch.nan_to_num(torch.softmax(logits, dim=1), nan=0.0)
    chosen = torch.argsort(-logits, dim=1, stable=True)[:, :c["k"]]
    there = open_.gather(1, chosen)
    w = p.gather(1, chosen) * there
    total = w.sum(1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total))
    v = w / total if c["renorm"] else w
    ids = torch.where(there, chosen, -1).to(torch.int32)
    if c["way"] == "fwd":
        return ids, v
    dw = s["dw"].double() * there
    # d loss / d p of the chosen, then through the softmax over all experts
    dp = (dw - (v * dw).sum(1, keepdim=True)) / total if c["renorm"] else dw
    full = torch.zeros_like(p).scatter(1, chosen, dp * there)
    return ids, v, p * (full - (p * full).sum(1, keepdim=True))
