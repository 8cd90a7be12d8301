"""The operators between the products of a block-quantized model, as measured
cases: the norm of the residual stream, the gated activation, each with the
output in the type that the next product reads, and the router of experts with
scores, a bias and groups.

`run` makes one pass through an operator: with ``own`` false in elementary
torch operations (32-bit; 64-bit for sums over a row or over experts and for
the scores that experts are chosen by), with ``own`` true through this
package's binding. `exact` computes the same outputs from the definitions in
64 bits.

Kinds of case:
  norm   h[m] = residual[m] + sum_j weights[m, j] x[m share + j] (a weight of 0
         leaves its row out), y = h / sqrt(mean(h^2) + eps) * gamma. h is
         written back as the new residual, y in f32 or bfloat16, as Q8_0 blocks
         or as E4M3 codes with a scale for each 128 columns.
  act    y = f(gate) * up with f SiLU or GELU (tanh form), gate and up the
         halves of one product's rows; y as above.
  route  scores s of E experts (softmax or sigmoid of the logits), the top_k
         experts by s + bias among the top_groups groups of neighbouring
         experts, a group ranked by the sum of its group_best largest; weights
         scale * s (over the chosen ones' sum with renorm), and the slots
         (t, j) sorted by expert.

Q8_0 outputs are returned as their values in binary16, E4M3 codes as
torch.float8_e4m3fn beside their scales.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-5


# ---------------------------------------------------------------------------
# Cases. Sizes: the 4096- and 14336-wide projections that this repository's
# benchmark multiplies; experts as its router's cases, and 256 in 8 groups.

def listed():
    return [
        # One token before an attention product over Q8_0 activations: latency.
        {"name": "norm f32 to q8 1x4096", "kind": "norm", "M": 1, "K": 4096, "share": 1, "residual": True, "act": "f32", "out": "q8", "dense": False},
        # 37 decoding tokens after their two experts: the experts' sum, the residual and the norm in one.
        {"name": "norm bf16 to f8 37x4096 of 2", "kind": "norm", "M": 37, "K": 4096, "share": 2, "residual": True, "act": "bf16", "out": "f8", "dense": True},
        # A prompt of odd length before an 8-bit product.
        {"name": "norm bf16 to f8 1001x4096", "kind": "norm", "M": 1001, "K": 4096, "share": 1, "residual": True, "act": "bf16", "out": "f8", "dense": False},
        # A 2048-token prompt after its two experts of 4-bit weights, whose products are f32.
        {"name": "norm f32 to bf16 2048x4096 of 2", "kind": "norm", "M": 2048, "K": 4096, "share": 2, "residual": True, "act": "f32", "out": "bf16", "dense": False},
        # The first norm of a model: no residual yet, f32 products next.
        {"name": "norm f32 to f32 300x4096", "kind": "norm", "M": 300, "K": 4096, "share": 1, "residual": False, "act": "f32", "out": "f32", "dense": False},
        # One token's two experts between their up and down products.
        {"name": "act bf16 to f8 2x14336", "kind": "act", "M": 2, "K": 14336, "f": "silu", "act": "bf16", "out": "f8"},
        # A batch of 37 tokens, 4-bit weights, Q8_0 activations next.
        {"name": "act f32 to q8 37x14336", "kind": "act", "M": 37, "K": 14336, "f": "gelu", "act": "f32", "out": "q8"},
        # A 1001-token prompt of a dense layer with 4-bit weights over bfloat16 activations.
        {"name": "act f32 to bf16 1001x14336", "kind": "act", "M": 1001, "K": 14336, "f": "silu", "act": "f32", "out": "bf16"},
        # The rows of a 2048-token prompt's two experts each.
        {"name": "act bf16 to f8 4096x14336", "kind": "act", "M": 4096, "K": 14336, "f": "silu", "act": "bf16", "out": "f8"},
        # A decoding batch at the router of many experts in groups.
        {"name": "route sigmoid 32 tokens 8 of 256", "kind": "route", "T": 32, "E": 256, "top_k": 8, "score": "sigmoid", "bias": True, "n_groups": 8, "top_groups": 4, "group_best": 2, "renorm": True, "scale": 2.5},
        # A long prompt at the same router.
        {"name": "route sigmoid 8192 tokens 8 of 256", "kind": "route", "T": 8192, "E": 256, "top_k": 8, "score": "sigmoid", "bias": True, "n_groups": 8, "top_groups": 4, "group_best": 2, "renorm": True, "scale": 2.5},
        # A prompt at a router with softmax scores and a bias, no groups.
        {"name": "route softmax 2048 tokens 6 of 64", "kind": "route", "T": 2048, "E": 64, "top_k": 6, "score": "softmax", "bias": True, "n_groups": 1, "top_groups": 1, "group_best": 1, "renorm": True, "scale": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "act", "act", "route"])
    act = rng.choice(["f32", "bf16"])
    out = rng.choice(["f32", "bf16", "q8", "f8", "f8"])
    if kind == "norm":
        K, share = 32 * _log(rng, 4, 448), rng.choice([1, 1, 1, 2, 4, 6, 8])
        most = min(4096, 16_000_000 // (K * share))
        return {"kind": kind, "M": _log(rng, 1, most), "K": K, "share": share, "residual": rng.random() < 0.8, "act": act, "out": out,
                "dense": out in ("q8", "f8") and rng.random() < 0.4}
    if kind == "act":
        K = 32 * _log(rng, 8, 448)
        return {"kind": kind, "M": _log(rng, 1, min(4096, 24_000_000 // K)), "K": K, "f": rng.choice(["silu", "silu", "gelu"]), "act": act, "out": out}
    G = rng.choice([1, 1, 4, 8])
    E = G * rng.choice([5, 8, 16, 32]) * rng.choice([1, 2] if G > 1 else [2, 8])
    top = rng.choice([g for g in (1, 2, 4, 8) if g <= G])
    return {"kind": kind, "T": _log(rng, 1, 8192), "E": E, "top_k": rng.choice([k for k in (1, 2, 4, 6, 8) if k <= top * E // G]),
            "score": rng.choice(["sigmoid", "sigmoid", "softmax"]), "bias": rng.random() < 0.8, "n_groups": G, "top_groups": top,
            "group_best": rng.choice([1, 2]), "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5])}


ACT_BYTES = {"f32": 4, "bf16": 2}


def _out_bytes(out, M, K):
    if out == "q8":
        return M * K // 32 * 34
    return M * K + 4 * M * -(-K // 128) if out == "f8" else M * K * ACT_BYTES[out]


def work(case):
    c = case
    if c["kind"] == "norm":
        M, K, e = c["M"], c["K"], ACT_BYTES[c["act"]]
        rows = c["share"] + (2 if c["residual"] or c["share"] > 1 else 0) - (0 if c["residual"] else (1 if c["share"] > 1 else 0))
        weights = 4 * M * c["share"] if c["share"] > 1 else 0
        return {"bytes": M * K * e * (rows + c["dense"]) + weights + 4 * K + _out_bytes(c["out"], M, K), "flops": M * K * (2 * c["share"] + 5)}
    if c["kind"] == "act":
        M, K = c["M"], c["K"]
        return {"bytes": 2 * M * K * ACT_BYTES[c["act"]] + _out_bytes(c["out"], M, K), "flops": 8 * M * K}
    S = c["T"] * c["top_k"]
    return {"bytes": 4 * c["T"] * c["E"] + (4 * c["E"] if c["bias"] else 0) + 12 * S + 4 * (c["E"] + 1), "flops": 24 * c["T"] * c["E"]}


# ---------------------------------------------------------------------------
# What a program has in hand before the call.

def _hidden(g, M, K, dev):
    """Hidden states: N(0, 1) with a few channels of larger spread and rows of differing size."""
    x = torch.randn(M, K, generator=g, device=dev)
    x *= 1 + 9 * (torch.rand(1, K, generator=g, device=dev) < 0.01)
    return x * torch.exp(0.5 * torch.randn(M, 1, generator=g, device=dev))


def _outputs(st, c, dev):
    """The buffers that a program keeps for the result."""
    M, K = c["M"], c["K"]
    if c["out"] == "q8":
        st["q"] = torch.empty(M, K // 32, 34, dtype=torch.uint8, device=dev)
    elif c["out"] == "f8":
        st["q"] = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=dev)
        st["s"] = torch.empty(M, -(-K // 128), device=dev)
    else:
        st["y"] = torch.empty(M, K, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c, st = case, {"case": case}
    if c["kind"] == "route":
        T, E = c["T"], c["E"]
        # Some experts are liked more than others; the bias evens them out.
        like = 0.5 * torch.randn(1, E, generator=g, device=dev)
        st["logits"] = torch.randn(T, E, generator=g, device=dev) + like
        st["bias"] = (-0.1 * like[0] + 0.02 * torch.randn(E, generator=g, device=dev)).contiguous() if c["bias"] else None
        S = T * c["top_k"]
        st["ids"] = torch.empty(S, dtype=torch.int32, device=dev)
        st["weights"] = torch.empty(S, device=dev)
        st["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=dev)
        st["order"] = torch.empty(S, dtype=torch.int32, device=dev)
        return st
    M, K = c["M"], c["K"]
    dtype = torch.bfloat16 if c["act"] == "bf16" else torch.float32
    if c["kind"] == "act":
        st["x"] = _hidden(g, M, 2 * K, dev).to(dtype)      # one product's rows: the gate, then the up half
    else:
        st["x"] = _hidden(g, M * c["share"], K, dev).to(dtype)
        st["residual"] = (3 * _hidden(g, M, K, dev)).to(dtype) if c["residual"] else None
        st["sum"] = torch.empty(M, K, dtype=dtype, device=dev) if c["residual"] or c["share"] > 1 else None
        st["gamma"] = 1 + 0.2 * torch.randn(K, generator=g, device=dev)
        st["weights"] = None
        if c["share"] > 1:
            st["weights"] = torch.softmax(torch.randn(M, c["share"], generator=g, device=dev), 1).contiguous()
        st["dense"] = torch.empty(M, K, dtype=dtype, device=dev) if c["dense"] else None
    _outputs(st, c, dev)
    return st


# ---------------------------------------------------------------------------
# One pass.

def _q8_values(codes, d):
    """int8-ranged codes [M, K / 32, 32] and binary16 scales -> their values, in binary16."""
    return codes * d


def _written(y, out):
    """y [M, K] in f32 in the form `out`."""
    M, K = y.shape
    if out == "f32":
        return [y]
    if out == "bf16":
        return [y.to(torch.bfloat16)]
    if out == "q8":
        b = y.reshape(M, K // 32, 32)
        d = b.abs().amax(-1, keepdim=True) / 127
        v = b / torch.where(d == 0, torch.ones_like(d), d)
        q = (torch.sign(v) * torch.floor(v.abs() + 0.5)).to(torch.int8)
        return [_q8_values(q, d.to(torch.float16))]
    Kp = -(-K // 128) * 128
    b = (torch.nn.functional.pad(y, (0, Kp - K)) if Kp != K else y).reshape(M, Kp // 128, 128)
    s = b.abs().amax(-1) / E4M3_MAX
    q = (b / torch.where(s == 0, torch.ones_like(s), s)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return [q.reshape(M, Kp)[:, :K].contiguous(), s]


def _group(ids, E):
    """Expert of each slot -> offsets [E + 1] and the slots in expert order, both int32; equal experts keep their order."""
    order = torch.sort(ids, stable=True)[1].to(torch.int32)
    bounds = torch.arange(E + 1, device=ids.device)
    return (ids[None, :] < bounds[:, None]).sum(1).to(torch.int32), order


def _route(st, c):
    """Scores in 64 bits: experts whose keys are a rounding apart are told apart."""
    T, E, G = c["T"], c["E"], c["n_groups"]
    x = st["logits"].double()
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-x))
    else:
        s = torch.exp(x - x.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    key = s + st["bias"].double() if c["bias"] else s
    if c["top_groups"] < G:
        best = torch.sort(key.reshape(T, G, E // G), dim=2, descending=True)[0][:, :, :c["group_best"]].sum(2)
        keep = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, keep, True)
        key = torch.where(kept.repeat_interleave(E // G, 1), key, -math.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :c["top_k"]]
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    offsets, order = _group(ids.reshape(-1), E)
    return [ids.reshape(-1).to(torch.int32), (w * c["scale"]).float().reshape(-1), offsets, order]


def run(state):
    st, c = state, state["case"]
    if own:
        return _run_own(st, c)
    if c["kind"] == "route":
        return _route(st, c)
    if c["kind"] == "act":
        x = st["x"].float()
        g, u = x[:, :c["K"]], x[:, c["K"]:]
        z = g if c["f"] == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)
        return _written(g / (1 + torch.exp(-z)) * u, c["out"])
    M, K, dtype = c["M"], c["K"], st["x"].dtype
    if c["share"] > 1:
        w = st["weights"].double()[:, :, None]
        h = torch.where(w == 0, 0.0, w * st["x"].reshape(M, c["share"], K).double()).sum(1)
        if st["residual"] is not None:
            h = h + st["residual"].double()
        h = h.float()
    else:
        h = st["x"].float()
        if st["residual"] is not None:
            h = h + st["residual"].float()
    rstd = (1 / torch.sqrt(h.double().square().mean(1, keepdim=True) + EPS)).float()
    y = h * rstd * st["gamma"]
    out = _written(y, c["out"])
    if st["dense"] is not None:
        out.append(y.to(dtype))
    if st["sum"] is not None:
        out.append(h.to(dtype))
    return out


def _values_of(blocks):
    """Q8_0 blocks -> their values in binary16."""
    return _q8_values(blocks[..., 2:].view(torch.int8), blocks[..., :2].view(torch.float16))


def _run_own(st, c):
    from block_quantized_weight_dequant_amd import binding as q4
    if c["kind"] == "route":
        q4.q4_route_groups(st["logits"], st["bias"], st["ids"], st["weights"], st["offsets"], st["order"], c["T"], c["E"], c["top_k"],
                           q4.Q4_SCORE_SIGMOID if c["score"] == "sigmoid" else q4.Q4_SCORE_SOFTMAX, c["n_groups"], c["top_groups"],
                           c["group_best"], c["renorm"], c["scale"])
        return [st["ids"], st["weights"], st["offsets"], st["order"]]
    M, K, tail = c["M"], c["K"], "_bf16" if c["act"] == "bf16" else ""
    if c["kind"] == "act":
        g, u = st["x"][:, :K], st["x"][:, K:]
        f = q4.Q4_ACT_GELU if c["f"] == "gelu" else q4.Q4_ACT_SILU
        if c["out"] == "q8":
            getattr(q4, "q8_act" + tail)(g, u, st["q"], M, K, f)
            return [_values_of(st["q"])]
        if c["out"] == "f8":
            getattr(q4, "f8_act" + tail)(g, u, st["q"], st["s"], M, K, f)
            return [st["q"], st["s"]]
        getattr(q4, "q4_act" + tail)(g, u, st["y"], M, K, f)
        return [st["y"]]
    more = {"residual": st["residual"], "sum": st["sum"], "weights": st["weights"], "share": c["share"]}
    if c["out"] == "q8":
        getattr(q4, "q8_norm" + tail)(st["x"], st["gamma"], st["q"], M, K, EPS, y=st["dense"], **more)
        out = [_values_of(st["q"])]
    elif c["out"] == "f8":
        getattr(q4, "f8_norm" + tail)(st["x"], st["gamma"], st["q"], st["s"], M, K, EPS, y=st["dense"], **more)
        out = [st["q"], st["s"]]
    else:
        getattr(q4, "q4_norm" + tail)(st["x"], st["gamma"], st["y"], M, K, EPS, **more)
        out = [st["y"]]
    return out + [t for t in (st["dense"], st["sum"]) if t is not None]


# ---------------------------------------------------------------------------
# The definitions, in 64 bits.

def _exact_written(y, out):
    M, K = y.shape
    if out in ("f32", "bf16"):
        return [y]
    wide = 32 if out == "q8" else 128
    n = -(-K // wide)
    d = torch.stack([y[:, wide * b:wide * b + wide].abs().amax(1) for b in range(n)], 1) / (127 if out == "q8" else E4M3_MAX)
    at = torch.arange(K, device=y.device) // wide
    v = y / torch.where(d == 0, torch.ones_like(d), d)[:, at]
    if out == "q8":
        half_up = torch.where(v < 0, torch.ceil(v - 0.5), torch.floor(v + 0.5))
        return [(half_up * d.to(torch.float16).double()[:, at]).reshape(M, n, 32)]
    # E4M3: three fraction bits, exponents from 2^-6, steps of 2^-9 below.
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return [torch.round(v / step) * step, d]


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["kind"] == "route":
        T, E, G, k = c["T"], c["E"], c["n_groups"], c["top_k"]
        x = st["logits"].double().cpu()
        s = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
        key = s + (st["bias"].double().cpu() if c["bias"] else 0.0)
        size = E // G
        rank = torch.zeros(T, G, dtype=torch.float64)
        for g in range(G):
            rank[:, g] = torch.topk(key[:, g * size:(g + 1) * size], c["group_best"], 1)[0].sum(1)
        left = torch.full_like(key, -math.inf)
        for _ in range(c["top_groups"]):       # the best group left, the lowest among equal ones
            best = (rank == rank.amax(1, keepdim=True)).to(torch.uint8).argmax(1)
            rank.scatter_(1, best[:, None], -math.inf)
            cols = best[:, None] * size + torch.arange(size)[None, :]
            left.scatter_(1, cols, key.gather(1, cols))
        ids = torch.empty(T, k, dtype=torch.long)
        for j in range(k):
            ids[:, j] = (left == left.amax(1, keepdim=True)).to(torch.uint8).argmax(1)
            left.scatter_(1, ids[:, j:j + 1], -math.inf)
        w = s.gather(1, ids)
        w = (w / w.sum(1, keepdim=True) if c["renorm"] else w) * c["scale"]
        slots = [[] for _ in range(E)]
        for r, e in enumerate(ids.reshape(-1).tolist()):
            slots[e].append(r)
        ends = [0]
        for one in slots:
            ends.append(ends[-1] + len(one))
        return [ids.reshape(-1).to(torch.int32), w.reshape(-1), torch.tensor(ends, dtype=torch.int32), torch.tensor([r for one in slots for r in one], dtype=torch.int32)]
    M, K = c["M"], c["K"]
    x = st["x"].double()
    if c["kind"] == "act":
        g, u = x[:, :K], x[:, K:]
        if c["f"] == "silu":
            f = g * torch.sigmoid(g)
        else:
            f = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
        return _exact_written(f * u, c["out"])
    h = torch.zeros(M, K, dtype=torch.float64, device=x.device)
    if st["residual"] is not None:
        h += st["residual"].double()
    for j in range(c["share"]):
        row = x[j::c["share"]]
        if st["weights"] is not None:
            w = st["weights"][:, j].double()
            row = torch.where((w == 0)[:, None], torch.zeros_like(row), w[:, None] * row)
        h += row
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * st["gamma"].double()
    out = _exact_written(y, c["out"])
    return out + ([y] if st["dense"] is not None else []) + ([h] if st["sum"] is not None else [])
