"""The operators of a mixture-of-experts feed-forward layer over block-quantized
weights, as measured cases: the 8-bit floating-point quantizer, the 8-bit
product with a scale for each block of 128, the router, and the products
grouped by expert.

`run` makes one pass through an operator: with ``own`` false in elementary
torch operations (32-bit), with ``own`` true through this package's binding.
`exact` computes the same outputs from the definitions in 64 bits.

Kinds of case:
  quantize  f32 or bfloat16 [M, K] -> E4M3 codes and one f32 scale per block of
            128 columns of a row (block_rows 1) or per 128 x 128 tile (128).
  product   y[m, n] = sum_b as[m, b] ws[n / 128, b] sum_{k in b} a[m, k] w[n, k],
            y in bfloat16 (the type the next layer's quantizer reads).
  route     logits [T, E] -> the top_k experts of each token, their softmax
            weights, and the slots (t, j) sorted by expert.
  grouped   y[r] = a[r / share] @ dequant(W[expert of r])^T for the slots r of
            each expert, the weights Q4_0 or Q8_0 (y in f32), or E4M3 with
            128 x 128 scales (y in bfloat16).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK_BYTES = {"q4": 18, "q8": 34}


# ---------------------------------------------------------------------------
# Cases. Sizes: the 4096- and 14336-wide projections that this repository's
# benchmark multiplies, and 1792, one eighth of the wider one.

def listed():
    return [
        # The activations of a 2048-token prompt before an 8-bit product.
        {"name": "quantize rows bf16 2048x4096", "kind": "quantize", "M": 2048, "K": 4096, "block_rows": 1, "act": "bf16"},
        # A weight matrix quantized once when a model is loaded.
        {"name": "quantize tiles f32 14336x4096", "kind": "quantize", "M": 14336, "K": 4096, "block_rows": 128, "act": "f32"},
        # One token through an attention projection: latency and the weight's bytes.
        {"name": "f8 product 1x4096x4096", "kind": "product", "M": 1, "N": 4096, "K": 4096},
        # A batch of 40 sequences decoding through a down projection.
        {"name": "f8 product 40x4096x14336", "kind": "product", "M": 40, "N": 4096, "K": 14336},
        # A prompt of odd length through an attention projection.
        {"name": "f8 product 1001x4096x4096", "kind": "product", "M": 1001, "N": 4096, "K": 4096},
        # A 2048-token prompt through an up projection.
        {"name": "f8 product 2048x14336x4096", "kind": "product", "M": 2048, "N": 14336, "K": 4096},
        # A decoding batch at the router of 8 experts.
        {"name": "route 32 tokens 2 of 8", "kind": "route", "T": 32, "E": 8, "top_k": 2, "renorm": True},
        # A long prompt at the router of many small experts.
        {"name": "route 8192 tokens 6 of 64", "kind": "route", "T": 8192, "E": 64, "top_k": 6, "renorm": True},
        # One token through its two experts, f32 activations, 4-bit weights.
        {"name": "grouped q4 f32 1 token", "kind": "grouped", "fmt": "q4", "act": "f32", "T": 1, "E": 8, "top_k": 2, "share": 2, "N": 4096, "K": 4096, "skew": 1.0},
        # A batch of 37 decoding tokens: a few rows for every expert.
        {"name": "grouped q4 bf16 37 tokens", "kind": "grouped", "fmt": "q4", "act": "bf16", "T": 37, "E": 8, "top_k": 2, "share": 2, "N": 14336, "K": 4096, "skew": 0.5},
        # A 2048-token prompt through the experts' up projections, unevenly routed.
        {"name": "grouped q4 bf16 2048 tokens", "kind": "grouped", "fmt": "q4", "act": "bf16", "T": 2048, "E": 8, "top_k": 2, "share": 2, "N": 14336, "K": 4096, "skew": 0.5},
        # A 1024-token prompt through the down projections of 32 narrow 8-bit experts, some of them empty.
        {"name": "grouped f8 1024 tokens 4 of 32", "kind": "grouped", "fmt": "f8", "act": "f8", "T": 1024, "E": 32, "top_k": 4, "share": 1, "N": 4096, "K": 1792, "skew": 1.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quantize", "product", "product", "route", "grouped", "grouped", "grouped"])
    if kind == "quantize":
        return {"kind": kind, "M": _log(rng, 1, 4096), "K": 32 * _log(rng, 4, 256), "block_rows": rng.choice([1, 1, 128]), "act": rng.choice(["f32", "bf16"])}
    if kind == "product":
        return {"kind": kind, "M": _log(rng, 1, 2048), "N": _log(rng, 200, 8192), "K": 32 * _log(rng, 8, 256)}
    if kind == "route":
        E = rng.choice([8, 16, 40, 64, 128, 200])
        return {"kind": kind, "T": _log(rng, 1, 8192), "E": E, "top_k": rng.choice([1, 2, 4, 6, 8]), "renorm": rng.random() < 0.7}
    fmt = rng.choice(["q4", "q8", "f8"])
    E = rng.choice([4, 8, 16, 32])
    k = rng.choice([1, 2, 4])
    wide = 64 if fmt != "f8" else 32
    return {"kind": kind, "fmt": fmt, "act": "f8" if fmt == "f8" else rng.choice(["f32", "bf16"]), "T": _log(rng, 1, 1024), "E": E, "top_k": k,
            "share": rng.choice([1, k]), "N": _log(rng, 128, 4096), "K": wide * _log(rng, 4, 4096 // wide), "skew": rng.choice([0.0, 0.5, 1.5])}


def work(case):
    c = case
    if c["kind"] == "quantize":
        n, rows = c["M"] * c["K"], -(-c["M"] // c["block_rows"])
        return {"bytes": n * (4 if c["act"] == "f32" else 2) + n + 4 * rows * -(-c["K"] // 128), "flops": 3 * n}
    if c["kind"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        kb = -(-K // 128)
        return {"bytes": M * K + 4 * M * kb + N * K + 4 * -(-N // 128) * kb + 2 * M * N, "flops": 2 * M * N * K}
    if c["kind"] == "route":
        S = c["T"] * c["top_k"]
        return {"bytes": 4 * c["T"] * c["E"] + 12 * S + 4 * (c["E"] + 1), "flops": 4 * c["T"] * c["E"]}
    S, N, K = c["T"] * c["top_k"], c["N"], c["K"]
    hit = min(c["E"], S)     # experts with a row, at most: each one's weights are read once
    if c["fmt"] == "f8":
        kb = -(-K // 128)
        per_w, per_a, out = N * K + 4 * -(-N // 128) * kb, K + 4 * kb, 2
    else:
        per_w, per_a, out = N * (K // 32) * BLOCK_BYTES[c["fmt"]], K * (4 if c["act"] == "f32" else 2), 4
    return {"bytes": hit * per_w + S // c["share"] * per_a + out * S * N + 4 * (S + c["E"] + 1), "flops": 2 * S * N * K}


# ---------------------------------------------------------------------------
# What a program has in hand before the call.

def _blocks_of_128(x, rows):
    """x [M, K] -> the [M / rows, rows, K / 128, 128] view of its zero-padded copy."""
    M, K = x.shape
    Mp, Kp = -(-M // rows) * rows, -(-K // 128) * 128
    if (Mp, Kp) != (M, K):
        x = torch.nn.functional.pad(x, (0, Kp - K, 0, Mp - M))
    return x.reshape(Mp // rows, rows, Kp // 128, 128)


def _quantize(x, rows):
    """E4M3 codes (as torch.float8_e4m3fn) and scales of x [M, K] in f32: scale = max|x| / 448 over the block, code = round(x / scale)."""
    M, K = x.shape
    b = _blocks_of_128(x.float(), rows)
    s = b.abs().amax(dim=(1, 3)) / E4M3_MAX
    d = torch.where(s == 0, torch.ones_like(s), s)[:, None, :, None]
    q = (b / d).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    q = q.reshape(b.shape[0] * rows, -1)[:M, :K].contiguous()
    return q, s.contiguous()


def _spread(s, rows, M, K, dtype):
    """Scales [M / rows, K / 128] -> one value for each element of [M, K]."""
    return s.to(dtype).repeat_interleave(rows, 0)[:M].repeat_interleave(128, 1)[:, :K]


def _gguf(x, fmt):
    """x [R, K] in f32 -> the Q4_0 or Q8_0 block bytes [R, K / 32, 18 or 34]."""
    b = x.reshape(x.shape[0], -1, 32)
    if fmt == "q4":
        at = b.abs().argmax(-1, keepdim=True)
        d = b.gather(-1, at) / -8
        q = torch.where(d == 0, torch.full_like(b, 8.0), b / torch.where(d == 0, torch.ones_like(d), d) + 8.5).clamp(0, 15).to(torch.uint8)
        q = q[..., :16] | (q[..., 16:] << 4)
    else:
        d = b.abs().amax(-1, keepdim=True) / 127
        q = torch.round(b / torch.where(d == 0, torch.ones_like(d), d)).to(torch.int8).view(torch.uint8)
    return torch.cat([d.to(torch.float16).view(torch.uint8), q], -1).contiguous()


def _ungguf(w, fmt, dtype):
    """Block bytes [..., K / 32, 18 or 34] -> values [..., K]."""
    d = w[..., :2].contiguous().view(torch.float16).to(dtype)
    if fmt == "q4":
        q = torch.cat([w[..., 2:] & 15, w[..., 2:] >> 4], -1).to(dtype) - 8
    else:
        q = w[..., 2:].contiguous().view(torch.int8).to(dtype)
    return (q * d).flatten(-2)


def _activations(g, M, K, dev):
    """Hidden states: N(0, 1) with a few channels of larger spread and rows of differing size, as normed activations have."""
    x = torch.randn(M, K, generator=g, device=dev)
    x *= 1 + 9 * (torch.rand(1, K, generator=g, device=dev) < 0.01)
    return x * torch.exp(0.5 * torch.randn(M, 1, generator=g, device=dev))


def _group(ids, E):
    """Expert of each slot -> offsets [E + 1] and the slots in expert order, both int32; equal experts keep their order."""
    order = torch.sort(ids, stable=True)[1].to(torch.int32)
    bounds = torch.arange(E + 1, device=ids.device)
    offsets = (ids[None, :] < bounds[:, None]).sum(1).to(torch.int32)
    return offsets, order


def _logits(g, T, E, skew, dev):
    return torch.randn(T, E, generator=g, device=dev) + skew * torch.randn(1, E, generator=g, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c = case
    st = {"case": c}
    if c["kind"] == "quantize":
        x = _activations(g, c["M"], c["K"], dev) if c["block_rows"] == 1 else 0.02 * torch.randn(c["M"], c["K"], generator=g, device=dev)
        st["x"] = x.to(torch.bfloat16) if c["act"] == "bf16" else x
        rows = -(-c["M"] // c["block_rows"])
        st["q"] = torch.empty(c["M"], c["K"], dtype=torch.float8_e4m3fn, device=dev)
        st["s"] = torch.empty(rows, -(-c["K"] // 128), device=dev)
    elif c["kind"] == "product":
        st["a"], st["a_s"] = _quantize(_activations(g, c["M"], c["K"], dev), 1)
        st["w"], st["w_s"] = _quantize(0.02 * torch.randn(c["N"], c["K"], generator=g, device=dev), 128)
        st["y"] = torch.empty(c["M"], c["N"], dtype=torch.bfloat16, device=dev)
    elif c["kind"] == "route":
        # Router outputs are often computed in bfloat16: equal logits occur.
        st["logits"] = _logits(g, c["T"], c["E"], 0.5, dev).to(torch.bfloat16).float()
        S = c["T"] * c["top_k"]
        st["ids"] = torch.empty(S, dtype=torch.int32, device=dev)
        st["weights"] = torch.empty(S, device=dev)
        st["offsets"] = torch.empty(c["E"] + 1, dtype=torch.int32, device=dev)
        st["order"] = torch.empty(S, dtype=torch.int32, device=dev)
    else:
        E, N, K, S = c["E"], c["N"], c["K"], c["T"] * c["top_k"]
        ids = torch.sort(_logits(g, c["T"], E, c["skew"], dev), dim=1, descending=True, stable=True)[1][:, :c["top_k"]].reshape(-1)
        st["offsets"], st["order"] = _group(ids, E)
        x = _activations(g, S // c["share"], K, dev)
        if c["fmt"] == "f8":
            st["a"], st["a_s"] = _quantize(x, 1)
            Nb, Kb = -(-N // 128), -(-K // 128)
            st["w"] = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device=dev)
            st["w_s"] = torch.empty(E, Nb, Kb, device=dev)
            for e in range(E):
                st["w"][e], st["w_s"][e] = _quantize(0.02 * torch.randn(N, K, generator=g, device=dev), 128)
        else:
            st["a"] = x.to(torch.bfloat16) if c["act"] == "bf16" else x
            st["w"] = torch.empty(E, N, K // 32, BLOCK_BYTES[c["fmt"]], dtype=torch.uint8, device=dev)
            for e in range(E):
                st["w"][e] = _gguf(0.02 * torch.randn(N, K, generator=g, device=dev), c["fmt"])
        st["y"] = torch.empty(S, N, dtype=torch.bfloat16 if c["fmt"] == "f8" else torch.float32, device=dev)
    return st


# ---------------------------------------------------------------------------
# One pass.

def run(state):
    st, c = state, state["case"]
    if own:
        return _run_own(st, c)
    if c["kind"] == "quantize":
        return list(_quantize(st["x"], c["block_rows"]))
    if c["kind"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        a = st["a"].float() * _spread(st["a_s"], 1, M, K, torch.float32)
        w = st["w"].float() * _spread(st["w_s"], 128, N, K, torch.float32)
        return (a @ w.t()).to(torch.bfloat16)
    if c["kind"] == "route":
        x = st["logits"]
        top, ids = torch.sort(x, dim=1, descending=True, stable=True)
        top, ids = top[:, :c["top_k"]], ids[:, :c["top_k"]].reshape(-1)
        e = torch.exp(top - x.amax(1, keepdim=True))
        total = e.sum(1, keepdim=True) if c["renorm"] else torch.exp(x - x.amax(1, keepdim=True)).sum(1, keepdim=True)
        offsets, order = _group(ids, c["E"])
        return [ids.to(torch.int32), (e / total).reshape(-1), offsets, order]
    return _grouped(st, c)


def _grouped(st, c):
    """The experts that have rows, their rows padded to the longest one's, one batched product."""
    E, N, K = c["E"], c["N"], c["K"]
    off, order = st["offsets"].long(), st["order"].long()
    counts = off[1:] - off[:-1]
    hit = counts.nonzero().flatten()
    at = torch.arange(int(counts.max()), device=off.device)[None, :]
    there = at < counts[hit][:, None]
    rows = order[torch.where(there, off[:-1][hit][:, None] + at, 0)]
    if c["fmt"] == "f8":
        a = st["a"].float() * _spread(st["a_s"], 1, st["a"].shape[0], K, torch.float32)
        w = st["w"].view(torch.uint8)[hit].view(torch.float8_e4m3fn).float() * st["w_s"][hit].repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    else:
        a = st["a"].float()
        w = _ungguf(st["w"][hit], c["fmt"], torch.float32)
    x = a[rows // c["share"]].transpose(1, 2).contiguous()
    out = torch.bmm(w, x).transpose(1, 2)
    y = torch.empty(order.numel(), N, dtype=st["y"].dtype, device=off.device)
    y[rows[there]] = out[there].to(y.dtype)
    return y


def _run_own(st, c):
    from block_quantized_weight_dequant_amd import binding as q4
    if c["kind"] == "quantize":
        f = q4.f8_quantize_bf16 if c["act"] == "bf16" else q4.f8_quantize
        f(st["x"], st["q"], st["s"], c["M"], c["K"], c["block_rows"])
        return [st["q"], st["s"]]
    if c["kind"] == "product":
        f = q4.f8_gemv if c["M"] <= q4.Q4_GEMV_MAX_ROWS else q4.f8_gemm
        f(st["a"], st["a_s"], st["w"], st["w_s"], st["y"], c["M"], c["N"], c["K"])
        return st["y"]
    if c["kind"] == "route":
        q4.q4_route(st["logits"], st["ids"], st["weights"], st["offsets"], st["order"], c["T"], c["E"], c["top_k"], c["renorm"])
        return [st["ids"], st["weights"], st["offsets"], st["order"]]
    S = c["T"] * c["top_k"]
    if c["fmt"] == "f8":
        q4.f8_gemm_grouped(st["a"], st["a_s"], st["w"], st["w_s"], st["offsets"], st["order"], st["y"], c["E"], S, c["N"], c["K"], share=c["share"])
    else:
        f = getattr(q4, c["fmt"] + "_gemm_grouped" + ("_bf16" if c["act"] == "bf16" else ""))
        f(st["a"], st["w"], st["offsets"], st["order"], st["y"], c["E"], S, c["N"], c["K"], share=c["share"])
    return st["y"]


# ---------------------------------------------------------------------------
# The definitions, in 64 bits.

def exact(case, seed):
    c, st = case, prepare(case, seed)
    f64 = torch.float64
    if c["kind"] == "quantize":
        M, K = c["M"], c["K"]
        x = st["x"].to(f64)
        R, C = -(-M // c["block_rows"]), -(-K // 128)
        s = torch.zeros(R, C, dtype=f64, device=x.device)
        for b in range(C):
            col = x[:, 128 * b:128 * b + 128].abs().amax(1)
            s[:, b] = torch.nn.functional.pad(col, (0, R * c["block_rows"] - M)).reshape(R, -1).amax(1) / E4M3_MAX
        d = s.repeat_interleave(c["block_rows"], 0)[:M].repeat_interleave(128, 1)[:, :K]
        v = x / torch.where(d == 0, torch.ones_like(d), d)
        # E4M3: three fraction bits, exponents from 2^-6, steps of 2^-9 below.
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        return [torch.round(v / step) * step, s]
    if c["kind"] == "product":
        y = torch.zeros(c["M"], c["N"], dtype=f64, device=st["a"].device)
        n_block = torch.arange(c["N"], device=y.device) // 128
        for b in range(-(-c["K"] // 128)):
            k = slice(128 * b, min(128 * b + 128, c["K"]))
            part = st["a"][:, k].to(f64) @ st["w"][:, k].to(f64).t().contiguous()
            y += part * st["a_s"][:, b].to(f64)[:, None] * st["w_s"][n_block, b].to(f64)[None, :]
        return y
    if c["kind"] == "route":
        x = st["logits"].to(f64).cpu()
        T, E, k = c["T"], c["E"], c["top_k"]
        left, ids = x.clone(), torch.empty(T, k, dtype=torch.long)
        for j in range(k):     # the largest left, the lowest expert among equal ones
            best = left.amax(1, keepdim=True)
            ids[:, j] = (left == best).to(torch.uint8).argmax(1)
            left.scatter_(1, ids[:, j:j + 1], -math.inf)
        p = torch.softmax(x, 1).gather(1, ids)
        if c["renorm"]:
            p = p / p.sum(1, keepdim=True)
        slots = [[] for _ in range(E)]
        for r, e in enumerate(ids.reshape(-1).tolist()):
            slots[e].append(r)
        ends = [0]
        for s in slots:
            ends.append(ends[-1] + len(s))
        return [ids.reshape(-1).to(torch.int32), p.reshape(-1), torch.tensor(ends, dtype=torch.int32), torch.tensor([r for s in slots for r in s], dtype=torch.int32)]
    N, K = c["N"], c["K"]
    y = torch.zeros(c["T"] * c["top_k"], N, dtype=f64, device=st["y"].device)
    off = st["offsets"].tolist()
    for e in range(c["E"]):
        if off[e] == off[e + 1]:
            continue
        rows = st["order"][off[e]:off[e + 1]].long()
        src = torch.div(rows, c["share"], rounding_mode="floor")
        if c["fmt"] == "f8":
            n_block = torch.arange(N, device=y.device) // 128
            k_block = torch.arange(K, device=y.device) // 128
            w = st["w"][e].to(f64) * st["w_s"][e].to(f64)[n_block][:, k_block]
            a = st["a"].view(torch.uint8)[src].view(torch.float8_e4m3fn).to(f64) * st["a_s"][src].to(f64)[:, k_block]
        else:
            b = st["w"][e]
            lo = b[..., 2:].to(f64) if c["fmt"] == "q8" else torch.cat([(b[..., 2:] % 16).to(f64), (b[..., 2:] // 16).to(f64)], -1)
            codes = torch.where(lo > 127, lo - 256, lo) if c["fmt"] == "q8" else lo - 8
            w = (codes * b[..., :2].contiguous().view(torch.float16).to(f64)).reshape(N, K)
            a = st["a"][src].to(f64)
        y[rows] = a @ w.t().contiguous()
    return y
