"""Cases, inputs and plain forms of the mixture-of-experts and 8-bit operators.

Four operators and the path that joins them, in the forms a served model casts its
gated FFN into: the router's choice (``route``), the products grouped by expert with
ragged sizes (``grouped_matmul``, bf16 and int8), per-token int8 codes
(``quantize_tokens``) with the product that takes them (``matmul_int8``), and the gated
experts' forward (``experts_forward``) behind the router.

With ``own`` false ``run`` computes an operator with elementary torch operations in
32 bits, rounded once at the end; with ``own`` true it calls the library.  ``exact``
computes the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
#: the gate's shift that leaves about 10 % of a ReLU gate's units live (the 0.9 normal quantile, in bf16)
SHIFT = -1.28125


def listed():
    return [
        # the router of one decoded token: 8 of 64 experts
        {"name": "route_token", "op": "route", "T": 1, "E": 64, "k": 8, "dtype": "f32", "score": "softmax",
         "normalize": True, "masked": 0.0},
        # the router of a long prompt batch over many experts; one expert in ten closed for a token (capacity, placement)
        {"name": "route_prompt", "op": "route", "T": 16384, "E": 256, "k": 8, "dtype": "bf16", "score": "sigmoid",
         "normalize": True, "masked": 0.1},
        # activations of a decode batch before an int8 product
        {"name": "quantize_decode", "op": "quantize", "T": 64, "K": 2560},
        # the FFN's hidden activations of a prompt batch, the widest rows of the D = 4096 layer
        {"name": "quantize_prompt", "op": "quantize", "T": 8192, "K": 14336},
        # one decoded token through an int8 up projection of the D = 2560 layer
        {"name": "int8_token", "op": "int8", "T": 1, "N": 7168, "K": 2560, "out": "bf16"},
        # an odd decode batch through its int8 down projection (few output rows, a long sum), fp32 out
        {"name": "int8_batch", "op": "int8", "T": 77, "N": 2560, "K": 7168, "out": "f32"},
        # a prompt batch through an int8 up projection of the D = 4096 layer
        {"name": "int8_prompt", "op": "int8", "T": 8192, "N": 14336, "K": 4096, "out": "bf16"},
        # decode: 32 tokens' choices spread over 64 experts, two rows each on average, some experts idle
        {"name": "grouped_decode", "op": "grouped", "R": 128, "E": 64, "N": 1024, "K": 2560, "type": "bf16",
         "skew": 1.0},
        # a prompt batch: ragged groups from a handful of rows to a thousand and more
        {"name": "grouped_prompt", "op": "grouped", "R": 16384, "E": 64, "N": 7168, "K": 2560, "type": "bf16",
         "skew": 0.7},
        # int8 experts, odd row count and widths: a mixed batch of prompts and decodes
        {"name": "grouped_int8", "op": "grouped", "R": 4093, "E": 16, "N": 1000, "K": 2560, "type": "int8",
         "skew": 0.7},
        # one decoded token through 8 of 64 fine-grained cast experts (90 % of the gate dead)
        {"name": "experts_token", "op": "experts", "T": 1, "E": 64, "k": 8, "D": 2560, "H": 1024, "act": "relu"},
        # a prompt batch through the same layer
        {"name": "experts_prompt", "op": "experts", "T": 4096, "E": 64, "k": 8, "D": 2560, "H": 1024, "act": "relu"},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number spread over the logarithm of [lo, hi], a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    most = work({"op": "int8", "T": 8192, "N": 14336, "K": 4096, "out": "bf16"})["flops"]
    while True:
        op = rng.choice(("route", "quantize", "int8", "grouped", "experts"))
        if op == "route":
            E = _log(rng, 4, 256)
            c = {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E)),
                 "dtype": rng.choice(("f32", "bf16")), "score": rng.choice(("softmax", "sigmoid")),
                 "normalize": rng.random() < 0.7, "masked": rng.choice((0.0, 0.1, 0.5))}
        elif op == "quantize":
            c = {"op": op, "T": _log(rng, 1, 8192), "K": _log(rng, 16, 14336)}
        elif op == "int8":
            c = {"op": op, "T": _log(rng, 1, 8192), "N": _log(rng, 16, 14336), "K": _log(rng, 64, 14336, 16),
                 "out": rng.choice(("bf16", "f32"))}
        elif op == "grouped":
            t = rng.choice(("bf16", "int8"))
            c = {"op": op, "R": _log(rng, 1, 16384), "E": _log(rng, 2, 128), "N": _log(rng, 16, 7168),
                 "K": _log(rng, 64, 7168, 8 if t == "bf16" else 16), "type": t, "skew": round(rng.uniform(0, 1.2), 2)}
            if c["E"] * c["N"] * c["K"] > 64 * 7168 * 2560:
                continue
        else:
            E = _log(rng, 4, 128)
            c = {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, min(8, E)),
                 "D": _log(rng, 128, 4096, 8), "H": _log(rng, 64, 4096), "act": rng.choice(("relu", "rsp", "silu"))}
            if c["E"] * c["D"] * c["H"] > 64 * 2560 * 1024 * 2:
                continue
        if work(c)["flops"] <= most:
            return c


def _busy(E, picks, k):
    """Experts that `picks` tokens of k choices each are expected to reach."""
    return E * (1 - (1 - k / E) ** picks)


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # logits in; weights, ids and rows out, and the offsets; a compare per logit and choice, an exp per logit
        return {"bytes": T * E * (4 if case["dtype"] == "f32" else 2) + T * k * 12 + (E + 1) * 4,
                "flops": T * E * (k + 4)}
    if op == "quantize":
        T, K = case["T"], case["K"]
        return {"bytes": T * K * 3 + T * 4, "flops": 3 * T * K}
    if op == "int8":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": T * K + N * K + T * N * (2 if case["out"] == "bf16" else 4) + 4 * (T + N),
                "flops": 2 * T * N * K}
    if op == "grouped":
        R, E, N, K = case["R"], case["E"], case["N"], case["K"]
        b = 2 if case["type"] == "bf16" else 1
        return {"bytes": R * K * b + _busy(E, R, 1) * N * K * b + R * N * 2, "flops": 2 * R * N * K}
    T, E, k, D, H = case["T"], case["E"], case["k"], case["D"], case["H"]
    # the gate W1 of the chosen experts in full; of W3 and W2 the rows of units that are live for some token
    # (10 % of a token's units with the shifted ReLU and R-S+ gates, all with SiLU); a tile of many tokens has no
    # dead unit, so the operations are the dense formula's
    live = 1.0 if case["act"] == "silu" else 1 - 0.9 ** max(1.0, T * k / E)
    return {"bytes": _busy(E, T, k) * H * D * 2 * (1 + 2 * live) + T * D * 4 + T * E * 4,
            "flops": 6 * T * k * H * D * (1.0 if T * k > 8 * E else (1 + 2 * live) / 3)}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 2654435761 % (1 << 62) + 17)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _logits(g, T, E, masked, dtype):
    z = _randn(g, T, E) + 0.5 * _randn(g, E)  # some experts are favoured
    if masked:
        z = z.masked_fill(torch.rand(T, E, generator=g, device=DEV) < masked, -math.inf)
        z[T // 2] = -math.inf  # a token whose mask leaves no expert
    return z.to(torch.float32 if dtype == "f32" else BF)


def _int8(g, rows, K):
    """Codes and scales as a symmetric quantiser makes them of normal values (the largest code of a row is near 127)."""
    q = (_randn(g, rows, K) * 32).round_().clamp_(-127, 127).to(torch.int8)
    return q, torch.rand(rows, generator=g, device=DEV) * 0.02 + 0.01


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "route":
        s["logits"] = _logits(g, case["T"], case["E"], case["masked"], case["dtype"])
    elif op == "quantize":
        x = _randn(g, case["T"], case["K"], dtype=BF)
        x *= (0.25 + 4 * torch.rand(case["T"], 1, generator=g, device=DEV)).to(BF)
        x[:, case["K"] // 3] *= 8  # an outlier channel
        if case["T"] > 2:
            x[case["T"] // 2] = 0  # a padded token
        s["x"] = x
    elif op == "int8":
        s["xq"], s["sx"] = _int8(g, case["T"], case["K"])
        s["wq"], s["sw"] = _int8(g, case["N"], case["K"])
        s["sw"] /= case["K"] ** 0.5
    elif op == "grouped":
        R, E, N, K = case["R"], case["E"], case["N"], case["K"]
        p = torch.exp(case["skew"] * _randn(g, E))
        picks = torch.multinomial(p, R, replacement=True, generator=g)
        counts = torch.bincount(picks, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["bounds"] = s["offsets"].tolist()
        if case["type"] == "bf16":
            s["x"], s["w"] = _randn(g, R, K, dtype=BF), _randn(g, E, N, K, dtype=BF)
            s["w"] *= K ** -0.5
        else:
            s["x"], s["sx"] = _int8(g, R, K)
            w, sw = _int8(g, E * N, K)
            s["w"], s["sw"] = w.view(E, N, K), sw.view(E, N) / K ** 0.5
    else:
        T, E, D, H = case["T"], case["E"], case["D"], case["H"]
        x = _randn(g, T, D, dtype=BF)
        x[:, -1] = 1
        W1, W3, W2t = (_randn(g, E, H, D, dtype=BF) for _ in range(3))
        W1 *= D ** -0.5
        W3 *= D ** -0.5
        W2t *= H ** -0.5
        if case["act"] != "silu":
            W1[:, :, -1] = SHIFT  # the gate's bias, carried by the channel that is 1
        s.update(x=x, W1=W1, W3=W3, W2t=W2t, logits=_logits(g, T, E, 0.0, "f32"))
    return s


# ---------------------------------------------------------------- the plain forms


def _chosen(logits, k, score, normalize):
    """Weights [T, k] and expert of each choice [T, k] (-1: no expert open), the largest first, ties to the lowest index."""
    z, ids = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    z, ids = z[:, :k], ids[:, :k]
    shut = z == -math.inf
    if score == "softmax":
        top = logits.float().amax(1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        w = torch.exp(z - top)
        total = w.sum(1, keepdim=True) if normalize else torch.exp(logits.float() - top).sum(1, keepdim=True)
    else:
        w = 1 / (1 + torch.exp(-z))
        total = w.sum(1, keepdim=True) if normalize else torch.ones_like(w[:, :1])
    w = torch.where(shut, torch.zeros_like(w), w / torch.where(total > 0, total, torch.ones_like(total)))
    return w, torch.where(shut, torch.full_like(ids, -1), ids)


def _grouping(ids, E):
    """offsets [E + 1], and for each grouped row the choice (token * k + place) that it serves, -1 past the last."""
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    rows = torch.argsort(key, stable=True)
    counts = (key[:, None] == torch.arange(E, device=key.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rows = torch.where(torch.arange(flat.numel(), device=rows.device) < offsets[-1], rows, torch.full_like(rows, -1))
    return offsets.to(torch.int32), rows.to(torch.int32)


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    v = z / (1 + torch.exp(-z))
    return v if act == "silu" else torch.where(z > 0, v, torch.zeros_like(v))


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        w, ids = _chosen(s["logits"], c["k"], c["score"], c["normalize"])
        offsets, rows = _grouping(ids, c["E"])
        return w, ids.to(torch.int32), offsets, rows
    if op == "quantize":
        x = s["x"].float()
        amax = x.abs().amax(1)
        scale = amax / torch.full_like(amax, 127)  # a tensor on both sides: the correctly rounded quotient
        q = x / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
        return q.round().clamp(-127, 127).to(torch.int8), scale
    if op == "int8":
        y = (s["xq"].float() @ s["wq"].float().T) * s["sx"][:, None] * s["sw"]
        return y if c["out"] == "f32" else y.to(BF)
    if op == "grouped":
        y = torch.empty(c["R"], c["N"], dtype=BF, device=DEV)
        b = s["bounds"]
        for e in range(c["E"]):
            if b[e] < b[e + 1]:
                v = s["x"][b[e]:b[e + 1]].float() @ s["w"][e].float().T
                y[b[e]:b[e + 1]] = v if c["type"] == "bf16" else v * s["sx"][b[e]:b[e + 1], None] * s["sw"][e]
        return y
    # the gated experts, one choice after another where there are few tokens, one expert after another else
    w, ids = _chosen(s["logits"], c["k"], "softmax", True)
    x = s["x"].float()
    y = torch.zeros_like(x)
    if c["T"] * c["k"] <= c["E"]:
        for j in range(c["k"]):
            e = ids[:, j]
            z = (s["W1"][e].float() @ x[:, :, None])[:, :, 0]
            u = (s["W3"][e].float() @ x[:, :, None])[:, :, 0]
            y += w[:, j:j + 1] * ((_act(z, c["act"]) * u)[:, None] @ s["W2t"][e].float())[:, 0]
        return y.to(BF)
    for e in range(c["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = _act(x[t] @ s["W1"][e].float().T, c["act"]) * (x[t] @ s["W3"][e].float().T)
        y.index_add_(0, t, w[t, j, None] * (h @ s["W2t"][e].float()))
    return y.to(BF)


def run(state):
    if not own:
        return _plain(state)
    import activation_sparse_gated_gb300 as sffn
    c = state["case"]
    op = c["op"]
    if op == "route":
        return tuple(sffn.route(state["logits"], c["k"], score=c["score"], normalize=c["normalize"]))
    if op == "quantize":
        return sffn.quantize_tokens(state["x"])
    if op == "int8":
        return sffn.matmul_int8(state["xq"], state["sx"], state["wq"], state["sw"], dtype=c["out"])
    if op == "grouped":
        return sffn.grouped_matmul(state["x"], state["w"], state["offsets"], sx=state.get("sx"), sw=state.get("sw"))
    routing = sffn.route(state["logits"], c["k"], score="softmax", normalize=True)
    return sffn.experts_forward(state["x"], routing, state["W1"], state["W3"], state["W2t"], act=c["act"])


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("route", "experts"):
        k, E, T = case["k"], case["E"], case["T"]
        z = s["logits"].double()
        # an expert's rank: how many others beat it (a larger logit, or the same with a lower index)
        ids = torch.full((T, k), -1, dtype=torch.int64, device=DEV)
        val = torch.full((T, k), -math.inf, dtype=torch.float64, device=DEV)
        left = z.clone()
        at = torch.arange(E, device=DEV)
        for j in range(k):
            v = left.amax(1)
            e = torch.where(left == v[:, None], at, torch.full_like(at, E)).amin(1)
            is_open = v > -math.inf
            ids[:, j] = torch.where(is_open, e, torch.full_like(e, -1))
            val[:, j] = v
            left[torch.arange(T, device=DEV), e] = -math.inf
        picked = ids >= 0
        if op == "experts" or case["score"] == "softmax":
            base = val if op == "experts" or case["normalize"] else z
            norm = torch.logsumexp(torch.where(torch.isfinite(base), base, torch.full_like(base, -1e300)), 1)
            w = torch.exp(val - norm[:, None])
        else:
            w = torch.sigmoid(val)
            if case["normalize"]:
                total = w.sum(1, keepdim=True)
                w = w / torch.where(total > 0, total, torch.ones_like(total))
        w = torch.where(picked, w, torch.zeros_like(w))
        if op == "route":
            flat = ids.reshape(-1).cpu()
            groups = [torch.nonzero(flat == e).reshape(-1) for e in range(E)]
            offsets = torch.tensor([0] + [len(x) for x in groups]).cumsum(0).to(torch.int32)
            rows = torch.cat(groups)
            rows = torch.cat([rows, torch.full((T * k - len(rows),), -1)]).to(torch.int32)
            return w, ids.to(torch.int32), offsets.to(DEV), rows.to(DEV)
        x, y = s["x"].double(), torch.zeros(T, case["D"], dtype=torch.float64, device=DEV)
        for e in range(E):
            m = ids == e
            t = torch.nonzero(m.any(1)).reshape(-1)
            if len(t):
                g = x[t] @ s["W1"][e].double().T
                a = torch.relu(g) if case["act"] == "relu" else g * torch.sigmoid(g)
                if case["act"] == "rsp":
                    a = a * (g > 0)
                a *= x[t] @ s["W3"][e].double().T
                y[t] += (w * m)[t].sum(1)[:, None] * (a @ s["W2t"][e].double())
        return y
    if op == "quantize":
        # the scale is held in binary32 and the codes are decided in it, by definition
        x = s["x"].float().cpu().numpy()
        amax = abs(x).max(1)
        scale = amax / amax.dtype.type(127)
        q = (x / (scale + (scale == 0))[:, None]).round()
        return torch.from_numpy(q).to(torch.int8), torch.from_numpy(scale)
    if op == "int8":
        y = s["xq"].double() @ s["wq"].double().T
        return y.mul_(s["sx"].double()[:, None]).mul_(s["sw"].double())
    y = torch.zeros(case["R"], case["N"], dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        rows = slice(s["bounds"][e], s["bounds"][e + 1])
        y[rows] = s["x"][rows].double() @ s["w"][e].double().T
        if case["type"] == "int8":
            y[rows] *= torch.outer(s["sx"][rows].double(), s["sw"][e].double())
    return y
